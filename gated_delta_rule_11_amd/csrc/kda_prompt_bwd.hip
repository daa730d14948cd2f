// kda_prompt_bwd.hip -- gradients of the packed prompts' causal attention.
//
// With P_ij = exp(scale q_i . k_j - lse_i), dP_ij = do_i . v_j, D_i = do_i . o_i,
// dS_ij = P_ij (dP_ij - D_i):
//   dv_j = sum_i P_ij do_i,   dk_j = scale sum_i dS_ij q_i,   dq_i = scale sum_j dS_ij k_j,
// the sums of dk and dv running over the query heads of the group as well.
//
// Two kernels, so that every sum has one owner and a fixed order (no atomics: the same bits every
// time), at the price of forming S and dP twice (seven products instead of five):
//   - dk and dv: a workgroup owns 128 keys of one key head and walks the rows that see them, 64
//     at a time, for every query head of the group; a wavefront owns 32 keys, whose K and V stay
//     in registers;
//   - dq: a workgroup owns 128 rows of one query head and walks the keys as the forward does.
// Both form S and dP with the owned index in the lanes (columns) and the other in the registers
// (rows), so that P and dS are in place as operands of the products that sum over the rows, and
// write their sums transposed.  D comes from a small kernel before.  The sums are fp32; with bf16
// elements P and dS are rounded to bf16 for the products that follow, 2^-8 relative each, as the
// gradients may be.
//
// Measured (bf16, 8192 rows in sequences of 4096, 1023, 2500, 64 and 509, 16 heads on 4, d = 128):
// dk and dv 338 us, dq 194, D 12, the join of the parts 22 (least of 20 calls; on average 360 and 208).
// What bounds the first is its K, V, dK and dV in registers (one wavefront per SIMD): left out, its
// products save 75 us, its exponentials 38, its copies 39, so none of them is hidden completely.  Four
// tiles of rows are in rotation there, read a step before their products; masks are formed without
// branches, and only in the tiles that need them (577 to 382 us).
#include <type_traits>

#include "kda_prompt.hpp"

namespace kda {

namespace {

constexpr int BM = 128;  // owned rows or keys
constexpr int BN = 64;   // walked keys
constexpr int BR = 64;   // walked rows
// D = do . o carries the roundings of o (of its element type, or of the probabilities that a forward with
// bf16 elements formed it from): up to 2^-8 sum |do| |o|, which dP - D does not forgive where few keys hold
// a row's weight, or where the values have much in common.  A row's dS sum to zero, so what they sum to is
// that error: the dq kernel corrects D by it, for dk and dv too, and forms those rows' dq again where it is
// more than this share of sum |dS|, a quarter of what dS may lose to its own rounding.  (Elements in
// fp32 round no dS: every row, when o is bf16.)  Measured, the gradients of the rows above: 537 us where few rows
// need it (530 without the correction; 554 at half this share), 690 where all do (a sink key in every
// sequence).
template <typename T> constexpr float kLeft = sizeof(T) == 2 ? 0.0009765625f : 0.f;

// Asks for N products with V vector instructions, and the LDS reads of two fragments, after each.
template <int N, int V>
__device__ __forceinline__ void interleave() {
  __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
  }
}

// D [n, Hq]: eight lanes a row of a head.
template <typename TO, typename TD>
__global__ __launch_bounds__(256) void prompt_dot_kernel(const PromptBwdArgs a) {
  const TO* o = static_cast<const TO*>(a.o);
  const TD* d_o = static_cast<const TD*>(a.d_o);
  float* D = a.D;
  const int d = a.d;
  const int64_t rows = int64_t(rows_used(a.cu, a.nseq, a.n)) * a.Hq;
  const int64_t r = int64_t(blockIdx.x) * 32 + threadIdx.x / 8;
  const int part = threadIdx.x % 8;
  float s = 0.f;
  if (r < rows)
    for (int c = part * 4; c < d; c += 32)
#pragma unroll
      for (int j = 0; j < 4; ++j) s += io<TO>::load(o, r * d + c + j) * io<TD>::load(d_o, r * d + c + j);
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) s += __shfl_xor(s, x);
  if (r < rows && part == 0) D[r] = s;
}

// Tiles of rows in rotation: one workgroup's registers fill a compute unit, so nothing else hides the
// copies' latency, and the LDS is its own.
template <typename T, int D>
struct KvShape {
  static constexpr int kTile = 2 * BR * D * int(sizeof(T)) + 4 * BR * 4;  // Q, dO, lse, D and two unused
  static constexpr int NS = 4 * kTile <= 160 * 1024 ? 4 : 2;
  static constexpr int kCopies = 2 * BR / (64 / Tile<T, D>::CH * 4) + 1;  // of each wavefront for a tile
  static constexpr size_t lds = size_t(NS) * kTile;
};

template <typename T, typename TG, int D>
__global__ __launch_bounds__(256, 1) void prompt_dkv_kernel(const PromptBwdArgs a) {
  using O = Op<T>;
  using F = typename O::frag;
  using TD = Tile<T, D>;
  constexpr int NK = D / 16, ND = D / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  using W = KvShape<T, D>;
  T* const buf = reinterpret_cast<T*>(smem);                                // [NS][Q tile, dO tile]
  float* const stat = reinterpret_cast<float*>(buf + W::NS * 2 * BR * D);   // [NS][lse, D, unused]

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h2 = lane >> 5, l32 = lane & 31;
  const HeadTile ht = head_tile(blockIdx.x, a.Hkv * a.parts);
  const int kvh = ht.head / a.parts, part = ht.head % a.parts;
  const int c0 = ht.tile * BM;  // keys with the most rows first
  const int used = rows_used(a.cu, a.nseq, a.n);
  if (a.zero_tail && a.parts == 1 && c0 + BM > used) {
    const int first = c0 > used ? c0 : used, last = c0 + BM < a.n ? c0 + BM : a.n;
    zero_rows<TG, D>(static_cast<TG*>(a.dk) + int64_t(kvh) * D, int64_t(a.Hkv) * D, first, last, tid);
    zero_rows<TG, D>(static_cast<TG*>(a.dv) + int64_t(kvh) * D, int64_t(a.Hkv) * D, first, last, tid);
  }
  if (c0 >= used) return;
  const int GP = a.Hq / (a.Hkv * a.parts), h0 = kvh * (a.Hq / a.Hkv) + part * GP;  // this part's query heads
  const int64_t qst = int64_t(a.Hq) * D, kst = int64_t(a.Hkv) * D;

  const int clast = c0 + BM - 1 < used ? c0 + BM - 1 : used - 1;
  const int hi = span_of(a.cu, a.nseq, a.n, clast).end < used ? span_of(a.cu, a.nseq, a.n, clast).end : used;
  const int w0 = c0 + 32 * wave, kj = w0 + l32;
  const int kr = kj < used ? kj : used - 1;
  const int end = span_of(a.cu, a.nseq, a.n, kr).end;
  const int emin = __shfl(end, 0), emax = __shfl(end, 31);
  const int lim = kj < used ? (end < hi ? end : hi) : kj;
  const float c = a.scale * kLog2e;

  F kf[NK], vf[NK];
  {
    const T* kp = static_cast<const T*>(a.k) + int64_t(kr) * kst + int64_t(kvh) * D;
    const T* vp = static_cast<const T*>(a.v) + int64_t(kr) * kst + int64_t(kvh) * D;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      kf[kk] = O::load(kp + 16 * kk + 8 * h2);
      vf[kk] = O::load(vp + 16 * kk + 8 * h2);
    }
  }
  f32x16 dk[ND], dv[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) dk[i] = dv[i] = zero16();

  const uint32_t brow = TD::b_row8_32(lane), bcol = TD::b_col44_32(lane);
  const int nt = (hi - c0 + BR - 1) / BR, steps = nt * GP;
  auto fetch = [&](int t) {
    const int head = h0 + t / nt, i0 = c0 + (t % nt) * BR;
    T* qb = buf + (t % W::NS) * 2 * BR * D;
    copy_rows<T, BR, D, 4>(qb, static_cast<const T*>(a.q) + int64_t(head) * D, qst, i0, hi, wave, lane);
    copy_rows<T, BR, D, 4>(qb + BR * D, static_cast<const T*>(a.d_o) + int64_t(head) * D, qst, i0, hi, wave, lane);
    // lse by the first wavefront, D by the second; the others repeat them into unused places, so that
    // every wavefront has the same number of copies to count
    const int r = i0 + lane < hi ? i0 + lane : hi - 1;
    lds_copy4((wave & 1 ? a.D : a.lse) + int64_t(r) * a.Hq + head, lds_offset(stat + (t % W::NS) * 4 * BR + wave * BR));
  };
#pragma unroll
  for (int i = 0; i < W::NS - 1; ++i)
    if (i < steps) fetch(i);
  int bad_lo = steps, bad_hi = -1;  // steps whose masked rows hold non-finite values
  for (int t = 0; t < steps; ++t) {
    if (t + W::NS - 2 < steps) copies_landed<(W::NS - 2) * W::kCopies>();  // tile t is there
    else copies_landed();
    lds_barrier();
    if (t + W::NS - 1 < steps) fetch(t + W::NS - 1);
    const T* Qs = buf + (t % W::NS) * 2 * BR * D;
    const T* Os = Qs + BR * D;
    const float* ls = stat + (t % W::NS) * 4 * BR;
    const float* Ds = ls + BR;
    const uint32_t qrow = TD::at(Qs) + brow, orow = TD::at(Os) + brow, qcol = TD::at(Qs) + bcol, ocol = TD::at(Os) + bcol;
    const int i0 = c0 + (t % nt) * BR;
    f32x16 s[2], dp[2];
    auto scores = [&](int sub) {
      s[sub] = dp[sub] = zero16();
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        s[sub] = O::mma32(TD::row8_32(qrow, sub, kk), kf[kk], s[sub]);
        dp[sub] = O::mma32(TD::row8_32(orow, sub, kk), vf[kk], dp[sub]);
      }
    };
    auto probabilities = [&](int sub, auto whole) {
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int rr = 32 * sub + 8 * r4 + 4 * h2;
        const f32x4 l4 = *reinterpret_cast<const f32x4*>(ls + rr), D4 = *reinterpret_cast<const f32x4*>(Ds + rr);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * r4 + j;
          float p = fast_exp2(s[sub][e] * c - l4[j] * kLog2e), d = p * (dp[sub][e] - D4[j]);
          if constexpr (!decltype(whole)::value) {  // rows kj .. lim - 1 see the key
            const bool in = unsigned(i0 + rr + j - kj) < unsigned(lim - kj);
            p = in ? p : 0.f;
            d = in ? d : 0.f;
          }
          s[sub][e] = p;
          dp[sub][e] = d;
        }
      }
    };
    auto products = [&](int sub, bool finite) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const F pf = frag_of<T>(s[sub], ks), df = frag_of<T>(dp[sub], ks);
        const int rr = 32 * sub + 16 * ks;
#pragma unroll
        for (int i = 0; i < ND; ++i) {
          F x = TD::col44_32(ocol, rr, i), y = TD::col44_32(qcol, rr, i);
          if (!finite) {
            x = Finite<T>::only(x);
            y = Finite<T>::only(y);
          }
          dv[i] = O::mma32(x, pf, dv[i]);
          dk[i] = O::mma32(y, df, dk[i]);
        }
      }
    };
    if (i0 >= w0 + 31 && i0 + BR <= emin && i0 + BR <= hi) {
      // Every row sees every key.  One wavefront per SIMD fits, so its own products have to run beside
      // its own exponentials: those of one half of the rows beside the other half's.
      scores(0);
      __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x8, 4, 0);
      __builtin_amdgcn_sched_barrier(0);
      scores(1);
      probabilities(0, std::true_type{});
      if constexpr (sizeof(T) == 2) interleave<2 * NK, 9>();
      __builtin_amdgcn_sched_barrier(0);
      products(0, true);
      probabilities(1, std::true_type{});
      if constexpr (sizeof(T) == 2) interleave<4 * ND, 9>();
      __builtin_amdgcn_sched_barrier(0);
      products(1, true);
    } else {
#pragma unroll
      for (int sub = 0; sub < BR / 32; ++sub) {
        const int s0 = i0 + 32 * sub;
        // some row at or past the wavefront's first key, before its last key's end
        if (w0 >= used || s0 + 31 < w0 || s0 >= emax || s0 >= hi) continue;
        scores(sub);
        if (s0 >= w0 + 31 && s0 + 32 <= emin && s0 + 32 <= hi) {
          probabilities(sub, std::true_type{});
          products(sub, true);
          continue;
        }
        // Zero times a NaN or infinity is not zero: where a masked row may hold one (its products with the
        // keys show it), such elements leave the products, and reach the keys that see them after the loop.
        float probe = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) probe += s[sub][e] * 0.f + dp[sub][e] * 0.f;
        const bool finite = !__any(probe != 0.f);
        probabilities(sub, std::false_type{});
        products(sub, finite);
        if (!finite) {
          bad_lo = t < bad_lo ? t : bad_lo;
          bad_hi = t;
        }
      }
    }
  }
  for (int t = bad_lo; t <= bad_hi; ++t)
    for (int r = 0; r < BR; ++r) {
      const int row = c0 + (t % nt) * BR + r;
      if (row >= hi) break;
      const bool in = unsigned(row - kj) < unsigned(lim - kj);
      const int64_t at = row * qst + int64_t(h0 + t / nt) * D + 4 * h2;
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = io<T>::load(static_cast<const T*>(a.d_o) + at, 32 * i + 8 * r4 + j),
                        y = io<T>::load(static_cast<const T*>(a.q) + at, 32 * i + 8 * r4 + j);
            dv[i][4 * r4 + j] += in && !(fabsf(x) < INFINITY) ? x : 0.f;
            dk[i][4 * r4 + j] += in && !(fabsf(y) < INFINITY) ? NAN : 0.f;  // the row's scores, and P, are NaN
          }
    }
  if (kj < used) {
    const int64_t at = int64_t(kj) * kst + int64_t(kvh) * D;
    TG* kp = (a.parts == 1 ? static_cast<TG*>(a.dk) : reinterpret_cast<TG*>(a.part + (2 * part) * a.n * kst)) + at;
    TG* vp = (a.parts == 1 ? static_cast<TG*>(a.dv) : reinterpret_cast<TG*>(a.part + (2 * part + 1) * a.n * kst)) + at;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 x, y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = dk[i][4 * r4 + j] * a.scale;
          y[j] = dv[i][4 * r4 + j];
        }
        store4(kp + 32 * i + 8 * r4 + 4 * h2, x);
        store4(vp + 32 * i + 8 * r4 + 4 * h2, y);
      }
  }
}

template <typename T, int D>
constexpr size_t q_lds() { return size_t(sizeof(T) == 2 ? 2 : 1) * 2 * BN * D * sizeof(T); }

template <typename T, typename TG, int D>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void prompt_dq_kernel(const PromptBwdArgs a, int ntile) {
  using O = Op<T>;
  using F = typename O::frag;
  using TD = Tile<T, D>;
  constexpr int NK = D / 16, ND = D / 32;
  constexpr bool DB = sizeof(T) == 2;  // two buffers
  extern __shared__ __align__(16) unsigned char smem[];
  T* const buf = reinterpret_cast<T*>(smem);  // [1 or 2][K tile, V tile]

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h2 = lane >> 5, l32 = lane & 31;
  const HeadTile ht = head_tile(blockIdx.x, a.Hq);
  const int head = ht.head, tile = ntile - 1 - ht.tile;
  const int r0 = tile * BM;
  const int used = rows_used(a.cu, a.nseq, a.n);
  if (a.zero_tail && r0 + BM > used)
    zero_rows<TG, D>(static_cast<TG*>(a.dq) + int64_t(head) * D, int64_t(a.Hq) * D, r0 > used ? r0 : used,
                     r0 + BM < a.n ? r0 + BM : a.n, tid);
  if (r0 >= used) return;
  const int kvh = head / (a.Hq / a.Hkv);
  const int64_t qst = int64_t(a.Hq) * D, kst = int64_t(a.Hkv) * D;
  const T* kp = static_cast<const T*>(a.k) + int64_t(kvh) * D;
  const T* vp = static_cast<const T*>(a.v) + int64_t(kvh) * D;

  int lo = span_of(a.cu, a.nseq, a.n, r0).start;
  const int hi = r0 + BM < used ? r0 + BM : used;
  const int w0 = r0 + 32 * wave, qi = w0 + l32;
  const int wlast = w0 + 31 < used ? w0 + 31 : used - 1;
  const int qr = qi < used ? qi : used - 1;
  const int start = span_of(a.cu, a.nseq, a.n, qr).start;
  int smin = __shfl(start, 0);
  const int smax = __shfl(start, 31);
  const float c = a.scale * kLog2e;
  float ls = a.lse[int64_t(qr) * a.Hq + head] * kLog2e;
  float Di = a.D[int64_t(qr) * a.Hq + head];

  F qf[NK], of[NK];
  {
    const T* qp = static_cast<const T*>(a.q) + int64_t(qr) * qst + int64_t(head) * D;
    const T* op = static_cast<const T*>(a.d_o) + int64_t(qr) * qst + int64_t(head) * D;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      qf[kk] = O::load(qp + 16 * kk + 8 * h2);
      of[kk] = O::load(op + 16 * kk + 8 * h2);
    }
  }
  f32x16 dq[ND];
  const uint32_t brow = TD::b_row8_32(lane), bcol = TD::b_col44_32(lane);
#pragma unroll
  for (int i = 0; i < ND; ++i) dq[i] = zero16();
  int bad_lo = hi, bad_hi = 0;  // keys of masked tiles with non-finite values
  const bool correct = sizeof(T) == 2 || a.o_bf16;  // D is not exact to fp32
  auto fetch = [&](int t) {
    T* kb = buf + (DB ? (t & 1) * 2 * BN * D : 0);
    copy_rows<T, BN, D, 4>(kb, kp, kst, lo + t * BN, hi, wave, lane);
    copy_rows<T, BN, D, 4>(kb + BN * D, vp, kst, lo + t * BN, hi, wave, lane);
  };
  for (bool again = false;; again = true) {
    const int nt = (hi - lo + BN - 1) / BN;
    float sum = 0.f, size = 0.f;  // of dS, and of |dS|
    fetch(0);
    for (int t = 0; t < nt; ++t) {
      copies_done();
      if (DB && t + 1 < nt) fetch(t + 1);
      const T* Ks = buf + (DB ? (t & 1) * 2 * BN * D : 0);
      const T* Vs = Ks + BN * D;
      const uint32_t krow = TD::at(Ks) + brow, vrow = TD::at(Vs) + brow, kcol = TD::at(Ks) + bcol;
      const int k0 = lo + t * BN;
#pragma unroll
      for (int j = 0; j < BN / 32; ++j) {
        const int s0 = k0 + 32 * j;
        if (wlast < w0 || s0 > wlast || s0 + 32 <= smin) continue;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          s = O::mma32(TD::row8_32(krow, j, kk), qf[kk], s);
          dp = O::mma32(TD::row8_32(vrow, j, kk), of[kk], dp);
        }
        auto gradients = [&](auto whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            dp[i] = fast_exp2(s[i] * c - ls) * (dp[i] - Di);
            if constexpr (!decltype(whole)::value)  // the row sees keys start .. qi
              dp[i] = unsigned(s0 + crow(i, h2) - start) <= unsigned(qi - start) ? dp[i] : 0.f;
            sum += dp[i];
            size += fabsf(dp[i]);
          }
        };
        auto products = [&](bool finite) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const F df = frag_of<T>(dp, ks);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
              F x = TD::col44_32(kcol, 32 * j + 16 * ks, i);
              if (!finite) x = Finite<T>::only(x);
              dq[i] = O::mma32(x, df, dq[i]);
            }
          }
        };
        if (s0 + 31 <= w0 && s0 >= smax) {
          gradients(std::true_type{});
          products(true);
        } else {
          float probe = 0.f;  // a non-finite key shows in its scores, as for dk and dv
#pragma unroll
          for (int i = 0; i < 16; ++i) probe += s[i] * 0.f;
          const bool finite = !__any(probe != 0.f);
          gradients(std::false_type{});
          products(finite);
          if (!finite) {
            bad_lo = s0 < bad_lo ? s0 : bad_lo;
            bad_hi = s0 + 32 > bad_hi ? s0 + 32 : bad_hi;
          }
        }
      }
      if (!DB) {
        __syncthreads();
        if (t + 1 < nt) fetch(t + 1);
      }
    }
    if (again || !correct) break;
    sum = sum_halves(sum);
    size = sum_halves(size);
    Di += sum;
    if (qi < used && h2 == 0) a.D[int64_t(qi) * a.Hq + head] = Di;
    // The rows to form again (both halves of the wavefront know): the first one's sequence is where the
    // keys begin, a row that is done takes probabilities of zero.
    const bool mine = qi < used && fabsf(sum) > kLeft<T> * size;
    const uint64_t rows = __ballot(mine);
    smin = rows ? __shfl(start, __builtin_ctzll(rows)) : hi;
    lds_barrier();
    int* const first = reinterpret_cast<int*>(smem);
    if (lane == 0) first[wave] = smin;
    lds_barrier();
    const int f0 = first[0] < first[1] ? first[0] : first[1], f1 = first[2] < first[3] ? first[2] : first[3];
    lo = f0 < f1 ? f0 : f1;
    if (lo >= hi) break;
    if (!mine) ls = INFINITY;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) dq[i][r] = mine ? 0.f : dq[i][r];
    lds_barrier();
  }
  for (int key = bad_lo; key < bad_hi && key < hi; ++key) {
    const bool seen = key <= qi && key >= start;
    const T* row = kp + int64_t(key) * kst + 4 * h2;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = io<T>::load(row, 32 * i + 8 * r4 + e);
          dq[i][4 * r4 + e] += seen && !(fabsf(x) < INFINITY) ? NAN : 0.f;
        }
  }
  if (qi < used) {
    TG* p = static_cast<TG*>(a.dq) + int64_t(qi) * qst + int64_t(head) * D;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = dq[i][4 * r4 + j] * a.scale;
        store4(p + 32 * i + 8 * r4 + 4 * h2, x);
      }
  }
}

// dk and dv from the parts of their groups' heads, in order.
template <typename TG>
__global__ __launch_bounds__(256) void prompt_join_kernel(const PromptBwdArgs a, int64_t count) {
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  const bool tail = i >= rows_used(a.cu, a.nseq, a.n) * int64_t(a.Hkv) * a.d;
  if (i >= count || (tail && !a.zero_tail)) return;
  f32x4 x = {0, 0, 0, 0}, y = x;
  for (int p = 0; p < (tail ? 0 : a.parts); ++p) {
    x += *reinterpret_cast<const f32x4*>(a.part + 2 * p * count + i);
    y += *reinterpret_cast<const f32x4*>(a.part + (2 * p + 1) * count + i);
  }
  store4(static_cast<TG*>(a.dk) + i, x);
  store4(static_cast<TG*>(a.dv) + i, y);
}

template <typename TO>
hipError_t launch_dot_o(const PromptBwdArgs& a, hipStream_t st) {
  const int64_t rows = int64_t(a.n) * a.Hq;
  const dim3 grid(uint32_t((rows + 31) / 32));
  if (a.in_bf16) prompt_dot_kernel<TO, bf16_t><<<grid, 256, 0, st>>>(a);
  else prompt_dot_kernel<TO, float><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, typename TG, int D>
hipError_t launch_dkv(const PromptBwdArgs& a, int ntile, hipStream_t st) {
  auto kern = prompt_dkv_kernel<T, TG, D>;
  constexpr size_t lds = KvShape<T, D>::lds;
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  static std::atomic<uint64_t> done{0};
  const hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kern), int(lds), done);
  if (e != hipSuccess) return e;
  kern<<<dim3(uint32_t(int64_t(ntile) * a.Hkv * a.parts)), 256, lds, st>>>(a);
  return hipGetLastError();
}

template <typename T, typename TG, int D>
hipError_t launch(const PromptBwdArgs& a, hipStream_t st) {
  auto kq = prompt_dq_kernel<T, TG, D>;
  constexpr size_t lds = q_lds<T, D>();
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  static std::atomic<uint64_t> done{0};
  hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kq), int(lds), done);
  if (e == hipSuccess) e = a.o_bf16 ? launch_dot_o<bf16_t>(a, st) : launch_dot_o<float>(a, st);
  if (e != hipSuccess) return e;
  const int ntile = (a.n + BM - 1) / BM;
  kq<<<dim3(uint32_t(int64_t(ntile) * a.Hq)), 256, lds, st>>>(a, ntile);  // corrects D, before dk and dv read it
  e = hipGetLastError();
  if (e == hipSuccess) e = a.parts == 1 ? launch_dkv<T, TG, D>(a, ntile, st) : launch_dkv<T, float, D>(a, ntile, st);
  if (e == hipSuccess && a.parts > 1) {
    const int64_t count = int64_t(a.n) * a.Hkv * a.d;
    prompt_join_kernel<TG><<<dim3(uint32_t((count / 4 + 255) / 256)), 256, 0, st>>>(a, count);
    e = hipGetLastError();
  }
  return e;
}

template <typename T, int D>
hipError_t launch_g(const PromptBwdArgs& a, hipStream_t st) {
  return a.grad_bf16 ? launch<T, bf16_t, D>(a, st) : launch<T, float, D>(a, st);
}

}  // namespace

// Parts that the query heads of a group are cut into for dk and dv.  The key tiles of a long
// sequence differ in length by as much as its length, so the GPU wants several times as many
// workgroups as compute units; each part beyond the first writes and rereads fp32 sums.  Measured,
// whole gradient and forward, parts while there are fewer than 1 (no parts) : 512 : 1024 : 2048
// workgroups, us: the rows above 959 : 701 : 682 : 681; one sequence of 8192 1990 : 1462 : 1456 :
// 1459; 1500 and 300 rows, 8 heads on 1, 571 : 182 : 180 : 181; 512 rows, 16 on 8, d = 64, 62 : 51 :
// 52 : 52.
int prompt_bwd_parts(int n, int Hq, int Hkv) {
  const int64_t units = (int64_t(n) + BM - 1) / BM * Hkv;
  const int G = Hq / Hkv;
  int parts = 1;
  for (int p = 2; p <= G; ++p)
    if (G % p == 0 && units * parts < 1024) parts = p;
  return parts;
}

hipError_t launch_prompt_bwd(const PromptBwdArgs& a, hipStream_t st) {
  if (a.in_bf16) return a.d == 64 ? launch_g<bf16_t, 64>(a, st) : launch_g<bf16_t, 128>(a, st);
  return a.d == 64 ? launch_g<float, 64>(a, st) : launch_g<float, 128>(a, st);
}

}  // namespace kda
