// kda_prompt_fwd.hip -- causal softmax attention over packed prompts, grouped heads.
//
//   o_i = sum_j P_ij v_j,  P_ij = exp(scale q_i . k_j - lse_i),  j in i's sequence, j <= i
//   lse_i = log sum_j exp(scale q_i . k_j)
//
// Rows of all sequences lie behind one another; a workgroup takes 128 consecutive rows of one
// query head, whichever sequences they belong to, and walks the keys from the start of its first
// row's sequence to its last row in tiles of 64: short sequences share a tile instead of filling
// one each, and the launch needs no list of lengths on the host.  Only tiles that a row's own
// start or end cuts are masked.  Where that gives too few workgroups, a workgroup takes 32 rows
// and its wavefronts share the keys (SPLIT).
//
// Four wavefronts of 32 rows.  Scores are formed transposed, S^T = K Q^T (keys x rows), so that
// a lane holds 32 keys of one row: the softmax needs one exchange between the half-wavefronts,
// and the probabilities are in place as the operand of O^T = V^T P^T (k steps over the keys in the
// order the registers have, which the transposing reads of V follow).  The running maximum is
// raised only when a tile exceeds it by 2^8 (any reference serves while nothing overflows), so
// most tiles do not touch the accumulators.  Maximum, sum and accumulators are fp32; with bf16
// elements P is rounded to bf16 for the second product, 2^-8 relative each, as bf16 outputs are (and fp32
// outputs of bf16 elements then carry).
//
// Measured (bf16, 16270 rows in sequences of 8192, 5000, 1, 2300 and 777, 32 heads on 8, d = 128):
// 919 us, 875 TFLOP/s of the masked half, where a large matrix product reaches 1230.  What bounds
// it is the issue of the matrix instructions (38 % of the cycles) and of the vector instructions between
// them (50 %, not counting that an exponential holds its unit four times as long); the LDS is read
// without conflicts (they were 34 % of its cycles before the rows were permuted, and the time did
// not change).  The order of the tiles, longest rows first, lets the short ones fill the end.
#include "kda_prompt.hpp"

namespace kda {

namespace {

// Rows of a workgroup and keys of a step: four wavefronts of 32 rows that share 64 keys, or (SPLIT)
// four that share 32 rows and take 32 of 128 keys each.
template <bool SPLIT> constexpr int kRows = SPLIT ? 32 : 128;
template <bool SPLIT> constexpr int kKeys = SPLIT ? 128 : 64;

template <typename T, int D, bool SPLIT>
struct FwdShape {
  static constexpr int kStep = 2 * kKeys<SPLIT> * D * int(sizeof(T));
  static constexpr int NB = 2 * kStep <= 128 * 1024 ? 2 : 1;  // steps in the LDS (fp32 shared keys at d = 128: one)
  static constexpr int kJoin = SPLIT ? 4 * 32 * (D + 4) * 4 + 2 * 4 * 32 * 4 : 0;
  static constexpr size_t lds = NB * kStep > kJoin ? NB * kStep : kJoin;
};

template <typename T, typename TO, int D, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(T) == 2 && !SPLIT ? 2 : 1) void prompt_fwd_kernel(const PromptArgs a, int ntile) {
  using O = Op<T>;
  using F = typename O::frag;
  using TD = Tile<T, D>;
  using W = FwdShape<T, D, SPLIT>;
  constexpr int NK = D / 16, ND = D / 32, BM = kRows<SPLIT>, BN = kKeys<SPLIT>, NJ = SPLIT ? 1 : 2;
  extern __shared__ __align__(16) unsigned char smem[];
  T* const buf = reinterpret_cast<T*>(smem);  // [NB][K tile, V tile]

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h2 = lane >> 5, l32 = lane & 31;
  const HeadTile ht = head_tile(blockIdx.x, a.Hq);
  const int head = ht.head, tile = ntile - 1 - ht.tile;  // long rows first
  const int r0 = tile * BM;
  const int used = rows_used(a.cu, a.nseq, a.n);
  if (a.zero_tail && r0 + BM > used) {
    const int first = r0 > used ? r0 : used, last = r0 + BM < a.n ? r0 + BM : a.n;
    zero_rows<TO, D>(static_cast<TO*>(a.o) + int64_t(head) * D, int64_t(a.Hq) * D, first, last, tid);
    if (a.lse && first + tid < last) a.lse[int64_t(first + tid) * a.Hq + head] = 0.f;
  }
  if (r0 >= used) return;
  const int kvh = head / (a.Hq / a.Hkv);
  const int64_t kst = int64_t(a.Hkv) * D;
  const T* kp = static_cast<const T*>(a.k) + int64_t(kvh) * D;
  const T* vp = static_cast<const T*>(a.v) + int64_t(kvh) * D;

  const int lo = span_of(a.cu, a.nseq, a.n, r0).start;
  const int hi = r0 + BM < used ? r0 + BM : used;
  const int w0 = SPLIT ? r0 : r0 + 32 * wave, qi = w0 + l32;
  const int wlast = w0 + 31 < used ? w0 + 31 : used - 1;  // the wavefront's last row (below w0: none)
  const int qr = qi < used ? qi : used - 1;
  const int start = span_of(a.cu, a.nseq, a.n, qr).start;
  // starts rise with the rows: the wavefront's first and last
  const int smin = __shfl(start, 0), smax = __shfl(start, 31);

  // a negative scale is the positive one with the queries' signs turned; a scale of zero is the
  // least normal number (a masked score, -inf, times zero would be NaN)
  const float c = fmaxf(fabsf(a.scale) * kLog2e, 1.1754944e-38f);
  F qf[NK];
  {
    const T* qp = static_cast<const T*>(a.q) + (int64_t(qr) * a.Hq + head) * D;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      qf[kk] = O::load(qp + 16 * kk + 8 * h2);
      if (a.scale < 0.f) qf[kk] = O::neg(qf[kk]);
    }
  }
  f32x16 acc[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) acc[i] = zero16();
  float m = -INFINITY, l = 0.f;
  int bad_lo = hi, bad_hi = 0;  // keys of masked tiles with non-finite values
  const uint32_t krow = TD::b_row8_32(lane), vcol = TD::b_col44_32(lane);

  const int nt = (hi - lo + BN - 1) / BN;
  auto fetch = [&](int t) {
    T* kb = buf + (W::NB == 2 ? t & 1 : 0) * 2 * BN * D;
    copy_rows<T, BN, D, 4>(kb, kp, kst, lo + t * BN, hi, wave, lane);
    copy_rows<T, BN, D, 4>(kb + BN * D, vp, kst, lo + t * BN, hi, wave, lane);
  };
  fetch(0);
  for (int t = 0; t < nt; ++t) {
    if (W::NB == 1 && t > 0) {
      lds_barrier();
      fetch(t);
    }
    copies_done();
    if (W::NB == 2 && t + 1 < nt) fetch(t + 1);
    const T* Ks = buf + (W::NB == 2 ? t & 1 : 0) * 2 * BN * D + (SPLIT ? 32 * wave * D : 0);
    const T* Vs = Ks + BN * D;
    const uint32_t kb = TD::at(Ks) + krow, vb = TD::at(Vs) + vcol;
    const int k0 = lo + t * BN + (SPLIT ? 32 * wave : 0);  // this wavefront's keys: 32 NJ of them
    if (wlast >= w0 && k0 <= wlast && k0 + 32 * NJ > smin) {
      f32x16 s[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        s[j] = zero16();
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) s[j] = O::mma32(TD::row8_32(kb, j, kk), qf[kk], s[j]);
      }
      const bool masked = !(k0 + 32 * NJ - 1 <= w0 && k0 >= smax);
      if (masked) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = k0 + 32 * j + crow(i, h2);
            s[j][i] = unsigned(key - start) <= unsigned(qi - start) ? s[j][i] : -INFINITY;
          }
      }
      float mt = s[0][0];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) mt = fmaxf(mt, s[j][i]);
      mt = c * max_halves(mt);
      if (__any(mt > m + 8.f)) {
        const float mn = fmaxf(m, mt);
        const float ref = mn == -INFINITY ? 0.f : mn;  // a row that has met no key yet
        const float al = fast_exp2(m - ref);
        l *= al;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][r] *= al;
        m = mn;
      }
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[j][i] = fast_exp2(s[j][i] * c - ref);
          l += s[j][i];
        }
      }
      // A masked probability is zero, but zero times a NaN or infinity is not: where a tile is
      // masked and holds such values, they leave the product, and after the loop reach the rows that
      // see them.
      if (masked) {
        Finite<T> fin;
#pragma unroll
        for (int e = 0; e < 2 * NJ * ND; ++e) fin.see(TD::col44_32(vb, 16 * (e % (2 * NJ)), e / (2 * NJ)));
        if (__any(!fin.all())) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const F pf = frag_of<T>(s[j], ks);
#pragma unroll
              for (int i = 0; i < ND; ++i)
                acc[i] = O::mma32(Finite<T>::only(TD::col44_32(vb, 32 * j + 16 * ks, i)), pf, acc[i]);
            }
          bad_lo = k0 < bad_lo ? k0 : bad_lo;
          bad_hi = k0 + 32 * NJ;
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const F pf = frag_of<T>(s[j], ks);
#pragma unroll
          for (int i = 0; i < ND; ++i) acc[i] = O::mma32(TD::col44_32(vb, 32 * j + 16 * ks, i), pf, acc[i]);
        }
    }
  }
  for (int key = bad_lo; key < bad_hi && key < hi; ++key) {
    if (SPLIT && ((key - lo) >> 5 & 3) != wave) continue;  // another wavefront's
    const bool seen = key <= qi && key >= start;
    const T* row = vp + int64_t(key) * kst + 4 * h2;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = io<T>::load(row, 32 * i + 8 * r4 + e);
          acc[i][4 * r4 + e] += seen && !(fabsf(x) < INFINITY) ? x : 0.f;
        }
  }
  l = sum_halves(l);
  if constexpr (SPLIT) {
    // the four wavefronts' sums of the same rows, to one reference
    float* const jo = reinterpret_cast<float*>(smem);  // [4][32][D + 4]
    float* const jm = jo + 4 * 32 * (D + 4);           // [4][32] maxima, then sums
    lds_barrier();
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4)
        *reinterpret_cast<f32x4*>(jo + (wave * 32 + l32) * (D + 4) + 32 * i + 8 * r4 + 4 * h2) =
            f32x4{acc[i][4 * r4], acc[i][4 * r4 + 1], acc[i][4 * r4 + 2], acc[i][4 * r4 + 3]};
    if (h2 == 0) {
      jm[wave * 32 + l32] = m;
      jm[128 + wave * 32 + l32] = l;
    }
    lds_barrier();
    for (int e = tid; e < 32 * (D / 4); e += 256) {
      const int r = e / (D / 4), c0 = 4 * (e % (D / 4));
      if (r0 + r >= used) continue;
      const float mm = fmaxf(fmaxf(jm[r], jm[32 + r]), fmaxf(jm[64 + r], jm[96 + r]));
      const float ref = mm == -INFINITY ? 0.f : mm;
      f32x4 x = {0, 0, 0, 0};
      float ls = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = fast_exp2(jm[32 * w + r] - ref);
        ls += f * jm[128 + 32 * w + r];
        x += *reinterpret_cast<const f32x4*>(jo + (32 * w + r) * (D + 4) + c0) * f;
      }
      store4(static_cast<TO*>(a.o) + (int64_t(r0 + r) * a.Hq + head) * D + c0, x * (1.0f / ls));
      if (a.lse && c0 == 0) a.lse[int64_t(r0 + r) * a.Hq + head] = (mm + log2f(ls)) * 0.6931471805599453f;
    }
    return;
  }
  if (qi < used) {
    const float inv = 1.0f / l;
    TO* op = static_cast<TO*>(a.o) + (int64_t(qi) * a.Hq + head) * D;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = acc[i][4 * r4 + j] * inv;
        store4(op + 32 * i + 8 * r4 + 4 * h2, x);
      }
    if (a.lse && h2 == 0) a.lse[int64_t(qi) * a.Hq + head] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <typename T, typename TO, int D, bool SPLIT>
hipError_t launch(const PromptArgs& a, hipStream_t st) {
  auto kern = prompt_fwd_kernel<T, TO, D, SPLIT>;
  constexpr size_t lds = FwdShape<T, D, SPLIT>::lds;
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  static std::atomic<uint64_t> done{0};
  if constexpr (lds > 65536) {
    const hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kern), int(lds), done);
    if (e != hipSuccess) return e;
  }
  const int ntile = (a.n + kRows<SPLIT> - 1) / kRows<SPLIT>;
  kern<<<dim3(uint32_t(int64_t(ntile) * a.Hq)), 256, lds, st>>>(a, ntile);
  return hipGetLastError();
}

// Fewer tiles of 128 rows than this are divided into tiles of 32 rows whose keys the wavefronts
// share: up to four times the workgroups for a quarter of the reuse of K and V, paid with one join.
// Measured, whole : shared, us, one sequence of d = 128: bf16 60 tiles 57 : 30, 192 84 : 79, 256
// 115 : 123, 376 168 : 246; fp32 60 tiles 269 : 91, 192 416 : 244, 256 572 : 385, 320 700 : 603,
// 376 839 : 809.  (With d = 64 the two meet at 376 tiles in both types.)
template <typename T> constexpr int64_t kSplitBelow = sizeof(T) == 2 ? 224 : 352;

template <typename T, int D>
hipError_t launch_o(const PromptArgs& a, hipStream_t st) {
  if (int64_t((a.n + 127) / 128) * a.Hq < kSplitBelow<T>)
    return a.out_bf16 ? launch<T, bf16_t, D, true>(a, st) : launch<T, float, D, true>(a, st);
  return a.out_bf16 ? launch<T, bf16_t, D, false>(a, st) : launch<T, float, D, false>(a, st);
}

}  // namespace

hipError_t launch_prompt_fwd(const PromptArgs& a, hipStream_t st) {
  if (a.in_bf16) return a.d == 64 ? launch_o<bf16_t, 64>(a, st) : launch_o<bf16_t, 128>(a, st);
  return a.d == 64 ? launch_o<float, 64>(a, st) : launch_o<float, 128>(a, st);
}

}  // namespace kda
