// kda_cache_rope.hip -- appending to the paged 8-bit cache with the rotary positions applied to the keys
// on the way, and to the same tokens' queries.
//
// Workgroups of two kinds in one launch: some for the (touched page, key head) pairs, as in plain appending
// (kda_cache.hip), and behind them some for the rows of queries.  Keys are turned in 64 bits and
// rounded once: the codes are those of the exactly turned keys, whatever the inputs' type.
// (From turned keys rounded to bf16 one code in eight would differ, from fp32 ones one in some millions.)
//
// The queries are bound by their bytes; the pages by a chain of latencies (search, table, keys, scale) and by issue: a
// sine and cosine in 64 bits take some 60 instructions, a pair turned by them some 20.  Measured: 14349 tokens of 8 key and
// 32 query heads of 128, bf16 (323 MB) 78 us, of which the keys and values alone 40, the sines 4, the turns 7, V's way
// through the LDS 1; 256 single tokens 13.8, bound by the chain and by one byte to each of 262144 rows of V's pages; 2963 fp32
// tokens of 4 heads of 64 9.4.
#include "kda_cache.hpp"
#include "kda_rotary.hpp"

namespace kda {

namespace {

// What one (page, key head) is to do.
struct PageWork {
  int64_t row0, p0;  // first row of k and v, its place in the sequence
  int off, cnt;      // of the page's tokens
};

// The finite values' largest magnitude.
__device__ __forceinline__ void see(float& most, const f32x8& x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = fabsf(x[j]);
    if (m < INFINITY && m > most) most = m;
  }
}

__device__ __forceinline__ u32x2v encode8(const f32x8& x, float inv) {
  u32x2v w;
  w[0] = encode4(to_range(x[0], inv), to_range(x[1], inv), to_range(x[2], inv), to_range(x[3], inv));
  w[1] = encode4(to_range(x[4], inv), to_range(x[5], inv), to_range(x[6], inv), to_range(x[7], inv));
  return w;
}

// A unit of k turned in 64 bits, its 16 channels in `own`, a column of the thread's own in LDS (for append_few).
constexpr int kColumns = 256;
__device__ __forceinline__ void turn_unit(const Rotation& t, int64_t row, int64_t place, int u, float* own, float& most) {
#pragma unroll 2
  for (int e = 0; e < 8; ++e) {
    double s, c;
    sine_cosine(angle_of(t, row, place, pair_of(u, e, t.half, t.interleaved)), s, c);
    float* const x = own + (t.interleaved ? 2 * e : e) * kColumns;
    float* const y = x + (t.interleaved ? 1 : 8) * kColumns;
    const double p = *x, q = *y;
    const float f = to_fp32(mul_add(p, c, -q * s)), g = to_fp32(mul_add(q, c, p * s));
    *x = f;
    *y = g;
    const float af = fabsf(f), ag = fabsf(g);
    most = af < INFINITY && af > most ? af : most;
    most = ag < INFINITY && ag > most ? ag : most;
  }
}
__device__ __forceinline__ void to_column(float* own, const f32x8& x0, const f32x8& x1) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    own[j * kColumns] = x0[j];
    own[(8 + j) * kColumns] = x1[j];
  }
}
__device__ __forceinline__ f32x8 from_column(const float* own) {
  f32x8 x;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = own[j * kColumns];
  return x;
}

// Slot `slot`'s work, false if there is none: sequence i's pages sit at slots cu[i] / P + 2 i onwards, which leaves
// each at least as many as it touches.  256 sequences at one look, with their lengths: what follows needs no other.
__device__ __forceinline__ bool page_work(const CacheAppendArgs& a, int slot, int lane, int& page, PageWork& x) {
  const int P = a.page, ps = page_shift(P);
  int lo = 0, up = a.N;
  while (up - lo > 256) {
    const int step = (up - lo + 63) / 64;
    const int64_t mid = lo + int64_t(step) * (lane + 1);
    lo += step * __popcll(__ballot(mid < up && (a.cu[mid] >> ps) + 2 * mid <= slot));
    up = lo + step < up ? lo + step : up;
  }
  int c[4], n[4], held4[4], count = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = lo + 64 * j + lane, at = i < up ? i : lo;
    c[j] = a.cu[at];
    n[j] = a.cu[at + 1];
    held4[j] = a.ctx[at];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t i = int64_t(lo) + 64 * j + lane;
    count += __popcll(__ballot(i < up && (i == lo || (c[j] >> ps) + 2 * i <= slot)));
  }
  const int at = count - 1, from = at & 63;  // (starts rise with the sequences: those before the slot come first)
  int first = 0, last = 0, ctx = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (at >> 6 == j) {
      first = __builtin_amdgcn_readlane(c[j], from);
      last = __builtin_amdgcn_readlane(n[j], from);
      ctx = __builtin_amdgcn_readlane(held4[j], from);
    }
  lo += at;
  const int64_t base = (first >> ps) + 2 * int64_t(lo);
  first = first < 0 ? 0 : first;
  last = last > a.n ? a.n : last;
  if (first >= last || slot < base) return false;
  const int64_t held = ctx < 0 ? 0 : ctx;
  const int64_t pi = (held >> ps) + (slot - base);
  x.p0 = pi * P > held ? pi * P : held;
  const int64_t end = held + (last - first), p1 = (pi + 1) * P < end ? (pi + 1) * P : end;
  if (x.p0 >= p1 || pi >= a.max_pages) return false;
  page = a.table[int64_t(lo) * a.max_pages + pi];
  x.off = int(x.p0 - pi * P);
  x.cnt = int(p1 - x.p0);
  x.row0 = first + (x.p0 - held);
  return true;
}

// A turned bf16 key stays in bf16, rounded to odd: eight bits so rounded give the same codes (of four, or fewer) as all.
__device__ __forceinline__ uint32_t odd_bf16(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u >> 16) | (u & 0xffffu ? 1u : 0u);
}
// elements 2 w and 2 w + 1 of a fragment, read and written by whole registers
__device__ __forceinline__ f32x2 two(const bf16x8& x, int w) {
  const uint32_t u = __builtin_bit_cast(u32x4, x)[w];
  return f32x2{__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)};
}
__device__ __forceinline__ f32x2 two(const f32x8& x, int w) { return f32x2{x[2 * w], x[2 * w + 1]}; }
__device__ __forceinline__ void put_two(bf16x8& x, int w, float a, float b) {
  u32x4 u = __builtin_bit_cast(u32x4, x);
  u[w] = odd_bf16(a) | odd_bf16(b) << 16;
  x = __builtin_bit_cast(bf16x8, u);
}
__device__ __forceinline__ void put_two(f32x8& x, int w, float a, float b) {
  x[2 * w] = a;
  x[2 * w + 1] = b;
}
// A unit of HB heads' k turned in 64 bits in place: the sines are formed once for all heads.
template <typename T, int HB>
__device__ __forceinline__ void turn_units(const Rotation& t, int64_t row, int64_t place, int u, typename Op<T>::frag (*k)[2], float* most) {
  if (t.interleaved)
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      const auto even = __builtin_shufflevector(k[b][0], k[b][1], 0, 2, 4, 6, 8, 10, 12, 14);
      k[b][1] = __builtin_shufflevector(k[b][0], k[b][1], 1, 3, 5, 7, 9, 11, 13, 15);
      k[b][0] = even;
    }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    double s[2], c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) sine_cosine(angle_of(t, row, place, pair_of(u, 2 * w + e, t.half, t.interleaved)), s[e], c[e]);
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      const f32x2 x = two(k[b][0], w), y = two(k[b][1], w);
      float f[2], g[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const double p = x[e], q = y[e];
        f[e] = to_fp32(mul_add(p, c[e], -q * s[e]));
        g[e] = to_fp32(mul_add(q, c[e], p * s[e]));
        const float af = fabsf(f[e]), ag = fabsf(g[e]);
        most[b] = af < INFINITY && af > most[b] ? af : most[b];
        most[b] = ag < INFINITY && ag > most[b] ? ag : most[b];
      }
      put_two(k[b][0], w, f[0], f[1]);
      put_two(k[b][1], w, g[0], g[1]);
      __builtin_amdgcn_sched_barrier(0);  // the terms of two pairs at a time: all of them would not fit the registers
    }
  }
  if (t.interleaved)
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      const auto low = __builtin_shufflevector(k[b][0], k[b][1], 0, 8, 1, 9, 2, 10, 3, 11);
      k[b][1] = __builtin_shufflevector(k[b][0], k[b][1], 4, 12, 5, 13, 6, 14, 7, 15);
      k[b][0] = low;
    }
}

// One workgroup for a page and HB key heads, a thread for each unit of its rows' keys: all at once in registers.
template <typename T, int D, int HB>
__device__ __forceinline__ void append_page(const CacheRopeArgs& ra, int id, uint8_t* image, float* red) {
  const CacheAppendArgs& a = ra.c;
  const Rotation& t = ra.q.turn;
  constexpr int CPR = D / 8, UPR = D / 16, NT = 64 * UPR;  // chunks of 8 channels, units of two, of a row; threads
  const int tid = threadIdx.x, P = a.page, sets = a.Hkv / HB;
  const int h = id % sets * HB, slot = id / sets;

  int page;
  PageWork w;
  if (!page_work(a, slot, tid & 63, page, w)) return;
  if (page < 0 || page >= a.pages) return;
  const int off = w.off, cnt = w.cnt;
  const int64_t row0 = w.row0, p0 = w.p0, ph = int64_t(page) * a.Hkv + h;
  float old_k[HB], old_v[HB];
#pragma unroll
  for (int b = 0; b < HB; ++b) {
    old_k[b] = a.ks[ph + b];
    old_v[b] = a.vs[ph + b];
  }

  typedef typename Op<T>::frag F;
  F kr[HB][2], vr[HB][2];
  const int row = tid / UPR, u = tid % UPR;
  const Unit un = unit_of(u, t.half);
  const T* src = static_cast<const T*>(a.k) + (row0 + row) * ra.k_stride + h * D;
#pragma unroll
  for (int b = 0; b < HB; ++b) {
    kr[b][0] = kr[b][1] = F{};
    if (row < cnt) {
      kr[b][0] = Op<T>::load(src + b * D + 8 * un.c0);
      kr[b][1] = Op<T>::load(src + b * D + 8 * un.c1);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = tid + NT * i, r = e / CPR, c = e % CPR;
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      vr[b][i] = F{};
      if (r < cnt) vr[b][i] = Op<T>::load(static_cast<const T*>(a.v) + (row0 + r) * ra.v_stride + (h + b) * D + 8 * c);
    }
  }
  float mk[HB] = {}, mv[HB] = {};
  if (row < cnt && un.turns)
    turn_units<T, HB>(t, row0 + row, p0 + row, u, kr, mk);
  else
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      see(mk[b], Op<T>::unpack(kr[b][0]));
      see(mk[b], Op<T>::unpack(kr[b][1]));
    }
#pragma unroll
  for (int b = 0; b < HB; ++b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) see(mv[b], Op<T>::unpack(vr[b][i]));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      mk[b] = fmaxf(mk[b], __shfl_xor(mk[b], d));
      mv[b] = fmaxf(mv[b], __shfl_xor(mv[b], d));
    }
    if ((tid & 63) == 0) {
      red[2 * b * UPR + (tid >> 6)] = mk[b];
      red[(2 * b + 1) * UPR + (tid >> 6)] = mv[b];
    }
  }
  __syncthreads();  // every thread has read the scales
#pragma unroll
  for (int b = 0; b < HB; ++b) {
    const float* m = red + 2 * b * UPR;  // (a wavefront for every unit of a row)
    float most_k = m[0], most_v = m[UPR];
#pragma unroll
    for (int i = 1; i < UPR; ++i) {
      most_k = fmaxf(most_k, m[i]);
      most_v = fmaxf(most_v, m[UPR + i]);
    }
    float sk = scale_for(most_k), sv = scale_for(most_v);
    if (off > 0) {
      sk = fmaxf(sk, old_k[b]);
      sv = fmaxf(sv, old_v[b]);
    }
    if (tid == 0) {
      a.ks[ph + b] = sk;
      a.vs[ph + b] = sv;
    }
    const float ik = inverse_pow2(sk), iv = inverse_pow2(sv);
    uint8_t *kc = a.kc + (ph + b) * P * D, *im = image + b * D * (64 + 4);  // im: new V codes, [d][P + 4]
    if (row < cnt) {
      *reinterpret_cast<u32x2v*>(kc + (off + row) * D + 8 * un.c0) = encode8(Op<T>::unpack(kr[b][0]), ik);
      *reinterpret_cast<u32x2v*>(kc + (off + row) * D + 8 * un.c1) = encode8(Op<T>::unpack(kr[b][1]), ik);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = tid + NT * i, r = e / CPR, c = e % CPR;
      if (r < cnt) {
        const u32x2v w = encode8(Op<T>::unpack(vr[b][i]), iv);
#pragma unroll
        for (int j = 0; j < 8; ++j) im[(8 * c + j) * (P + 4) + off + r] = uint8_t(w[j / 4] >> (8 * (j % 4)));
      }
    }
    if (off > 0 && sk > old_k[b]) {
      const float f = old_k[b] * ik;
      for (int e = tid; e < off * D / 4; e += NT) {
        uint32_t* p = reinterpret_cast<uint32_t*>(kc) + e;
        *p = recode4(*p, f);
      }
    }
    lds_barrier();
    store_v_image<D, NT>(a.vc + (ph + b) * P * D, im, P, off, cnt, off > 0 && sv > old_v[b], old_v[b] * iv, tid);
  }
}

__device__ __forceinline__ u32x4 recode16(const u32x4& x, float f) {
  return u32x4{recode4(x[0], f), recode4(x[1], f), recode4(x[2], f), recode4(x[3], f)};
}

// One wavefront for a page and key head, rows in passes of 64 / (D / 16): the form for few tokens to a page, where
// a workgroup's other lanes would have nothing to do.  Of several passes the last stays in registers, the others are
// turned again once the scale is known.
template <typename T, int D>
__device__ __forceinline__ void append_few(const CacheRopeArgs& ra, int64_t item, int lane, float* own) {
  const CacheAppendArgs& a = ra.c;
  const Rotation& t = ra.q.turn;
  constexpr int UPR = D / 16, RT = 64 / UPR;
  const int P = a.page, h = int(item % a.Hkv), slot = int(item / a.Hkv);
  int page;
  PageWork w;
  if (!page_work(a, slot, lane, page, w)) return;
  const int u = lane % UPR, passes = (w.cnt + RT - 1) / RT;
  const Unit un = unit_of(u, t.half);
  f32x8 v0, v1;
  float mk = 0.f, mv = 0.f;
  auto load = [&](int pass) {
    const int r = pass * RT + lane / UPR;
    typename Op<T>::frag f0{}, f1{}, g0{}, g1{};
    if (r < w.cnt) {
      const T* k = static_cast<const T*>(a.k) + (w.row0 + r) * ra.k_stride + h * D;
      const T* v = static_cast<const T*>(a.v) + (w.row0 + r) * ra.v_stride + h * D;
      f0 = Op<T>::load(k + 8 * un.c0);
      f1 = Op<T>::load(k + 8 * un.c1);
      g0 = Op<T>::load(v + 8 * un.c0);
      g1 = Op<T>::load(v + 8 * un.c1);
    }
    const f32x8 k0 = Op<T>::unpack(f0), k1 = Op<T>::unpack(f1);
    v0 = Op<T>::unpack(g0);
    v1 = Op<T>::unpack(g1);
    if (r >= w.cnt) return;
    to_column(own, k0, k1);
    if (un.turns) {
      turn_unit(t, w.row0 + r, w.p0 + r, u, own, mk);
    } else {
      see(mk, k0);
      see(mk, k1);
    }
    see(mv, v0);
    see(mv, v1);
  };
  for (int pass = 0; pass < passes; ++pass) load(pass);
  if (page < 0 || page >= a.pages) return;
  const int64_t ph = int64_t(page) * a.Hkv + h;
  const float old_k = a.ks[ph], old_v = a.vs[ph];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    mk = fmaxf(mk, __shfl_xor(mk, d));
    mv = fmaxf(mv, __shfl_xor(mv, d));
  }
  float sk = scale_for(mk), sv = scale_for(mv);
  if (w.off > 0) {
    sk = fmaxf(sk, old_k);
    sv = fmaxf(sv, old_v);
  }
  const float ik = inverse_pow2(sk), iv = inverse_pow2(sv);
  uint8_t *kc = a.kc + ph * P * D, *vc = a.vc + ph * P * D;
  // The earlier codes at a larger scale: every load on its way before the first is waited for.
  if (w.off > 0 && sk > old_k) {
    const float f = old_k * ik;
    u32x4 x[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      if (lane + 64 * j < w.off * (D / 16)) x[j] = reinterpret_cast<const u32x4*>(kc)[lane + 64 * j];
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      if (lane + 64 * j < w.off * (D / 16)) reinterpret_cast<u32x4*>(kc)[lane + 64 * j] = recode16(x[j], f);
  }
  if (w.off > 0 && sv > old_v) {
    // of a channel's row of tokens three times sixteen, three words and three bytes; what lies behind is not touched
    const float f = old_v * iv;
    const int n16 = w.off / 16, n4 = w.off % 16 / 4, n1 = w.off % 4;
    u32x4 x[D / 64][3];
    uint32_t y[D / 64][3], z[D / 64][3];
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint8_t* p = vc + (lane + 64 * j) * P;
        if (i < n16) x[j][i] = *reinterpret_cast<const u32x4*>(p + 16 * i);
        if (i < n4) y[j][i] = *reinterpret_cast<const uint32_t*>(p + 16 * n16 + 4 * i);
        if (i < n1) z[j][i] = p[16 * n16 + 4 * n4 + i];
      }
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        uint8_t* p = vc + (lane + 64 * j) * P;
        if (i < n16) *reinterpret_cast<u32x4*>(p + 16 * i) = recode16(x[j][i], f);
        if (i < n4) *reinterpret_cast<uint32_t*>(p + 16 * n16 + 4 * i) = recode4(y[j][i], f);
        if (i < n1) p[16 * n16 + 4 * n4 + i] = uint8_t(recode4(z[j][i], f));
      }
  }
  for (int pass = passes - 1; pass >= 0; --pass) {
    if (pass + 1 < passes) load(pass);
    const int r = pass * RT + lane / UPR;
    if (r < w.cnt) {
      *reinterpret_cast<u32x2v*>(kc + (w.off + r) * D + 8 * un.c0) = encode8(from_column(own), ik);
      *reinterpret_cast<u32x2v*>(kc + (w.off + r) * D + 8 * un.c1) = encode8(from_column(own + 8 * kColumns), ik);
      const u32x2v x0 = encode8(v0, iv), x1 = encode8(v1, iv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        vc[(8 * un.c0 + j) * P + w.off + r] = uint8_t(x0[j / 4] >> (8 * (j % 4)));
        vc[(8 * un.c1 + j) * P + w.off + r] = uint8_t(x1[j / 4] >> (8 * (j % 4)));
      }
    }
  }
  if (lane == 0) {
    a.ks[ph] = sk;
    a.vs[ph] = sv;
  }
}

// FORM 0: append_few, four (page, head) pairs to a workgroup; else append_page with FORM heads.  The queries' workgroups
// follow the pages': the two kinds in turn took 100 us where this order took 85 (14300 tokens, 32 and 8 heads of 128).
template <int D, int FORM> constexpr int kThreads = FORM == 0 ? 256 : 4 * D;
template <typename T, typename TO, int D, int FORM>
__global__ __launch_bounds__((kThreads<D, FORM>), (FORM == 0 ? 1 : 4)) void cache_append_rope_kernel(const CacheRopeArgs a, int pages) {
  constexpr int NW = kThreads<D, FORM> / 64, kRows = NW * 2 * kSines * 4, kImages = FORM * D * (64 + 4);  // rows' sines; V's codes
  static_assert(16 * kColumns * 4 <= kRows, "a wavefront's unit of keys");
  __shared__ __align__(16) uint8_t lds[kImages > kRows ? kImages : kRows];
  __shared__ float red[FORM == 0 ? 1 : 2 * FORM * NW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), id = int(blockIdx.x);
  if (id < pages) {
    if constexpr (FORM == 0) {
      const int64_t item = int64_t(id) * 4 + wave;
      if (item < (int64_t(a.c.n) / a.c.page + 2 * int64_t(a.c.N)) * a.c.Hkv) append_few<T, D>(a, item, lane, reinterpret_cast<float*>(lds) + threadIdx.x);
    } else {
      append_page<T, D, FORM>(a, id, lds, red);
    }
    return;
  }
  const int64_t item = (int64_t(id) - pages) * NW + wave;
  const int parts = (a.q.H + a.q.heads - 1) / a.q.heads, h0 = int(item % parts) * a.q.heads;
  const int64_t row = item / parts;
  if (row >= a.q.n) return;
  if (a.N == 0 || row >= rows_in_use(a.c.cu, a.N, a.q.n)) {
    if (a.zero_tail) {
      const int end = h0 + a.q.heads < a.q.H ? h0 + a.q.heads : a.q.H;
      TO* y = static_cast<TO*>(a.q.y) + row * a.q.y_stride;
      for (int e = h0 * (D / 8) + lane; e < end * (D / 8); e += 64) store8(y + 8 * int64_t(e), f32x8{0, 0, 0, 0, 0, 0, 0, 0});
    }
    return;
  }
  int64_t place = 0;
  if (!a.q.turn.pos) {
    const int i = sequence_of(a.c.cu, a.N, row, lane);
    const int64_t first = a.c.cu[i] < 0 ? 0 : a.c.cu[i], held = a.c.ctx[i] < 0 ? 0 : a.c.ctx[i];
    place = held + row - first;
  }
  rotate_rows<T, TO>(a.q, row, place, h0, reinterpret_cast<float(*)[kSines]>(lds) + 2 * wave, lane);
}

template <typename T, typename TO, int D, int FORM>
hipError_t launch(const CacheRopeArgs& a, hipStream_t st) {
  constexpr int NT = kThreads<D, FORM>, NW = NT / 64;
  const int64_t pairs = a.c.N > 0 ? (int64_t(a.c.n) / a.c.page + 2 * int64_t(a.c.N)) * a.c.Hkv : 0;
  const int64_t pages = FORM == 0 ? (pairs + 3) / 4 : pairs / (FORM == 0 ? 1 : FORM);
  const int64_t items = a.q.x ? rope_items(a.q) : 0;
  cache_append_rope_kernel<T, TO, D, FORM><<<dim3(uint32_t(pages + (items + NW - 1) / NW)), NT, 0, st>>>(a, int(pages));
  return hipGetLastError();
}

template <typename T, typename TO, int D>
hipError_t launch_form(const CacheRopeArgs& a, hipStream_t st) {
  // Few tokens to a sequence, and so to a page: 8 rows are one pass (d = 128) of one wavefront.  64 sequences of 8 tokens
  // take 9.4 us so and 11.9 by workgroups, of 16 tokens 20.2 and 14.5; 256 single tokens 13 and 31.
  // So do pages too many for one launch of the larger workgroups, which holds fewer than 2^32 threads.
  const int64_t pairs = (int64_t(a.c.n) / a.c.page + 2 * int64_t(a.c.N)) * a.c.Hkv, items = a.q.x ? rope_items(a.q) : 0;
  if (int64_t(a.c.n) <= 8 * int64_t(a.c.N) || (pairs + items + 1) * kThreads<D, 1> >= int64_t(1) << 32)
    return launch<T, TO, D, 0>(a, st);
  // Two heads that share the sines, where that leaves every compute unit three workgroups: 14300 tokens of 8 heads of 128
  // with 32 of queries take 78 us so and 80 by single heads, 2400 tokens of 64 sequences 25.3 and 24.5.
  if (a.c.Hkv % 2 == 0 && pairs >= 2 * 768) return launch<T, TO, D, 2>(a, st);
  return launch<T, TO, D, 1>(a, st);
}

template <typename T, typename TO>
hipError_t launch_d(const CacheRopeArgs& a, hipStream_t st) {
  return a.c.d == 64 ? launch_form<T, TO, 64>(a, st) : launch_form<T, TO, 128>(a, st);
}

}  // namespace

hipError_t launch_cache_append_rope(const CacheRopeArgs& a, hipStream_t st) {
  const bool out_bf16 = a.q.x ? a.q.out_bf16 : a.c.in_bf16;
  if (a.c.in_bf16) return out_bf16 ? launch_d<bf16_t, bf16_t>(a, st) : launch_d<bf16_t, float>(a, st);
  return out_bf16 ? launch_d<float, bf16_t>(a, st) : launch_d<float, float>(a, st);
}

}  // namespace kda
