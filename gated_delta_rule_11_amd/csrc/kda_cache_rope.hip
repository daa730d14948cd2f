// kda_cache_rope.hip -- appending to the paged 8-bit cache with the rotary positions applied to the keys
// on the way, and to the same tokens' queries.
//
// Workgroups of two kinds in one launch: one for each (touched page, key head), as in plain appending
// (kda_cache.hip), and behind them one for every four rows of queries.  Keys are turned in 64 bits and
// rounded once: the codes are those of the exactly turned keys, whatever the inputs' type.
// (From turned keys rounded to bf16 one code in eight would differ, from fp32 ones one in some millions.)
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

// A unit of k turned in 64 bits, its 16 channels in `own`, a column of the thread's own in LDS: with the channels in
// registers the eight pairs would have to be written out, and their terms held at once (160 registers against 90).
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

// One workgroup for a page and key head: all of its rows at once in registers.
template <typename T, int D>
__device__ __forceinline__ void append_page(const CacheRopeArgs& ra, int id, uint8_t* lds, float* red) {
  const CacheAppendArgs& a = ra.c;
  const Rotation& t = ra.q.turn;
  constexpr int CPR = D / 8, NV = 64 * CPR / 256;  // 8-element chunks of a row; chunks of a thread
  constexpr int UPR = D / 16, NK = 64 * UPR / 256;  // units of two chunks, of a row and of a thread
  const int tid = threadIdx.x, P = a.page;
  const int h = id % a.Hkv, slot = id / a.Hkv;

  int page;
  PageWork w;
  if (!page_work(a, slot, tid & 63, page, w)) return;
  if (page < 0 || page >= a.pages) return;
  const int off = w.off, cnt = w.cnt;
  const int64_t row0 = w.row0, p0 = w.p0, ph = int64_t(page) * a.Hkv + h;
  const float old_k = a.ks[ph], old_v = a.vs[ph];

  typedef typename Op<T>::frag F;
  F kr[NK][2], vr[NV];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = tid + 256 * i, r = e / UPR;
    const Unit w = unit_of(e % UPR, t.half);
    const T* src = static_cast<const T*>(a.k) + (row0 + r) * ra.k_stride + h * D;
    kr[i][0] = kr[i][1] = F{};
    if (r < cnt) {
      kr[i][0] = Op<T>::load(src + 8 * w.c0);
      kr[i][1] = Op<T>::load(src + 8 * w.c1);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = tid + 256 * i, r = e / CPR, c = e % CPR;
    vr[i] = F{};
    if (r < cnt) vr[i] = Op<T>::load(static_cast<const T*>(a.v) + (row0 + r) * ra.v_stride + h * D + 8 * c);
  }
  // The turned keys wait in LDS for the scale.
  float* const own = reinterpret_cast<float*>(lds) + tid;
  float mk = 0.f, mv = 0.f;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = tid + 256 * i, r = e / UPR, u = e % UPR;
    const f32x8 x0 = Op<T>::unpack(kr[i][0]), x1 = Op<T>::unpack(kr[i][1]);
    if (r < cnt) {
      to_column(own + 16 * i * kColumns, x0, x1);
      if (unit_of(u, t.half).turns) {
        turn_unit(t, row0 + r, p0 + r, u, own + 16 * i * kColumns, mk);
      } else {
        see(mk, x0);
        see(mk, x1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) see(mv, Op<T>::unpack(vr[i]));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    mk = fmaxf(mk, __shfl_xor(mk, d));
    mv = fmaxf(mv, __shfl_xor(mv, d));
  }
  if ((tid & 63) == 0) {
    red[tid >> 6] = mk;
    red[4 + (tid >> 6)] = mv;
  }
  __syncthreads();  // every thread has read the scales
  float sk = scale_for(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  float sv = scale_for(fmaxf(fmaxf(red[4], red[5]), fmaxf(red[6], red[7])));
  if (off > 0) {
    sk = fmaxf(sk, old_k);
    sv = fmaxf(sv, old_v);
  }
  if (tid == 0) {
    a.ks[ph] = sk;
    a.vs[ph] = sv;
  }
  const float ik = inverse_pow2(sk), iv = inverse_pow2(sv);
  uint8_t* kc = a.kc + ph * P * D;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = tid + 256 * i, r = e / UPR;
    const Unit w = unit_of(e % UPR, t.half);
    if (r < cnt) {
      *reinterpret_cast<u32x2v*>(kc + (off + r) * D + 8 * w.c0) = encode8(from_column(own + 16 * i * kColumns), ik);
      *reinterpret_cast<u32x2v*>(kc + (off + r) * D + 8 * w.c1) = encode8(from_column(own + (16 * i + 8) * kColumns), ik);
    }
  }
  lds_barrier();  // the keys are out of the LDS
  uint8_t* const image = lds;  // new V codes, [d][P + 4]
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = tid + 256 * i, r = e / CPR, c = e % CPR;
    if (r < cnt) {
      const u32x2v w = encode8(Op<T>::unpack(vr[i]), iv);
#pragma unroll
      for (int j = 0; j < 8; ++j) image[(8 * c + j) * (P + 4) + off + r] = uint8_t(w[j / 4] >> (8 * (j % 4)));
    }
  }
  if (off > 0 && sk > old_k) {
    const float f = old_k * ik;
    for (int e = tid; e < off * D / 4; e += 256) {
      uint32_t* p = reinterpret_cast<uint32_t*>(kc) + e;
      *p = recode4(*p, f);
    }
  }
  __syncthreads();
  store_v_image<D>(a.vc + ph * P * D, image, P, off, cnt, off > 0 && sv > old_v, old_v * iv, tid);
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
  if (w.off > 0 && sk > old_k) {
    const float f = old_k * ik;
#pragma unroll 4
    for (int e = lane; e < w.off * D / 4; e += 64) {
      uint32_t* p = reinterpret_cast<uint32_t*>(kc) + e;
      *p = recode4(*p, f);
    }
  }
  if (w.off > 0 && sv > old_v) {
    const float f = old_v * iv;
    const int words = w.off / 4, rest = w.off % 4;  // of a channel's row of tokens; what lies behind them is not touched
#pragma unroll 4
    for (int e = lane; e < D * words; e += 64) {
      uint32_t* p = reinterpret_cast<uint32_t*>(vc + (e / words) * P) + e % words;
      *p = recode4(*p, f);
    }
    for (int e = lane; e < D * rest; e += 64) {
      uint8_t* p = vc + (e / rest) * P + 4 * words + e % rest;
      *p = uint8_t(recode4(*p, f));
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

// FEW: append_few, four (page, head) pairs to a workgroup; else one.  The queries' workgroups follow the pages': the two
// kinds in turn took 100 us where this order takes 85 (14300 tokens, 32 and 8 heads of 128).
template <typename T, typename TO, int D, bool FEW>
__global__ __launch_bounds__(256) void cache_append_rope_kernel(const CacheRopeArgs a, int pages) {
  __shared__ __align__(16) uint8_t lds[FEW ? 16 * kColumns * 4 : 64 * D * 4];  // (also four rows' sines)
  __shared__ float red[8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), id = int(blockIdx.x);
  if (id < pages) {
    if constexpr (FEW) {
      const int64_t item = int64_t(id) * 4 + wave;
      if (item < (int64_t(a.c.n) / a.c.page + 2 * int64_t(a.c.N)) * a.c.Hkv) append_few<T, D>(a, item, lane, reinterpret_cast<float*>(lds) + threadIdx.x);
    } else {
      append_page<T, D>(a, id, lds, red);
    }
    return;
  }
  const int64_t item = (int64_t(id) - pages) * 4 + wave;
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

template <typename T, typename TO, int D, bool FEW>
hipError_t launch(const CacheRopeArgs& a, hipStream_t st) {
  const int64_t pairs = a.c.N > 0 ? (int64_t(a.c.n) / a.c.page + 2 * int64_t(a.c.N)) * a.c.Hkv : 0;
  const int64_t pages = FEW ? (pairs + 3) / 4 : pairs;
  const int64_t items = a.q.x ? rope_items(a.q) : 0;
  cache_append_rope_kernel<T, TO, D, FEW><<<dim3(uint32_t(pages + (items + 3) / 4)), 256, 0, st>>>(a, int(pages));
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t launch_d(const CacheRopeArgs& a, hipStream_t st) {
  // few tokens to a sequence, and so to a page: 16 rows are two passes (d = 128) of one wavefront
  const bool few = int64_t(a.c.n) <= 16 * int64_t(a.c.N);
  if (a.c.d == 64) return few ? launch<T, TO, 64, true>(a, st) : launch<T, TO, 64, false>(a, st);
  return few ? launch<T, TO, 128, true>(a, st) : launch<T, TO, 128, false>(a, st);
}

}  // namespace

hipError_t launch_cache_append_rope(const CacheRopeArgs& a, hipStream_t st) {
  const bool out_bf16 = a.q.x ? a.q.out_bf16 : a.c.in_bf16;
  if (a.c.in_bf16) return out_bf16 ? launch_d<bf16_t, bf16_t>(a, st) : launch_d<bf16_t, float>(a, st);
  return out_bf16 ? launch_d<float, bf16_t>(a, st) : launch_d<float, float>(a, st);
}

}  // namespace kda
