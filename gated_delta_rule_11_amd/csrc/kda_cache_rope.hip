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

template <typename T, int D>
__device__ __forceinline__ void append_page(const CacheRopeArgs& ra, int id, uint8_t* image, float* red) {
  const CacheAppendArgs& a = ra.c;
  const Rotation& t = ra.q.turn;
  constexpr int CPR = D / 8, NV = 64 * CPR / 256;  // 8-element chunks of a row; chunks of a thread
  constexpr int UPR = D / 16, NK = 64 * UPR / 256;  // units of two chunks, of a row and of a thread
  const int tid = threadIdx.x, P = a.page, ps = page_shift(P);
  const int h = id % a.Hkv, slot = id / a.Hkv;

  // the last sequence whose pages start at or before this slot, 64 candidates at a time
  int lo = 0, up = a.N;
  while (up - lo > 1) {
    const int step = (up - lo + 63) / 64;
    const int64_t mid = lo + int64_t(step) * ((tid & 63) + 1);
    const bool before = mid < up && (a.cu[mid] >> ps) + 2 * mid <= slot;
    lo += step * __popcll(__ballot(before));
    up = lo + step < up ? lo + step : up;
  }
  int first = a.cu[lo], last = a.cu[lo + 1];
  const int64_t base = (first >> ps) + 2 * int64_t(lo);
  first = first < 0 ? 0 : first;
  last = last > a.n ? a.n : last;
  if (first >= last || slot < base) return;
  const int64_t held = a.ctx[lo] < 0 ? 0 : a.ctx[lo];
  const int64_t pi = (held >> ps) + (slot - base);
  const int64_t p0 = pi * P > held ? pi * P : held;
  const int64_t end = held + (last - first), p1 = (pi + 1) * P < end ? (pi + 1) * P : end;
  if (p0 >= p1 || pi >= a.max_pages) return;
  const int page = a.table[int64_t(lo) * a.max_pages + pi];
  if (page < 0 || page >= a.pages) return;
  const int off = int(p0 - pi * P), cnt = int(p1 - p0);
  const int64_t row0 = first + (p0 - held);
  const int64_t ph = int64_t(page) * a.Hkv + h;
  const float old_k = a.ks[ph], old_v = a.vs[ph];

  const f32x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  f32x8 k[NK][2], v[NV];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = tid + 256 * i, r = e / UPR;
    const Unit w = unit_of(e % UPR, t.half);
    const T* src = static_cast<const T*>(a.k) + (row0 + r) * ra.k_stride + h * D;
    k[i][0] = r < cnt ? Op<T>::unpack(Op<T>::load(src + 8 * w.c0)) : zero;
    k[i][1] = r < cnt ? Op<T>::unpack(Op<T>::load(src + 8 * w.c1)) : zero;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = tid + 256 * i, r = e / CPR, c = e % CPR;
    v[i] = r < cnt ? Op<T>::unpack(Op<T>::load(static_cast<const T*>(a.v) + (row0 + r) * ra.v_stride + h * D + 8 * c)) : zero;
  }
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = tid + 256 * i, r = e / UPR, u = e % UPR;
    if (r < cnt && unit_of(u, t.half).turns) {
      double c[8], s[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) sine_cosine(angle_of(t, row0 + r, p0 + r, pair_of(u, x, t.half, t.interleaved)), s[x], c[x]);
      turn(k[i][0], k[i][1], c, s, t.interleaved);
    }
  }
  float mk = 0.f, mv = 0.f;
  auto see = [](float& most, const f32x8& x) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(x[j]);
      if (m < INFINITY && m > most) most = m;
    }
  };
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    see(mk, k[i][0]);
    see(mk, k[i][1]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) see(mv, v[i]);
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
  auto encode8 = [](const f32x8& x, float inv) {
    u32x2v w;
    w[0] = encode4(to_range(x[0], inv), to_range(x[1], inv), to_range(x[2], inv), to_range(x[3], inv));
    w[1] = encode4(to_range(x[4], inv), to_range(x[5], inv), to_range(x[6], inv), to_range(x[7], inv));
    return w;
  };

  uint8_t* kc = a.kc + ph * P * D;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = tid + 256 * i, r = e / UPR;
    const Unit w = unit_of(e % UPR, t.half);
    if (r < cnt) {
      *reinterpret_cast<u32x2v*>(kc + (off + r) * D + 8 * w.c0) = encode8(k[i][0], ik);
      *reinterpret_cast<u32x2v*>(kc + (off + r) * D + 8 * w.c1) = encode8(k[i][1], ik);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = tid + 256 * i, r = e / CPR, c = e % CPR;
    if (r < cnt) {
      const u32x2v w = encode8(v[i], iv);
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

template <typename T, typename TO, int D>
__global__ __launch_bounds__(256) void cache_append_rope_kernel(const CacheRopeArgs a, int pages) {
  __shared__ __align__(16) uint8_t image[D * 68];  // new V codes, [d][P + 4]; or four rows' sines
  __shared__ float red[8];
  if (int(blockIdx.x) < pages) {
    append_page<T, D>(a, blockIdx.x, image, red);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t item = (int64_t(blockIdx.x) - pages) * 4 + wave;
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
  rotate_row<T, TO>(a.q, row, place, h0, reinterpret_cast<float(*)[128]>(image) + 2 * wave, lane);
}

template <typename T, typename TO, int D>
hipError_t launch(const CacheRopeArgs& a, hipStream_t st) {
  const int64_t pages = a.c.N > 0 ? (int64_t(a.c.n) / a.c.page + 2 * int64_t(a.c.N)) * a.c.Hkv : 0;
  const int64_t items = a.q.x ? int64_t(a.q.n) * ((a.q.H + a.q.heads - 1) / a.q.heads) : 0;
  cache_append_rope_kernel<T, TO, D><<<dim3(uint32_t(pages + (items + 3) / 4)), 256, 0, st>>>(a, int(pages));
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t launch_d(const CacheRopeArgs& a, hipStream_t st) {
  return a.c.d == 64 ? launch<T, TO, 64>(a, st) : launch<T, TO, 128>(a, st);
}

}  // namespace

hipError_t launch_cache_append_rope(const CacheRopeArgs& a, hipStream_t st) {
  const bool out_bf16 = a.q.x ? a.q.out_bf16 : a.c.in_bf16;
  if (a.c.in_bf16) return out_bf16 ? launch_d<bf16_t, bf16_t>(a, st) : launch_d<bf16_t, float>(a, st);
  return out_bf16 ? launch_d<float, bf16_t>(a, st) : launch_d<float, float>(a, st);
}

}  // namespace kda
