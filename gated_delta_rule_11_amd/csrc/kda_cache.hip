// kda_cache.hip -- a paged key-value cache held in 8 bits, and single-token attention over it.
//
// A page holds P tokens (16, 32 or 64) of one sequence.  For each page and key head, K and V have
// one scale each, a power of two: the smallest 2^k with max |x| <= 448 2^k, 448 being the largest
// e4m3 value; a value is held as round(x / 2^k) (nearest even), so every quotient is exact and
// the only rounding is the 8-bit one, at most 2^-4 of the value.  A token added to a page already
// begun may need a larger scale; the page's earlier values are then rounded again at it.
//
// Layout: K pages [page, Hkv, P, d], V pages [page, Hkv, d, P].  V's tokens are contiguous because
// the second product sums over them: both operands then load as they lie, 16 bytes a lane.
#include "kda_cache.hpp"

namespace kda {

namespace {

// Appending.  One workgroup per (touched page, key head): the new tokens' largest magnitudes,
// the scales, the codes.  Sequence i's pages sit at slots cu[i] / P + 2 i onwards: n new tokens
// touch at most n / P + 2 pages, and these starts leave at least that many slots to each sequence,
// so a slot finds its sequence by a search over cu alone.  One workgroup to a page because a page
// has one scale, which all of its values wait for.  Measured (bf16, 8 heads, d = 128, pages of 64):
// 5 sequences with 400 to 6000 new tokens each, 88 MB, 28.7 us, 3.1 TB/s (17.5 us at a copy's
// rate), for the latency of each workgroup's chain of search, load, maximum, scale, store (more of
// them at once, or wider LDS stores of V's codes, did not shorten it); 256 single tokens 17.7 us:
// the same chain, and one byte to each of V's 262144 rows of tokens.
template <typename T, int D>
__global__ __launch_bounds__(256) void cache_append_kernel(const CacheAppendArgs a) {
  constexpr int CPR = D / 8, N = 64 * CPR / 256;  // 8-element chunks of a row; chunks of a thread
  __shared__ __align__(16) uint8_t image[D * 68];               // new V codes, [d][P + 4]
  __shared__ float red[8];
  const int tid = threadIdx.x, P = a.page, ps = page_shift(P);
  const int h = blockIdx.x % a.Hkv, slot = blockIdx.x / a.Hkv;

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

  f32x8 x[2][N];
  float amax[2] = {0.f, 0.f};
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const T* src = static_cast<const T*>(side ? a.v : a.k);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = tid + 256 * i, r = e / CPR, c = e % CPR;
      x[side][i] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
      if (r < cnt) x[side][i] = Op<T>::unpack(Op<T>::load(src + ((row0 + r) * a.Hkv + h) * D + 8 * c));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(x[side][i][j]);
        if (m < INFINITY && m > amax[side]) amax[side] = m;
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    amax[0] = fmaxf(amax[0], __shfl_xor(amax[0], d));
    amax[1] = fmaxf(amax[1], __shfl_xor(amax[1], d));
  }
  if ((tid & 63) == 0) {
    red[tid >> 6] = amax[0];
    red[4 + (tid >> 6)] = amax[1];
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
  for (int i = 0; i < N; ++i) {
    const int e = tid + 256 * i, r = e / CPR, c = e % CPR;
    if (r < cnt) {
      const f32x8 y = x[0][i], z = x[1][i];
      u32x2v w;
      w[0] = encode4(to_range(y[0], ik), to_range(y[1], ik), to_range(y[2], ik), to_range(y[3], ik));
      w[1] = encode4(to_range(y[4], ik), to_range(y[5], ik), to_range(y[6], ik), to_range(y[7], ik));
      *reinterpret_cast<u32x2v*>(kc + (off + r) * D + 8 * c) = w;
      w[0] = encode4(to_range(z[0], iv), to_range(z[1], iv), to_range(z[2], iv), to_range(z[3], iv));
      w[1] = encode4(to_range(z[4], iv), to_range(z[5], iv), to_range(z[6], iv), to_range(z[7], iv));
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

// Attention of one query token per sequence.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = e^{scale q . k_j}
//
// One workgroup per (sequence, key head, up to 16 query heads of its group, part of the context);
// each of its four wavefronts takes every fourth tile of 64 tokens and keeps its own running
// maximum, sum and accumulators; they are joined through LDS, and the parts of a context by a
// second small kernel.  Bound by the cache's bytes: a lane's loads are 16 bytes and the next
// tile's are in flight while one is used.  Measured (bf16 queries, 32 heads on 8, d = 128): 256
// sequences of 1 to 4096 tokens 219 us, 5.2 TB/s, a large copy's rate; one of 131072 tokens 57 us,
// 4.7 TB/s, with a join of 6 us in it.  Scores are formed transposed, S^T = K Q^T, on
// 16x16x32 products whose 64 rows are dealt so that group g of 16 lanes ends up with tokens
// 16 g .. + 15 of its column's head: row r of product t is token 16 (r / 4) + 4 t + r % 4.  The
// probabilities are then in place as the operand of O^T = V^T P^T, and V's 16 tokens of a lane are one load.
// Codes are exact in bf16; the scales (powers of two) multiply scores and probabilities in fp32
// and cost nothing; with bf16 queries P is rounded to bf16, 2^-8 of each term, as a bf16 output is.
// fp32 queries and their probabilities go in as three bf16 parts that sum to them: every product
// is exact, and three bf16 instructions take a fifth of the time of the eight fp32 ones.
template <typename T, typename TO, int D>
__global__ __launch_bounds__(256, 2) void cache_step_kernel(const CacheStepArgs a) {
  using O = Op<bf16_t>;
  constexpr int NM = D / 64, ND = D / 16, NP = sizeof(T) == 2 ? 1 : 3;
  using Parts8 = Parts<bf16_t, NP, 8>;
  __shared__ float jm[4][16], jl[4][16];
  __shared__ float jo[4][16][D + 4];
  // the parts of fp32 queries, fragment by fragment (in registers they would push out the next tile)
  __shared__ bf16x8 qs[NP == 3 ? NM * 2 * NP : 1][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r16 = lane & 15, g4 = lane >> 4;
  const int G = a.Hq / a.Hkv, GT = (G + 15) / 16;
  int id = blockIdx.x;
  const int sp = id % a.splits;
  id /= a.splits;
  const int gt = id % GT;
  id /= GT;
  const int kvh = id % a.Hkv, n = id / a.Hkv;
  const int P = a.page, ps = page_shift(P);
  const int64_t room = int64_t(a.max_pages) * P;
  int64_t ctx = a.ctx[n] < 0 ? 0 : a.ctx[n];
  ctx = ctx < room ? ctx : room;
  const int64_t nt = (ctx + 63) / 64, per = (nt + a.splits - 1) / a.splits;
  const int64_t t0 = sp * per, t1 = t0 + per < nt ? t0 + per : nt;
  const int hd = gt * 16 + r16;  // this lane's head within the group
  const int head = kvh * G + hd;
  const int* table = a.table + int64_t(n) * a.max_pages;

  bf16x8 qf[NM][2];
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f32x8 x = {0, 0, 0, 0, 0, 0, 0, 0};
      if (hd < G)
        x = Op<T>::unpack(Op<T>::load(static_cast<const T*>(a.q) + (int64_t(n) * a.Hq + head) * D + 16 * (g4 + 4 * m) + 8 * e));
      const Parts8 xp(x);
      if constexpr (NP == 1) qf[m][e] = part_of(xp, 0);
      else if (wave == 0)
#pragma unroll
        for (int p = 0; p < NP; ++p) qs[(m * 2 + e) * NP + p][lane] = part_of(xp, p);
    }
  if constexpr (NP == 3) __syncthreads();
  const float c = a.scale * kLog2e;

  struct Tile64 {
    u32x4 k[4][NM], v[ND];
    float ks, vs;
    bool live;  // this lane's 16 tokens lie in a page of the cache
  };
  auto load = [&](Tile64& x, int64_t t) {
    const int64_t tok = t * 64;
    int pk = -1, pv = -1;
    if (tok + 16 * (r16 >> 2) < ctx) pk = table[(tok + 16 * (r16 >> 2)) >> ps];
    if (tok + 16 * g4 < ctx) pv = table[(tok + 16 * g4) >> ps];
    const bool lk = pk >= 0 && pk < a.pages;
    x.live = pv >= 0 && pv < a.pages;
    const int64_t kh = int64_t(lk ? pk : 0) * a.Hkv + kvh, vh = int64_t(x.live ? pv : 0) * a.Hkv + kvh;
    const uint8_t* kp = a.kc + (kh * P + ((16 * (r16 >> 2)) & (P - 1)) + (r16 & 3)) * D + 16 * g4;
    const uint8_t* vp = a.vc + (vh * D + r16) * P + ((16 * g4) & (P - 1));
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int m = 0; m < NM; ++m)
        x.k[q][m] = lk ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(kp + 4 * q * D + 64 * m)) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < ND; ++d)
      x.v[d] = x.live ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(vp + 16 * d * P)) : u32x4{0, 0, 0, 0};
    x.ks = x.live ? a.ks[vh] : 0.f;
    x.vs = x.live ? a.vs[vh] : 0.f;
  };

  f32x4 acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = f32x4{0, 0, 0, 0};
  float m_ = -INFINITY, l = 0.f;

  auto use = [&](Tile64& x, int64_t t) {
    const int64_t left = ctx - (t * 64 + 16 * g4);  // live tokens from this lane's first on
    int ql = lane;
    if constexpr (NP == 3) asm volatile("" : "+v"(ql));  // read again for each tile
    f32x4 s[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        bf16x8 kf[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) kf[q] = codes(x.k[q][m][2 * e], x.k[q][m][2 * e + 1]);
#pragma unroll
        for (int p = NP - 1; p >= 0; --p) {
          bf16x8 qp;
          if constexpr (NP == 1) qp = qf[m][e];
          else qp = qs[(m * 2 + e) * NP + p][ql];
#pragma unroll
          for (int q = 0; q < 4; ++q) s[q] = O::mma16(kf[q], qp, s[q]);
        }
      }
    const float cs = c * x.ks;
    float mt = -INFINITY;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[q][i] = x.live && 4 * q + i < left ? s[q][i] * cs : -INFINITY;
        mt = fmaxf(mt, s[q][i]);
      }
    mt = max_groups(mt);
    if (__any(mt > m_)) {
      const float mn = fmaxf(m_, mt);
      const float al = fast_exp2(m_ - (mn == -INFINITY ? 0.f : mn));
      l *= al;
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[d] *= al;
      m_ = mn;
    }
    const float ref = m_ == -INFINITY ? 0.f : m_;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[q][i] = fast_exp2(s[q][i] - ref);
        l += s[q][i];
        s[q][i] *= x.vs;
      }
    if (left < 16) {  // what lies behind the last token may be anything, NaN too
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int nb = int(left < 0 ? 0 : left) - 4 * w;
        const uint32_t mask = nb >= 4 ? 0xffffffffu : (nb <= 0 ? 0u : (1u << (8 * nb)) - 1u);
#pragma unroll
        for (int d = 0; d < ND; ++d) x.v[d][w] &= mask;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const f32x8 p8 = __builtin_shufflevector(s[2 * u], s[2 * u + 1], 0, 1, 2, 3, 4, 5, 6, 7);
      const Parts8 pf(p8);
#pragma unroll
      for (int d0 = 0; d0 < ND; d0 += 4) {
        bf16x8 vf[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) vf[d] = codes(x.v[d0 + d][2 * u], x.v[d0 + d][2 * u + 1]);
#pragma unroll
        for (int p = NP - 1; p >= 0; --p)
#pragma unroll
          for (int d = 0; d < 4; ++d) acc[d0 + d] = O::mma16(vf[d], part_of(pf, p), acc[d0 + d]);
      }
    }
  };

  Tile64 x, y;
  int64_t t = t0 + wave;
  if (t < t1) load(x, t);
  for (; t < t1; t += 8) {
    if (t + 4 < t1) load(y, t + 4);
    use(x, t);
    if (t + 8 < t1) load(x, t + 8);
    if (t + 4 < t1) use(y, t + 4);
  }
  l = sum_groups(l);

  if (g4 == 0) {
    jm[wave][r16] = m_;
    jl[wave][r16] = l;
  }
#pragma unroll
  for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(&jo[wave][r16][16 * d + 4 * g4]) = acc[d];
  __syncthreads();
  for (int e = tid; e < 16 * D; e += 256) {
    const int hh = e / D, d = e % D;
    if (gt * 16 + hh >= G) continue;
    float mm = fmaxf(fmaxf(jm[0][hh], jm[1][hh]), fmaxf(jm[2][hh], jm[3][hh]));
    const float ref = mm == -INFINITY ? 0.f : mm;
    float ls = 0.f, os = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = fast_exp2(jm[w][hh] - ref);
      ls += f * jl[w][hh];
      os += f * jo[w][hh][d];
    }
    const int64_t row = int64_t(n) * a.Hq + kvh * G + gt * 16 + hh;
    if (a.splits == 1) {
      io<TO>::store(static_cast<TO*>(a.o), row * D + d, ls == 0.f ? 0.f : os / ls);
      if (a.lse && d == 0) a.lse[row] = (mm + log2f(ls)) * 0.6931471805599453f;
    } else {
      float* p = a.part + (row * a.splits + sp) * (D + 2);
      p[2 + d] = os;
      if (d == 0) {
        p[0] = mm;
        p[1] = ls;
      }
    }
  }
}

// Joins the parts of a context: one workgroup per (sequence, query head).  256 / D groups of
// D threads take the parts in turn, so that the loads of many are in flight.
template <typename TO, int D>
__global__ __launch_bounds__(256) void cache_join_kernel(const float* part, TO* o, float* lse, int splits) {
  constexpr int NG = 256 / D;
  __shared__ float sm[4], sl[NG][D], sx[NG][D];
  const int tid = threadIdx.x, d = tid % D, grp = tid / D;
  const int64_t row = blockIdx.x;
  const float* p = part + row * splits * (D + 2);
  float m = -INFINITY;
  for (int s = tid; s < splits; s += 256) m = fmaxf(m, p[int64_t(s) * (D + 2)]);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
  if ((tid & 63) == 0) sm[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, x = 0.f;
#pragma unroll 8
  for (int s = grp; s < splits; s += NG) {
    const float* ps = p + int64_t(s) * (D + 2);
    const float f = fast_exp2(ps[0] - ref);
    l += f * ps[1];
    x += f * ps[2 + d];
  }
  sl[grp][d] = l;
  sx[grp][d] = x;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int g = 1; g < NG; ++g) {
      l += sl[g][d];
      x += sx[g][d];
    }
    io<TO>::store(o, row * D + d, l == 0.f ? 0.f : x / l);
    if (lse && d == 0) lse[row] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <typename T, typename TO, int D>
hipError_t launch_step(const CacheStepArgs& a, hipStream_t st) {
  const int GT = (a.Hq / a.Hkv + 15) / 16;
  cache_step_kernel<T, TO, D><<<dim3(uint32_t(int64_t(a.N) * a.Hkv * GT * a.splits)), 256, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  cache_join_kernel<TO, D><<<dim3(uint32_t(int64_t(a.N) * a.Hq)), 256, 0, st>>>(a.part, static_cast<TO*>(a.o), a.lse,
                                                                               a.splits);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_step_o(const CacheStepArgs& a, hipStream_t st) {
  return a.out_bf16 ? launch_step<T, bf16_t, D>(a, st) : launch_step<T, float, D>(a, st);
}

template <typename T, int D>
hipError_t launch_append(const CacheAppendArgs& a, hipStream_t st) {
  const int64_t slots = int64_t(a.n) / a.page + 2 * int64_t(a.N);
  cache_append_kernel<T, D><<<dim3(uint32_t(slots * a.Hkv)), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const CacheAppendArgs& a, hipStream_t st) {
  if (a.in_bf16) return a.d == 64 ? launch_append<bf16_t, 64>(a, st) : launch_append<bf16_t, 128>(a, st);
  return a.d == 64 ? launch_append<float, 64>(a, st) : launch_append<float, 128>(a, st);
}

// Parts of a context: enough workgroups to fill the GPU with a few each, none with less than one
// tile for each of its wavefronts.  The rule goes by max_pages and the batch, not by each context's length:
// from 1024 sequence and key head pairs on no context is cut, and one that is far longer than the others ends
// late (8 key heads: one of 131072 tokens among 31, 127 or 255 of 1024 takes 317, 1236, 1243 us; alone 58).
// Measured, 512 : 1024 : 2048 workgroups, us, 8 key heads, d = 128:
// contexts alike, 1 of 131072 tokens 54 : 57 : 65, 8 of 16384 53 : 54 : 58; contexts of any length up
// to 16384, 8 of them 37 : 32 : 39, 32 of them 142 : 125 : 123.
int cache_step_splits(int N, int Hq, int Hkv, int page, int max_pages) {
  const int64_t units = int64_t(N) * Hkv * ((Hq / Hkv + 15) / 16);
  const int64_t tiles = (int64_t(max_pages) * page + 63) / 64;
  int64_t s = 1024 / (units < 1 ? 1 : units);
  const int64_t most = (tiles + 3) / 4;
  s = s < most ? s : most;
  return int(s < 1 ? 1 : s);
}

hipError_t launch_cache_step(const CacheStepArgs& a, hipStream_t st) {
  if (a.in_bf16) return a.d == 64 ? launch_step_o<bf16_t, 64>(a, st) : launch_step_o<bf16_t, 128>(a, st);
  return a.d == 64 ? launch_step_o<float, 64>(a, st) : launch_step_o<float, 128>(a, st);
}

}  // namespace kda
