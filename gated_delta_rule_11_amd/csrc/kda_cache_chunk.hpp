// kda_cache_chunk.hpp -- attention of a chunk of new tokens over the paged 8-bit cache.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = e^{scale q_r . k_j},  j <= ctx - new + (r's token)
//
// The new tokens of sequence i are the last of its ctx tokens, all of them in the cache.  The query heads
// of a group read the same keys, so the rows of a tile are (token, head of the group) pairs, 128 of them.
//
// Tiles of more than 32 rows ("wide"): four wavefronts of 32 rows walk the keys in steps of 64.  A
// step's codes are loaded 16 to a lane as they lie, turned into bf16 values (scale and all, exact)
// once for all four wavefronts, and put into LDS while the step before is multiplied.  Tiles of up to 32
// rows ("narrow": single tokens, drafted tokens) are bound by the cache's bytes: each wavefront takes
// every fourth step for all rows, codes go straight to registers, and the four are joined at the end.
//
// Scores are formed transposed, S^T = K Q^T, with the rows of K dealt so that a lane ends up with runs of eight
// consecutive tokens of one query row; P is then in place as the operand of O^T = V^T P^T, and V's pages,
// [d][token], are that product's other operand as they lie.
//
// What bounds it (MI355X, 32 heads on 8 of 128, bf16): long chunks by the products and what stands between them, 1024 tokens
// behind 64511 in 1110 to 1140 us, 957 to 980 TFLOP/s, where the matrix pipe is busy in 43 % of the cycles and the rest goes to
// the exponentials, the conversions of codes and the LDS (an 8192^3 library product reaches 1070 to 1110 on such cards);
// drafted tokens by the cache's bytes, 64 x 5 tokens over up to 8192 in 104 us and 7 for the joins, 4.7 TB/s; whole prompts of
// 500 to 2048 tokens, 110 us for 69 GFLOP, by the order of the tiles (counted with the long chunk's 2.2 us a step, a long
// sequence that starts late costs 20 us) and the 5 us that each takes to start and to end (pages, queries, first codes,
// outputs; 13 us in all).  A wavefront that
// forms the scores of the next step beside the products of this one needs more registers than two to a SIMD have (135 us
// grew to 170), 64 rows to a wavefront likewise; orders asked of the scheduler changed nothing.
//
// Sums and statistics are fp32.  bf16 queries: P is rounded to bf16, 2^-8 of a term, as a bf16 output is.  fp32
// queries and their P go in as three bf16 parts that sum to them: against the codes' exact values
// every product is exact.  The reference that exponents are taken to stays up to 2^8 above the
// largest score seen, so that p <= 1 and most steps leave the accumulators alone.
//
// The sums of p v are divided at the end only: values of 2^119 and more can take them beyond fp32 although the mean is
// not.  A tile that ends with a sum that is not finite and has such values in its pages is done once more with the values
// 2^-26 times what they are, and l likewise: sums of up to 2^26 tokens then stay finite.  (The look at the sums and the
// way back: 1 % of the times above.)
#pragma once

#include "kda_cache.hpp"

namespace kda {

constexpr int kNarrowRows = 32;
constexpr int kShrinkBits = 26;  // (the least scale, 2^-100, stays a normal number)

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(x)), hi = __builtin_amdgcn_readfirstlane(uint32_t(uint64_t(x) >> 32));
  return int64_t(uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Sixteen codes without those whose value (code times a power of two) is no finite fp32 number: NaN, and
// from a scale of 2^120 on the largest; whether there were any.  By bytes: a magnitude plus 128 less the least
// such magnitude carries into the sign's place.  (NAN_INSTEAD: those codes become NaN instead.)
template <bool NAN_INSTEAD = false>
__device__ __forceinline__ bool finite_codes(u32x4& w, float scale) {
  const int k = int(__float_as_uint(scale) >> 23) - 127;
  int least = (135 - k) * 8;  // the magnitude of 2^(128 - k)
  least = least > 0x7f ? 0x7f : (least < 1 ? 1 : least);
  const uint32_t add = 0x01010101u * uint32_t(0x80 - least);
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = ((w[i] & 0x7f7f7f7fu) + add) & 0x80808080u;
    any |= m;
    if constexpr (NAN_INSTEAD) w[i] |= m - (m >> 7);
    else w[i] &= ~((m << 1) - (m >> 7));
  }
  return any != 0;
}

// ---- the division of the work -------------------------------------------------------------
//
// Cost of a tile, in units of (64 keys, one head of a group): its steps, weighted, and a start.  Linear
// in the tile's number, so that a sequence's sum is a closed form.  A narrow step at half a wide one's cost (at a quarter
// 26 single tokens among 6 chunks take 180 us, at three eighths 148, at a half 133); a start of 16 instead of 20 gives the
// same batch 138 and four prompts 120 for 122, of 12 135 and 122; a workgroup takes no less than kLeastCost, so that short
// work is not cut into starts alone (16 and 24 differ by 3 %).
constexpr int64_t kNarrowCost = 2, kWideCost = 4, kStartCost = 20, kLeastCost = 16;

struct ChunkSeq {
  int first, len, ctx;  // rows of q, new tokens, tokens held
};
__device__ __forceinline__ ChunkSeq chunk_seq(const CacheChunkArgs& a, int i) {
  int first = a.cu[i], last = a.cu[i + 1];
  first = first < 0 ? 0 : first;
  last = last > a.n ? a.n : last;
  const int c = a.ctx[i];
  return {first, last > first ? last - first : 0, c < 0 ? 0 : c};
}
__device__ __forceinline__ ChunkSeq uniform(const ChunkSeq& s) { return {uniform(s.first), uniform(s.len), uniform(s.ctx)}; }

struct ChunkCost {
  int64_t tiles, wide, last;  // wide tile t costs wide + 2 kWideCost t; the last one `last`
  __device__ __forceinline__ ChunkCost(const CacheChunkArgs& a, const ChunkSeq& s) {
    const int64_t G = a.Hq / a.Hkv, room = int64_t(a.max_pages) * a.page;
    const int64_t R = int64_t(s.len) * G, ctx = s.ctx < room ? int64_t(s.ctx) : room;
    const int64_t base = ctx > s.len ? ctx - s.len : 0;
    tiles = (R + kChunkRows - 1) / kChunkRows;
    wide = kWideCost * ((base >> 6) * G + 2) + kStartCost * G;
    const bool narrow = R - (tiles - 1) * kChunkRows <= kNarrowRows;
    last = tiles == 0 ? 0 : (narrow ? kNarrowCost : kWideCost) * (((ctx + 63) >> 6) * G) + kStartCost * G;
  }
  __device__ __forceinline__ int64_t before(int64_t t) const { return wide * t + kWideCost * t * (t - 1); }  // t < tiles
  __device__ __forceinline__ int64_t of(int64_t t) const { return t + 1 == tiles ? last : wide + 2 * kWideCost * t; }
  __device__ __forceinline__ int64_t all() const { return tiles == 0 ? 0 : before(tiles - 1) + last; }
  // the tile at x of the sequence's line: the root of before(t) = x, and the tiles beside it
  __device__ __forceinline__ int64_t at(int64_t x) const {
    const double b = double(wide - kWideCost);
    int64_t t = int64_t((__builtin_sqrt(b * b + 4.0 * kWideCost * double(x)) - b) / (2.0 * kWideCost));
    t = t < tiles ? t : tiles - 1;
    while (t > 0 && before(t) > x) --t;
    while (t + 1 < tiles && before(t + 1) <= x) ++t;
    return t;
  }
};

// x / y, y > 0: from 64-bit floating point, put right by at most a few steps.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  int64_t q = int64_t(double(x) / double(y));
  while (q * y > x) --q;
  while ((q + 1) * y <= x) ++q;
  return q;
}

struct ChunkItem {
  ChunkSeq s;
  int kvh;
  int r0, rows;    // of the sequence's (token, head) rows
  int t0, t1, nt;  // steps of 64 keys: this workgroup's, and all
  int end;         // keys that the tile's last row sees
  int base;        // position of the sequence's first new token
  int slot;        // part to write, or -1: the tile is whole
};

__device__ __forceinline__ ChunkItem chunk_item(const CacheChunkArgs& a, const ChunkSeq& s, int kvh, int tile) {
  ChunkItem x;
  const int G = a.Hq / a.Hkv;
  const int64_t R = int64_t(s.len) * G, room = int64_t(a.max_pages) * a.page, r0 = int64_t(tile) * kChunkRows;
  x.s = s;
  x.kvh = kvh;
  x.r0 = int(r0);
  x.rows = int(R - r0 < kChunkRows ? R - r0 : kChunkRows);
  x.base = s.ctx - s.len;
  const int64_t e = int64_t(x.base) + uniform(int(uint32_t(x.r0 + x.rows - 1) / uint32_t(G))) + 1;
  x.end = int(e < 0 ? 0 : (e < room ? e : room));
  x.nt = int((int64_t(x.end) + 63) >> 6);
  x.t0 = 0;
  x.t1 = x.nt;
  x.slot = -1;
  return x;
}

// Eight fp32 values of a query row, its sign turned with the scale's.
template <typename T>
__device__ __forceinline__ f32x8 load_q(const T* p, bool neg) {
  typename Op<T>::frag f = Op<T>::load(p);
  if (neg) f = Op<T>::neg(f);
  return Op<T>::unpack(f);
}

template <typename T, int D>
struct ChunkShape {
  static constexpr int NP = sizeof(T) == 2 ? 1 : 3;
  static constexpr int kStage = 2 * 64 * D * 2;  // one step's K and V in bf16
  static constexpr int kJoin = (4 * kNarrowRows * (D + 4) + 2 * 4 * kNarrowRows) * 4;
  static constexpr int kQ = (D / 64) * 2 * 2 * NP * 64 * 16;  // the narrow form's parts of queries
  static constexpr int most(int x, int y) { return x > y ? x : y; }
  static constexpr size_t lds = most(most(2 * kStage, kJoin), kQ) + 128;  // and a flag, and where the division of the work stands
};

// One wavefront's share of a tile of rows, with what reads and writes it.
template <typename T, typename TO, int D>
struct ChunkWork {
  using O = Op<bf16_t>;
  using W = ChunkShape<T, D>;
  static constexpr int NP = W::NP;
  using Parts8 = Parts<bf16_t, NP, 8>;

  const CacheChunkArgs& a;
  unsigned char* smem;
  int* bad;   // set where values that are not finite have been left out
  int* over;  // set where a sum is not finite
  int lift;   // the values are taken as 2^-lift of what they are
  int tid, lane, wave, G, P, ps;
  float c;
  bool neg;

  __device__ __forceinline__ ChunkWork(const CacheChunkArgs& args, unsigned char* lds) : a(args), smem(lds) {
    bad = reinterpret_cast<int*>(lds + W::lds - 128);
    over = bad + 1;
    lift = 0;
    tid = threadIdx.x;
    lane = tid & 63;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    G = a.Hq / a.Hkv;
    P = a.page;
    ps = page_shift(P);
    // a negative scale is the positive one with the queries' signs turned; a scale of zero is the
    // least normal number (a masked score, -inf, times zero would be NaN)
    c = fmaxf(fabsf(a.scale) * kLog2e, 1.1754944e-38f);
    neg = a.scale < 0.f;
  }

  // Four channels (c0 a multiple of 4) of row rr within a part of a tile of `rows`: as the wide form holds them, its 64
  // lanes one behind another; row by row in the narrow form.
  __device__ __forceinline__ static int part_at(int rows, int rr, int c0) {
    if (rows <= kNarrowRows) return rr * D + c0;
    return (((rr >> 5) * (D / 8) + (c0 >> 3)) * 64 + (c0 >> 2 & 1) * 32 + (rr & 31)) * 4;
  }
  __device__ __forceinline__ float shrink() const { return __uint_as_float(uint32_t(127 - uniform(lift)) << 23); }
  __device__ __forceinline__ float* part(int slot) const { return a.part + int64_t(slot) * chunk_part_floats(D); }

  __device__ __forceinline__ void wide(const ChunkItem& x, const int* table) {
    using TK = Tile<bf16_t, D>;
    using TV = Tile<bf16_t, 64>;
    constexpr int NPC = D / 64, NK = D / 16, ND = D / 32;  // pieces of 1 KB of a wavefront; k steps; blocks of channels
    bf16_t* const buf = reinterpret_cast<bf16_t*>(smem);
    const int h2 = lane >> 5, l32 = lane & 31, w0 = 32 * wave;
    const bool alive = w0 < x.rows;
    // A step's pages, group g's in lanes g, g + 4, ...  They come by vector loads, ahead of what they are for: a
    // scalar load on its way makes every wait for the LDS a wait for it too.
    auto ask = [&](int t) {
      const uint32_t tok = uint32_t(t) * 64 + 16 * (lane & 3);
      return t < x.t1 && tok < uint32_t(x.end) ? table[tok >> ps] : -1;
    };
    const int asked0 = ask(x.t0), asked1 = ask(x.t0 + 1);
    int asked = ask(x.t0 + 2);
    const uint32_t r = uint32_t(x.r0 + (w0 + l32 < x.rows ? w0 + l32 : 0)), tok = r / uint32_t(G), hd = r % uint32_t(G);
    const int qp = x.base + int(tok), qpos = qp < -1 ? -1 : qp;  // (rows past the end repeat the first one)
    const int tmin = uniform(x.base + int(uint32_t(x.r0) / uint32_t(G)));  // position of the tile's first row

    bf16x8 qf[NK][NP];
    const T* q = static_cast<const T*>(a.q) + (int64_t(x.s.first) + tok) * a.q_stride + int64_t(x.kvh * G + int(hd)) * D;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      const Parts8 p(load_q(q + 16 * kk + 8 * h2, neg));
#pragma unroll
      for (int i = 0; i < NP; ++i) qf[kk][i] = part_of(p, i);
    }
    f32x16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) acc[i] = zero16();
    float ref = -INFINITY, l = 0.f;

    // Its pages, and which of its four groups of 16 tokens lie in no page (or behind the last token).
    struct Ids { int page, gone; };
    auto ids_of = [&](int asked) {
      const bool none = asked < 0 || asked >= a.pages;
      return Ids{none ? 0 : asked, int(__ballot(none)) & 15};  // (what is read for no page is not used)
    };
    struct Codes { u32x4 w[NPC]; float scale[NPC]; };
    auto fetch = [&](Codes& to, const uint8_t* cache, const float* scales, const Ids& z) {
#pragma unroll
      for (int i = 0; i < NPC; ++i) {
        const int at = (wave * NPC + i) * 1024, g = (at / (P * D)) << (ps - 4);  // the page's first 16 tokens
        const int64_t ph = int64_t(__builtin_amdgcn_readlane(z.page, g)) * a.Hkv + x.kvh;
        to.w[i] = *reinterpret_cast<const u32x4*>(cache + ph * P * D + (at & (P * D - 1)) + lane * 16);
        // (lane >> 6 is zero, which the compiler does not know: a vector load, as the pages' are, not a scalar one)
        to.scale[i] = scales[ph + (lane >> 6)];
      }
    };
    auto put_k = [&](bf16_t* K, const Codes& k) {
#pragma unroll
      for (int i = 0; i < NPC; ++i) {
        const int at = (wave * NPC + i) * 1024, key = (at + lane * 16) / D, ch = (lane * 16) % D;
        // row of the tile for a key: bits 2 and 3 change places, so that a result's registers hold runs of eight keys
        const int kw = (key & ~12) | ((key & 4) << 1) | ((key & 8) >> 1);
        *reinterpret_cast<bf16x8*>(K + TK::off(kw, ch)) = codes(k.w[i][0], k.w[i][1], k.scale[i]);
        *reinterpret_cast<bf16x8*>(K + TK::off(kw, ch + 8)) = codes(k.w[i][2], k.w[i][3], k.scale[i]);
      }
    };
    const int first_edge = (tmin + 1) >> 6;  // the first step that some row does not see all of
    const int first_look = lift == 0 ? first_edge : 0;  // (smaller values: all)
    // The values of a step that some row does not see all of, or with tokens in no page.
    auto clean_v = [&](Codes& v, int t, const Ids& z) {
      if (t < first_look && z.gone == 0) return;
#pragma unroll
      for (int i = 0; i < NPC; ++i) {
        const int at = (wave * NPC + i) * 1024, o = (at & (P * D - 1)) + lane * 16;
        const int vt = ((at / (P * D)) << ps) + (o & (P - 1));
        const int left = z.gone >> (vt >> 4) & 1 ? 0 : x.end - t * 64 - vt;
        if (left <= 0) v.scale[i] = 1.f;  // (a zero by the scale of a page that is none could be NaN)
#pragma unroll
        for (int w = 0; w < 4; ++w) {  // what lies behind the last token may be anything, NaN too
          const int nb = int(left < 0 ? 0 : (left > 16 ? 16 : left)) - 4 * w;
          v.w[i][w] &= nb >= 4 ? 0xffffffffu : (nb <= 0 ? 0u : (1u << (8 * nb)) - 1u);
        }
        // A masked probability is zero, but zero times a NaN is not: where a step is masked for some rows such
        // values leave the product, and the rows that see them are set at the end (set_bad, from this step on).
        if (t >= first_edge) {
          if (finite_codes(v.w[i], v.scale[i])) *bad = 1;
        } else if (t >= first_look) {
          finite_codes<true>(v.w[i], v.scale[i]);  // (2^-lift of it would be finite)
        }
      }
    };
    auto put_v = [&](bf16_t* V, const Codes& v) {
#pragma unroll
      for (int i = 0; i < NPC; ++i) {
        const int at = (wave * NPC + i) * 1024, o = (at & (P * D - 1)) + lane * 16;
        const int d = o >> ps, vt = ((at / (P * D)) << ps) + (o & (P - 1));
        *reinterpret_cast<bf16x8*>(V + TV::off(d, vt)) = codes(v.w[i][0], v.w[i][1], v.scale[i] * shrink());
        *reinterpret_cast<bf16x8*>(V + TV::off(d, vt + 8)) = codes(v.w[i][2], v.w[i][3], v.scale[i] * shrink());
      }
    };
    const uint32_t krow = TK::b_row8_32(lane), vrow = TV::b_row8_32(lane);
    auto k_of = [&](int t) { return buf + (t & 1) * (2 * 64 * D); };
    Ids one = ids_of(asked0), two = ids_of(asked1), three;
    Codes kc, vc;
    if (x.t0 < x.t1) {
      Codes k0, v0;
      fetch(k0, a.kc, a.ks, one);
      fetch(v0, a.vc, a.vs, one);
      fetch(kc, a.kc, a.ks, two);
      fetch(vc, a.vc, a.vs, two);
      put_k(k_of(x.t0), k0);
      clean_v(v0, x.t0, one);
      put_v(k_of(x.t0) + 64 * D, v0);
    }
    lds_barrier();
    if (!alive) {  // no rows: this wavefront only brings its share of the steps
      for (int t = x.t0; t < x.t1; ++t) {
        three = ids_of(asked);
        asked = ask(t + 3);
        put_k(k_of(t + 1), kc);
        clean_v(vc, t + 1, two);
        put_v(k_of(t + 1) + 64 * D, vc);
        fetch(kc, a.kc, a.ks, three);
        fetch(vc, a.vc, a.vs, three);
        two = three;
        lds_barrier();
      }
      return;
    }
    for (int t = x.t0; t < x.t1; ++t) {
      three = ids_of(asked);
      asked = ask(t + 3);
      const uint32_t kb = TK::at(k_of(t)) + krow, vb = TV::at(k_of(t) + 64 * D) + vrow;
      __builtin_amdgcn_s_setprio(1);
      f32x16 s[2];
      s[0] = s[1] = zero16();
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bf16x8 kf = TK::row8_32(kb, j, kk);
#pragma unroll
          for (int i = NP - 1; i >= 0; --i) s[j] = O::mma32(kf, qf[kk][i], s[j]);
        }
      if (t + 1 < x.t1) {
        clean_v(vc, t + 1, two);
        put_k(k_of(t + 1), kc);
        put_v(k_of(t + 1) + 64 * D, vc);
      }
      __builtin_amdgcn_s_setprio(0);
      bf16x8 vf[2][ND];
#pragma unroll
      for (int i = 0; i < ND; ++i) vf[0][i] = TV::row8_32(vb, i, 0);
      if (t + 2 < x.t1) {
        fetch(kc, a.kc, a.ks, three);
        fetch(vc, a.vc, a.vs, three);
      }
      if (t >= first_edge || one.gone != 0) {
        const int left = qpos - t * 64 - 8 * h2;  // tokens of this half that the row sees: up to `left`
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[j][i] = 32 * j + 16 * (i >> 3) + (i & 7) <= left && !(one.gone >> (2 * j + (i >> 3)) & 1) ? s[j][i] : -INFINITY;
      }
      float mt = s[0][0];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) mt = fmaxf(mt, s[j][i]);
      mt = c * max_halves(mt);
      if (__any(mt > ref)) {
        const float up = mt > ref ? mt + 8.f : ref;
        const float al = up == ref ? 1.f : fast_exp2(ref - up);
        l *= al;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][e] *= al;
        ref = up;
      }
      __builtin_amdgcn_s_setprio(1);
      const float from = ref == -INFINITY ? 0.f : ref;  // a row that has met no key yet
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u < 3)
#pragma unroll
          for (int i = 0; i < ND; ++i) vf[(u + 1) & 1][i] = TV::row8_32(vb, i, u + 1);
        f32x8 p8;
#pragma unroll
        for (int e = 0; e < 8; ++e) p8[e] = fast_exp2(s[u >> 1][8 * (u & 1) + e] * c - from);
        // (summed in pairs: a long row's sum would lose its terms' last bits one by one)
        l += ((p8[0] + p8[1]) + (p8[2] + p8[3])) + ((p8[4] + p8[5]) + (p8[6] + p8[7]));
        const Parts8 pf(p8);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int k = NP - 1; k >= 0; --k) acc[i] = O::mma32(vf[u & 1][i], part_of(pf, k), acc[i]);
      }
      __builtin_amdgcn_s_setprio(0);
      one = two;
      two = three;
      lds_barrier();
    }
    l = sum_halves(l) * shrink();
    ref += float(uniform(lift));
    f32x4 none = {0, 0, 0, 0};  // of finite sums
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) none[e & 3] = __builtin_fmaf(acc[i][e], 0.f, none[e & 3]);
    if ((none[0] + none[1]) + (none[2] + none[3]) != 0.f) *over = 1;
    const bool mine = w0 + l32 < x.rows;
    if (x.slot < 0) {
      // through the LDS, so that a row's channels leave side by side (every wavefront has left the last step)
      constexpr int E = 16 / int(sizeof(TO)), RS = D + E, RPI = 64 * E / D;  // rows of one store of the wavefront
      TO* const rows = reinterpret_cast<TO*>(smem) + wave * 32 * RS;
      const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4)
          store4(rows + l32 * RS + 32 * i + 8 * r4 + 4 * h2,
                 f32x4{acc[i][4 * r4] * inv, acc[i][4 * r4 + 1] * inv, acc[i][4 * r4 + 2] * inv, acc[i][4 * r4 + 3] * inv});
      if (a.lse && h2 == 0 && mine) a.lse[(int64_t(x.s.first) + tok) * a.Hq + x.kvh * G + int(hd)] = (ref + log2f(l)) * 0.6931471805599453f;
      __builtin_amdgcn_wave_barrier();
      int rr = lane / (D / E), at = int(uint32_t(x.r0 + w0 + rr) / uint32_t(G)), h = x.r0 + w0 + rr - at * G;
      const int c0 = lane % (D / E) * E, tokens = RPI / G, heads = RPI % G;
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        if (w0 + rr < x.rows)
          *reinterpret_cast<u32x4*>(static_cast<TO*>(a.o) + ((int64_t(x.s.first) + at) * a.Hq + x.kvh * G + h) * D + c0) =
              *reinterpret_cast<const u32x4*>(rows + rr * RS + c0);
        rr += RPI;
        at += tokens;
        h += heads;
        if (h >= G) {
          h -= G;
          ++at;
        }
      }
    } else {
      float* pp = part(x.slot);
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4)
          store4(pp + ((wave * (D / 8) + 4 * i + r4) * 64 + lane) * 4,
                 f32x4{acc[i][4 * r4], acc[i][4 * r4 + 1], acc[i][4 * r4 + 2], acc[i][4 * r4 + 3]});
      if (h2 == 0 && mine) {
        pp[kChunkRows * D + 2 * (w0 + l32)] = ref;
        pp[kChunkRows * D + 2 * (w0 + l32) + 1] = l;
      }
    }
  }

  // NC groups of 16 rows.
  template <int NC>
  __device__ __forceinline__ void narrow(const ChunkItem& x, const int* table) {
    constexpr int NM = D / 64, ND = D / 16;
    const int r16 = lane & 15, g4 = lane >> 4;
    // queries of 32 rows, and the parts of fp32 ones, in LDS: in registers they would push out the next step
    constexpr bool QL = NP == 3 || NC == 2;
    bf16x8(*const qs)[64] = reinterpret_cast<bf16x8(*)[64]>(smem);  // [NC][NM][2][NP]
    const int tmin = uniform(x.base + int(uint32_t(x.r0) / uint32_t(G)));

    u32x4 kr[4][NM], vr[ND];
    float ksc = 1.f, vsc = 1.f;
    // the page of this lane's tokens of a step, as the rows of K (groups by r16) and as the values (by g4)
    auto page_id = [&](uint32_t tok) {
      int p = -1;
      if (tok < uint32_t(x.end)) p = table[tok >> ps];
      return p >= 0 && p < a.pages ? p : -1;
    };
    auto k_page = [&](int t) { return page_id(t < x.t1 ? uint32_t(t) * 64 + 16 * (r16 >> 2) : uint32_t(x.end)); };
    auto v_page = [&](int t) { return page_id(t < x.t1 ? uint32_t(t) * 64 + 16 * g4 : uint32_t(x.end)); };
    auto load_k = [&](int p) {
      const int64_t ph = int64_t(p < 0 ? 0 : p) * a.Hkv + x.kvh;
      const uint8_t* kp = a.kc + (ph * P + ((16 * (r16 >> 2)) & (P - 1)) + (r16 & 3)) * D + 16 * g4;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int m = 0; m < NM; ++m)
          kr[q][m] = p >= 0 ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(kp + 4 * q * D + 64 * m)) : u32x4{0, 0, 0, 0};
      ksc = p >= 0 ? a.ks[ph] : 1.f;
    };
    auto load_v = [&](int p) {
      const int64_t ph = int64_t(p < 0 ? 0 : p) * a.Hkv + x.kvh;
      const uint8_t* vp = a.vc + (ph * D + r16) * P + ((16 * g4) & (P - 1));
#pragma unroll
      for (int d = 0; d < ND; ++d)
        vr[d] = p >= 0 ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(vp + 16 * d * P)) : u32x4{0, 0, 0, 0};
      vsc = p >= 0 ? a.vs[ph] : 1.f;
    };

    f32x4 acc[NC][ND];
    float ref[NC], l[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      ref[n] = -INFINITY;
      l[n] = 0.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[n][d] = f32x4{0, 0, 0, 0};
    }
    // (the first step is on its way before the queries are waited for)
    int t = x.t0 + wave;
    const int pk = k_page(t);
    int pv = v_page(t), pk1 = k_page(t + 4), pv1 = v_page(t + 4);
    if (t < x.t1) {
      load_k(pk);
      load_v(pv);
    }
    int qpos[NC];
    bf16x8 qf[NC][NM][2];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const bool live = 16 * n + r16 < x.rows;
      const uint32_t r = uint32_t(x.r0 + (live ? 16 * n + r16 : 0)), tok = r / uint32_t(G), hd = r % uint32_t(G);
      const int qp = x.base + int(tok);
      qpos[n] = qp < -1 ? -1 : qp;
      const T* q = static_cast<const T*>(a.q) + (int64_t(x.s.first) + tok) * a.q_stride + int64_t(x.kvh * G + int(hd)) * D;
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Parts8 p(load_q(q + 16 * (g4 + 4 * m) + 8 * e, neg));
          if constexpr (!QL) qf[n][m][e] = part_of(p, 0);
          else if (wave == 0)
#pragma unroll
            for (int i = 0; i < NP; ++i) qs[((n * NM + m) * 2 + e) * NP + i][lane] = part_of(p, i);
        }
    }
    if constexpr (QL) lds_barrier();
    for (; t < x.t1; t += 4) {
      f32x4 s[NC][4];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[n][q] = f32x4{0, 0, 0, 0};
      int ql = lane;
      if constexpr (QL) asm volatile("" : "+v"(ql));  // read again for each step
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          bf16x8 kf[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) kf[q] = codes(kr[q][m][2 * e], kr[q][m][2 * e + 1], ksc);
#pragma unroll
          for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int i = NP - 1; i >= 0; --i) {
              bf16x8 qp;
              if constexpr (!QL) qp = qf[n][m][e];
              else qp = qs[((n * NM + m) * 2 + e) * NP + i][ql];
#pragma unroll
              for (int q = 0; q < 4; ++q) s[n][q] = O::mma16(kf[q], qp, s[n][q]);
            }
        }
      const int64_t k0 = int64_t(t) * 64 + 16 * g4;  // this lane's tokens
      const bool here = pv >= 0;
      load_k(pk1);
      pk1 = k_page(t + 8);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const int64_t seen = int64_t(qpos[n]) + 1 - k0;
        const int left = here ? int(seen < 0 ? 0 : (seen > 16 ? 16 : seen)) : 0;
        float mt = -INFINITY;
        if (__any(left < 16)) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][q][i] = 4 * q + i < left ? s[n][q][i] : -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) mt = fmaxf(mt, s[n][q][i]);
        mt = c * max_groups(mt);
        if (__any(mt > ref[n])) {
          const float up = mt > ref[n] ? mt + 8.f : ref[n];
          const float al = up == ref[n] ? 1.f : fast_exp2(ref[n] - up);
          l[n] *= al;
#pragma unroll
          for (int d = 0; d < ND; ++d) acc[n][d] *= al;
          ref[n] = up;
        }
        const float from = ref[n] == -INFINITY ? 0.f : ref[n];
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[n][q][i] = fast_exp2(s[n][q][i] * c - from);
            sum += s[n][q][i];
          }
        l[n] += sum;
      }
      if (x.end - t * 64 < 64) {  // what lies behind the last token may be anything, NaN too
        const int64_t left = x.end - k0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int nb = int(left < 0 ? 0 : (left > 16 ? 16 : left)) - 4 * w;
          const uint32_t mask = nb >= 4 ? 0xffffffffu : (nb <= 0 ? 0u : (1u << (8 * nb)) - 1u);
#pragma unroll
          for (int d = 0; d < ND; ++d) vr[d][w] &= mask;
        }
      }
      if (tmin - t * 64 < 63) {  // (as in the wide form)
        bool any = false;
#pragma unroll
        for (int d = 0; d < ND; ++d) any |= finite_codes(vr[d], vsc);
        if (any) *bad = 1;
      } else if (lift != 0) {
#pragma unroll
        for (int d = 0; d < ND; ++d) finite_codes<true>(vr[d], vsc);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int d0 = 0; d0 < ND; d0 += 4) {
          bf16x8 vf[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) vf[d] = codes(vr[d0 + d][2 * u], vr[d0 + d][2 * u + 1], vsc * shrink());
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const Parts8 pf(__builtin_shufflevector(s[n][2 * u], s[n][2 * u + 1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int i = NP - 1; i >= 0; --i)
#pragma unroll
              for (int d = 0; d < 4; ++d) acc[n][d0 + d] = O::mma16(vf[d], part_of(pf, i), acc[n][d0 + d]);
          }
        }
      }
      pv = pv1;
      load_v(pv1);
      pv1 = v_page(t + 8);
    }
    float* const jo = reinterpret_cast<float*>(smem);  // [4][16 NC][D + 4]
    float* const jm = jo + 4 * 16 * NC * (D + 4);      // [4][16 NC] references, then sums
    if constexpr (QL) lds_barrier();                   // the queries have been read
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const float ls = sum_groups(l[n]) * shrink();
      if (g4 == 0) {
        jm[wave * 16 * NC + 16 * n + r16] = ref[n] + float(uniform(lift));
        jm[(4 + wave) * 16 * NC + 16 * n + r16] = ls;
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(jo + (wave * 16 * NC + 16 * n + r16) * (D + 4) + 16 * d + 4 * g4) = acc[n][d];
    }
    lds_barrier();
    for (int e = tid; e < x.rows * (D / 4); e += 256) {
      const int rr = e / (D / 4), c0 = 4 * (e % (D / 4));
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) m = fmaxf(m, jm[w * 16 * NC + rr]);
      const float from = m == -INFINITY ? 0.f : m;
      float ls = 0.f;
      f32x4 y = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = fast_exp2(jm[w * 16 * NC + rr] - from);
        ls += f * jm[(4 + w) * 16 * NC + rr];
        y += *reinterpret_cast<const f32x4*>(jo + (w * 16 * NC + rr) * (D + 4) + c0) * f;
      }
      if (((y[0] * 0.f + y[1] * 0.f) + (y[2] * 0.f + y[3] * 0.f)) != 0.f) *over = 1;
      if (x.slot < 0) {
        const uint32_t r = uint32_t(x.r0 + rr);
        const int64_t row = (int64_t(x.s.first) + r / uint32_t(G)) * a.Hq + x.kvh * G + int(r % uint32_t(G));
        store4(static_cast<TO*>(a.o) + row * D + c0, y * (ls == 0.f ? 0.f : 1.0f / ls));
        if (a.lse && c0 == 0) a.lse[row] = (m + log2f(ls)) * 0.6931471805599453f;
      } else {
        float* pp = part(x.slot);
        store4(pp + part_at(x.rows, rr, c0), y);
        if (c0 == 0) {
          pp[kChunkRows * D + 2 * rr] = m;
          pp[kChunkRows * D + 2 * rr + 1] = ls;
        }
      }
    }
  }

  // Writes the values that are not finite into the outputs (parts) of the rows that see them: no finite
  // sum, nor a factor, changes them.
  __device__ __forceinline__ void set_bad(const ChunkItem& x, const int* table) {
    const int tmin = uniform(x.base + int(uint32_t(x.r0) / uint32_t(G)));
    int64_t k0 = tmin < 0 ? 0 : (tmin + 1) & ~63;
    k0 = k0 > int64_t(x.t0) * 64 ? k0 : int64_t(x.t0) * 64;
    const int64_t k1 = x.end < int64_t(x.t1) * 64 ? x.end : int64_t(x.t1) * 64;
    for (int e = tid; e < x.rows * D; e += 256) {
      const int rr = e / D, d = e % D;
      const uint32_t r = uint32_t(x.r0 + rr), tok = r / uint32_t(G);
      float y = 0.f;
#pragma unroll 1
      for (int64_t key = k0; key < k1 && key <= int64_t(x.base) + tok; ++key) {
        const int p = table[key >> ps];
        if (p < 0 || p >= a.pages) continue;
        const int64_t ph = int64_t(p) * a.Hkv + x.kvh;
        const float v = float(codes(a.vc[(ph * D + d) * P + (key & (P - 1))], 0, a.vs[ph])[0]);
        if (!(fabsf(v) < INFINITY)) y += v;
      }
      if (y == 0.f) continue;
      if (x.slot < 0)
        io<TO>::store(static_cast<TO*>(a.o), ((int64_t(x.s.first) + tok) * a.Hq + x.kvh * G + int(r % uint32_t(G))) * D + d, y);
      else
        part(x.slot)[part_at(x.rows, rr, d & ~3) + (d & 3)] = y;
    }
  }

  // Whether some page's values can add up to more than fp32 holds: 448 2^88 times 2^31 tokens cannot.
  __device__ __forceinline__ bool large_values(const ChunkItem& x, const int* table) {
    const int64_t k1 = x.end < int64_t(x.t1) * 64 ? x.end : int64_t(x.t1) * 64;
    bool any = false;
#pragma unroll 1
    for (int64_t key = int64_t(x.t0) * 64 + 16 * tid; key < k1; key += 16 * 256) {
      const int p = table[key >> ps];
      if (p >= 0 && p < a.pages) any |= a.vs[int64_t(p) * a.Hkv + x.kvh] > 0x1p88f;
    }
    return any;
  }

  // The item's outputs or part; false if it has to be done again, with `lift` set.
  __device__ __forceinline__ bool run(const ChunkItem& x, int seq) {
    const int* table = a.table + int64_t(seq) * a.max_pages;
    // what follows from the lane's number is formed again for each item: held over the loop, all three forms'
    // would be in registers at once
    asm volatile("" : "+v"(tid), "+v"(lane));
    lds_barrier();  // the item before is out of the LDS
    if (tid == 0) *bad = *over = 0;
    lds_barrier();
    if (x.rows > kNarrowRows) wide(x, table);
    else if (x.rows > 16) narrow<2>(x, table);
    else narrow<1>(x, table);
    lds_barrier();
    if (lift == 0 && uniform(*over)) {
      if (large_values(x, table)) *over = 2;
      lds_barrier();
      if (uniform(*over) == 2) {
        lift = kShrinkBits;
        return false;
      }
    }
    lift = 0;
    if (*bad) {
      __threadfence();  // behind the stores of the sums
      __syncthreads();
      set_bad(x, table);
    }
    return true;
  }
};

// Where a workgroup stands: its share still to do, the tile (-1: to be found, `rest` into the sequence's line).
struct ChunkState {
  int64_t todo, rest;
  int seq, kvh, tile, w;
  ChunkSeq s;
};

// What a part is, for the kernel that joins them.
struct ChunkPart {
  int kind;  // 0: none; 1: the tile goes on in the next workgroup; 2: its end
  int first, kvh, r0, rows, pad[3];
};

// (Three workgroups to a compute unit for bf16 at d = 64: 83.1 us for a mixed batch, 84.3 where the registers were left to
// themselves.)
template <typename T, typename TO, int D>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? (D == 64 ? 3 : 2) : 1) void cache_chunk_kernel(const CacheChunkArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  if (a.zero_tail) {
    const int64_t used = a.N > 0 ? rows_in_use(a.cu, a.N, a.n) : 0;
    for (int64_t row = used + blockIdx.x; row < a.n; row += gridDim.x) {
      for (int e = tid; e < a.Hq * (D / 4); e += 256)
        store4(static_cast<TO*>(a.o) + row * a.Hq * D + 4 * int64_t(e), f32x4{0, 0, 0, 0});
      if (a.lse)
        for (int e = tid; e < a.Hq; e += 256) a.lse[row * a.Hq + e] = 0.f;
    }
  }
  if (a.N == 0) return;
  ChunkWork<T, TO, D> work(a, smem);
  const int G = a.Hq / a.Hkv;

  const bool shared = a.groups > 0;
  ChunkState z{};
  z.todo = 1;
  ChunkPart* const parts = reinterpret_cast<ChunkPart*>(a.part + int64_t(a.groups) * 2 * chunk_part_floats(D));
  if (!shared) {
    // Sequence i's tiles sit at slots cu[i] G / 128 + i onwards, which leaves each at least as many as it has.
    const int slots = int(gridDim.x / a.Hkv), slot = slots - 1 - int(blockIdx.x / a.Hkv);
    // (the last sequence first, of each sequence the longest tiles first: a long sequence that comes early ends late)
    z.kvh = int(blockIdx.x % a.Hkv);
    int lo = 0, up = a.N;
    auto start = [&](int64_t i) {
      const int64_t c = a.cu[i];
      return (c < 0 ? 0 : c) * G / kChunkRows + i;
    };
    while (up - lo > 1) {
      const int step = (up - lo + 63) / 64;
      const int64_t mid = lo + int64_t(step) * (lane + 1);
      lo += step * __popcll(__ballot(mid < up && start(mid) <= slot));
      up = lo + step < up ? lo + step : up;
    }
    const int64_t tile = slot - start(lo);
    z.s = chunk_seq(a, lo);
    if (tile < 0 || tile >= ChunkCost(a, z.s).tiles) return;
    z.seq = lo;
    z.tile = int(tile);
  } else {
    // Every workgroup takes an equal piece of the line of all tiles' costs, key heads outermost.
    int64_t* const sums = reinterpret_cast<int64_t*>(smem);  // [256] costs of the threads' sequences before each, [4]
    const int per = (a.N + 255) / 256;
    int64_t mine = 0;
    for (int i = tid * per; i < (tid + 1) * per && i < a.N; ++i) mine += ChunkCost(a, chunk_seq(a, i)).all();
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t y = __shfl_up((long long)upto, d);
      upto += lane >= d ? y : 0;
    }
    if (lane == 63) sums[256 + (tid >> 6)] = upto;
    __syncthreads();
    int64_t head = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < (tid >> 6)) upto += sums[256 + i];
      head += sums[256 + i];
    }
    head = uniform(head);
    sums[tid] = upto - mine;
    __syncthreads();
    const int64_t all = head * a.Hkv, most = all / (kLeastCost * G);
    const int groups = int(most < 1 ? 1 : (most < a.groups ? most : a.groups));
    const int w = xcd_order(blockIdx.x, a.groups);
    if (tid == 0) parts[2 * w].kind = parts[2 * w + 1].kind = 0;
    if (w >= groups || all == 0) return;
    const int64_t each = quotient(all, groups), more = all - each * groups;
    const int64_t x = uniform(each * w + (w < more ? w : more));
    z.todo = each + (w < more ? 1 : 0);
    z.kvh = int(quotient(x, head));
    const int64_t rest = x - z.kvh * head;  // to go within this key head's line
    int lo = 0, up = 256;
    while (up - lo > 1) {
      const int mid = (lo + up) / 2;
      if (sums[mid] <= rest) lo = mid;
      else up = mid;
    }
    z.rest = rest - sums[lo];
    z.seq = lo * per;
    z.tile = -1;  // to be found
    z.s = chunk_seq(a, z.seq);
    z.w = w;
  }
  // What comes next, and what the item began with, are kept in the LDS while it is worked on: in scalar registers
  // they would push others out.
  ChunkState* const state = reinterpret_cast<ChunkState*>(smem + ChunkShape<T, D>::lds - 112);
  static_assert(2 * sizeof(ChunkState) <= 112);
  if (tid == 0) state[0] = z;
  int now = 0;  // the item's own
  for (;;) {
    int64_t from = 0, to = 1, full = 1, rest = uniform(z.rest);
    ChunkSeq s = uniform(z.s);
    int tile = uniform(z.tile), seq = uniform(z.seq), kvh = uniform(z.kvh);
    const int64_t todo = uniform(z.todo);
    const int w = uniform(z.w);
    if (shared) {
      ChunkCost cost(a, s);
      while (tile >= cost.tiles || (tile < 0 && rest >= cost.all())) {  // behind this sequence's tiles
        rest = tile < 0 ? rest - cost.all() : 0;
        tile = rest > 0 ? -1 : 0;
        if (++seq == a.N) {
          seq = 0;
          ++kvh;
        }
        s = uniform(chunk_seq(a, seq));
        cost = ChunkCost(a, s);
      }
      if (tile < 0) {
        tile = int(cost.at(rest));
        from = rest - cost.before(tile);
      }
      full = cost.of(tile);
      to = from + todo < full ? from + todo : full;
    }
    ChunkItem it = chunk_item(a, s, kvh, tile);
    if (shared && (from > 0 || to < full)) {
      // (the same step from both sides of a cut: both form it from the same numbers)
      it.t0 = from > 0 ? uniform(int(double(from) * double(it.nt) / double(full))) : 0;
      if (to < full) it.t1 = uniform(int(double(to) * double(it.nt) / double(full)));
      it.slot = 2 * w + (from > 0 ? 0 : 1);
      if (tid == 0) parts[it.slot] = ChunkPart{to < full ? 1 : 2, s.first, kvh, it.r0, it.rows, {0, 0, 0}};
    }
    lds_barrier();  // the state has been read
    if (tid == 0) state[now ^ 1] = ChunkState{todo - (to - from), 0, seq, kvh, tile + 1, w, s};
    now ^= work.run(it, seq);
    lds_barrier();
    z = state[now];
    if (uniform(z.todo) <= 0) return;
  }
}

// Joins the parts of the tile that begins in workgroup blockIdx.x and ends in a later one: a sixteenth of its
// rows.  D / 4 threads to a row.  Most tiles have two to four parts, which are read all at once (a walk of their number
// first: one token over 131072 106 us instead of 64); of more, several groups of threads share a row's.  Bound by the
// parts' bytes where tiles are wide: 58 MB in 18 us, launch and all; 12 MB of narrow ones in 6.7.
// Each part's factor is 2^-10 of its own (at most 512 parts): sums that are finite add up to a finite one.
constexpr int kJoinBlocks = 16, kJoinFew = 4;
constexpr float kJoinFactor = 1.f / 1024;
static_assert(kJoinBlocks * 8 >= kChunkRows, "every row has a group of threads");
template <typename TO, int D>
__global__ __launch_bounds__(256) void cache_chunk_join_kernel(const CacheChunkArgs a) {
  constexpr int L = D / 4, NG = 256 / L;
  __shared__ f32x4 sy[NG][L];
  __shared__ float sl[NG];
  __shared__ int end;
  const ChunkPart* const parts = reinterpret_cast<const ChunkPart*>(a.part + int64_t(a.groups) * 2 * chunk_part_floats(D));
  const int w = blockIdx.x, tid = threadIdx.x, G = a.Hq / a.Hkv, g = tid / L, e = tid % L;
  const ChunkPart p = parts[2 * w + 1];
  int few[kJoinFew];
#pragma unroll
  for (int i = 1; i < kJoinFew; ++i) few[i] = w + i < a.groups ? parts[2 * (w + i)].kind : 0;
  if (p.kind != 1) return;  // (the rest of p says nothing then)
  int lg = 0;               // rows of a block: 1 << lg
#pragma unroll
  for (int i = 0; i < 3; ++i) lg += (kJoinBlocks << i) < p.rows;
  const int per = 1 << lg, row0 = int(blockIdx.y) << lg, r = row0 + (g & (per - 1));
  if (row0 >= p.rows) return;
  const bool live = r < p.rows;
  const int at = ChunkWork<TO, TO, D>::part_at(p.rows, r, 4 * e);
  auto part = [&](int i) { return a.part + int64_t(i == 0 ? 2 * w + 1 : 2 * (w + i)) * chunk_part_floats(D); };
  auto write = [&](f32x4 y, float l, float m) {
    const uint32_t rr = uint32_t(p.r0 + r);
    const int64_t row = (int64_t(p.first) + rr / uint32_t(G)) * a.Hq + p.kvh * G + int(rr % uint32_t(G));
    store4(static_cast<TO*>(a.o) + row * D + 4 * e, y * (l == 0.f ? 0.f : 1.0f / l));
    if (a.lse && e == 0) a.lse[row] = (m + log2f(l * (1.f / kJoinFactor))) * 0.6931471805599453f;
  };
  int n = 0;  // parts, where they are few
#pragma unroll
  for (int i = kJoinFew - 1; i > 0; --i) n = few[i] == 2 ? i + 1 : n;
  if (n > 0) {
    if (!live || g >= per) return;
    f32x4 y[kJoinFew];
    f32x2 ml[kJoinFew];
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i) {
      const float* pp = part(i < n ? i : 0);
      y[i] = f32x4{0, 0, 0, 0};
      if (i < n) y[i] = *reinterpret_cast<const f32x4*>(pp + at);
      ml[i] = *reinterpret_cast<const f32x2*>(pp + kChunkRows * D + 2 * r);
    }
    float m = ml[0][0];
#pragma unroll
    for (int i = 1; i < kJoinFew; ++i) m = i < n ? fmaxf(m, ml[i][0]) : m;
    const float from = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i)
      if (i < n) {
        const float f = fast_exp2(ml[i][0] - from) * kJoinFactor;
        l += f * ml[i][1];
        sum += y[i] * f;
      }
    write(sum, l, m);
    return;
  }
  if (tid == 0) end = a.groups - 1;
  __syncthreads();
  for (int i = w + 1; i < a.groups; i += 256) {  // its last part: the first one that does not go on
    if (i + tid < a.groups && parts[2 * (i + tid)].kind != 1) atomicMin(&end, i + tid);
    __syncthreads();
    if (end < i + 256) break;
  }
  n = end - w + 1;
  const int share = NG >> lg;  // groups to a row
  float m = -INFINITY;
  if (live)
    for (int i = e; i < n; i += L) m = fmaxf(m, part(i)[kChunkRows * D + 2 * r]);
#pragma unroll
  for (int d = 1; d < L; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float from = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  f32x4 y = {0, 0, 0, 0};
  if (live)
#pragma unroll 4
    for (int i = g >> lg; i < n; i += share) {
      const float* pp = part(i);
      const float f = fast_exp2(pp[kChunkRows * D + 2 * r] - from) * kJoinFactor;
      l += f * pp[kChunkRows * D + 2 * r + 1];
      y += *reinterpret_cast<const f32x4*>(pp + at) * f;
    }
  sy[g][e] = y;
  if (e == 0) sl[g] = l;
  __syncthreads();
  if (g >= per || !live) return;
  for (int i = g + per; i < NG; i += per) {
    y += sy[i][e];
    l += sl[i];
  }
  write(y, l, m);
}

template <typename T, typename TO, int D>
hipError_t launch_chunk(const CacheChunkArgs& a, hipStream_t st) {
  auto kern = cache_chunk_kernel<T, TO, D>;
  constexpr size_t lds = ChunkShape<T, D>::lds;
  static_assert(lds <= 80 * 1024, "two workgroups of a compute unit");
  static std::atomic<uint64_t> done{0};
  if constexpr (lds > 65536) {
    const hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kern), int(lds), done);
    if (e != hipSuccess) return e;
  }
  const int64_t grid = a.groups > 0 ? a.groups : cache_chunk_slots(a.n, a.N, a.Hq, a.Hkv) * a.Hkv;
  kern<<<dim3(uint32_t(grid < 1 ? 1 : grid)), 256, lds, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.groups == 0) return e;
  cache_chunk_join_kernel<TO, D><<<dim3(uint32_t(a.groups), kJoinBlocks), 256, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_chunk_any(const CacheChunkArgs& a, hipStream_t st) {
  if (a.d == 64) return a.out_bf16 ? launch_chunk<T, bf16_t, 64>(a, st) : launch_chunk<T, float, 64>(a, st);
  return a.out_bf16 ? launch_chunk<T, bf16_t, 128>(a, st) : launch_chunk<T, float, 128>(a, st);
}

}  // namespace kda
