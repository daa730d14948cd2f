// kda_linear_walk.hpp -- linear attention with a decay per head, chunked: the kernel that walks a
// sequence's chunks, forwards for the outputs and for dq, backwards for dk and dv.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// per (b, h), g_t <= 0 a scalar.  In a chunk of C tokens with entry state S and in-chunk sums
// G_t = g_1 + .. + g_t,
//   o_t   = scale (e^{G_t} S^T q_t + sum_{s <= t} e^{G_t - G_s} (q_t . k_s) v_s)
//   S_out = e^{G_C} S + sum_s e^{G_C - G_s} k_s v_s^T.
// Every exponent is a difference of sums over later tokens, so at most 0: nothing overflows,
// whatever the decays.  The sums are formed in 64 bits and kept as two fp32 parts, so a strong
// decay earlier in the chunk does not cost the later differences their low bits.
//
// The gradients are the same computation with the tensors in other roles.  With R = dL/dS,
//   dq_t = scale sum_{s <= t} e^{G_t - G_s} (do_t . v_s) k_s + ..   forwards,  (q, k, v) <- (do, v, k)
//   dk_s = scale sum_{t >= s} e^{G_t - G_s} (v_s . do_t) q_t + ..   backwards, (q, k, v) <- (v, do, q)
//   dv_s = scale sum_{t >= s} e^{G_t - G_s} (k_s . q_t) do_t + ..   backwards, (q, k, v) <- (k, q, do)
// where the backward walk (REV) holds R_in = e^{G_C} R + scale sum_t e^{G_t} q_t do_t^T (or its
// transpose) and its outputs take e^{G_C - G_s} of it.  A log-decay scales all that crosses it, so
//   dg_t = <R_c, S_c> + sum_{t <= u, u before c} (q_u . dq_u - k_u . dk_u)
// for any boundary c at or behind t.  The walks for dq and dk (DOT) leave those dot products, of
// the unrounded gradients, and every kBlockChunks chunks the one keeps S, the other multiplies its
// R with it: the sums above then never run over more than one such block, and cancel no more than it holds.
//
// One workgroup per (b, h, slice of up to 64 value columns, segment).  Wavefronts 0 .. NSW - 1 each
// own 16 value columns and hold that dk x 16 block of the state in their accumulators; with
// outputs, the others (one per 16 tokens of a chunk) form the decayed scores P of the chunk while
// the former take S^T q and the update, and copy later chunks into LDS, three in rotation: a copy has
// two steps to land.  P V and the outputs follow behind a barrier.  All products are
// 16x16x32 with fp32 accumulation: (S^T q) takes the state straight from the accumulators (their
// layout is an operand's), the values' transposing reads serve both P V and the update.
//
// With bf16 elements P, and the copy of S that the outputs read, are rounded to bf16, 2^-8 of each
// term, half a unit of the last place that the outputs have anyway where they are bf16 (fp32 outputs of
// bf16 elements carry it too).  The state takes its rows
// e^{G_C - G_s} v_s as three bf16 parts (24 bits), so it is fp32-accurate however long the
// sequence; with DOT, P and S too.
//
// Measured (bf16, B = 4, T = 32768, H = 32, 128 x 128): 1145 us for 4.33 GB, 3.8 TB/s (857 us at a
// copy's rate, 720 at the best of the library's kernels; the memory accesses alone take 933 us in this
// shape, all but them 870).  Matrix pipe 27 %, vector issue 39 % of the cycles, 4.74 GB moved.  Left out
// one at a time, the exact parts save 135 us, the scores 115, the stores 118, the copies 207: the
// sum of issue and bytes in one workgroup per compute unit bounds it, the LDS being full with three
// chunks in rotation.  The walk without outputs (segments' end states) takes 142 to 172 us for 0.54 GB.
//
// Few, long sequences are cut into segments (the ABI layer's rule).  The decay being a scalar, a
// segment's transition is one number: a first walk leaves every segment's end state from zero, a
// scan joins them, a second walk from the true entry states writes the outputs.
#pragma once

#include "kda_mix_launch.hpp"
#include "kda_mma.hpp"

namespace kda {

namespace {

// A decay below this is zero in fp32 whatever follows; -inf (a reset) would make differences NaN.
constexpr float kLeastLog = -1.0e4f;

// OUT: 0 the state only, 1 outputs, 2 outputs and their dot products, unrounded
template <typename T, int DK, int DV, int OUT>
struct WalkShape {
  static constexpr int C = linear_chunk(sizeof(T) == 2);
  static constexpr int DKP = DK < 32 ? 32 : DK;    // key channels in LDS
  static constexpr int DVS = DV < 64 ? DV : 64;    // value columns of a workgroup
  static constexpr int VC = DVS < 32 ? 32 : DVS;   // and in LDS
  static constexpr int NSL = DV / DVS, NSW = DVS / 16, TT = C / 16, U = C / 32;
  static constexpr int NPW = OUT ? TT : 1;         // scoring and copying wavefronts
  static constexpr int NT = 64 * (NSW + NPW);
  static_assert(NT <= linear_threads(sizeof(T) == 2, DV) && NSL == linear_slices(DV), "what the ABI layer checks launches by");
  static constexpr int NKK = DKP / 32, NKT = DK / 16;
  static constexpr int kExact = sizeof(T) == 2 ? 3 : 1;  // parts of an fp32-accurate operand
  static constexpr int kOut = OUT == 2 ? kExact : 1;     // parts of P and S in the outputs
  static constexpr int kK = C * DKP * int(sizeof(T)), kV = C * VC * int(sizeof(T)), kP1 = C * C * int(sizeof(T)), kP = kP1 * kOut;
  static constexpr int kG = (4 * C + 4) * 4;  // G hi, G lo, the outputs' and the update's weights, e^{G_C}
  // chunks in rotation: one in use, the others on their way (two, or three where only k and v are)
  static constexpr int NS = OUT ? 3 : 4;
  static constexpr int oQ = NS * kK, oV = oQ + (OUT ? NS * kK : 0), oP = oV + NS * kV, oG = oP + (OUT ? kP : 0),
                       oR = oG + 2 * kG;  // raw log-decays of NS + 1 chunks
  static constexpr size_t lds = size_t(oR) + (NS + 1) * 64 * 4;
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  // copies that each wavefront issues for a chunk
  static constexpr int kCopies = (C / (64 / Tile<T, DKP>::CH) + NPW - 1) / NPW * (OUT ? 2 : 1) +
                                 (C / (64 / Tile<T, VC>::CH) + NPW - 1) / NPW + 1;
  static_assert(C % (64 / Tile<T, DKP>::CH * NPW) == 0 && C % (64 / Tile<T, VC>::CH * NPW) == 0, "the same for each");
};

template <typename T, typename TO, int DK, int DV, int OUT, bool REV>
__global__ __launch_bounds__((WalkShape<T, DK, DV, OUT>::NT)) void linear_walk_kernel(const LinearArgs a) {
  using W = WalkShape<T, DK, DV, OUT>;
  using O = Op<T>;
  using F = typename O::frag;
  using TK = Tile<T, W::DKP>;
  using TV = Tile<T, W::VC>;
  using TP = Tile<T, W::C>;
  constexpr int C = W::C, NSW = W::NSW, TT = W::TT, U = W::U, NKK = W::NKK, NKT = W::NKT;
  constexpr int kExact = W::kExact, kOut = W::kOut;
  extern __shared__ __align__(1024) unsigned char smem[];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15,
            g4 = lane >> 4;
  int id = xcd_order(blockIdx.x, gridDim.x);
  const int slice = id % W::NSL;
  id /= W::NSL;
  const int seg = id % a.nseg;
  const int64_t bh = id / a.nseg;
  const int64_t b = bh / a.H, head = bh % a.H;
  const int nch = (a.T + C - 1) / C;
  const int n0 = seg * a.seg_chunks, n1 = n0 + a.seg_chunks < nch ? n0 + a.seg_chunks : nch;
  const int64_t tok = b * a.T;  // the sequence's first row
  auto chunk_of = [&](int n) { return REV ? nch - 1 - n : n; };
  auto Ks = [&](int n) { return reinterpret_cast<T*>(smem + (n % W::NS) * W::kK); };
  auto Qs = [&](int n) { return reinterpret_cast<T*>(smem + W::oQ + (n % W::NS) * W::kK); };
  auto Vs = [&](int n) { return reinterpret_cast<T*>(smem + W::oV + (n % W::NS) * W::kV); };
  T* const P = reinterpret_cast<T*>(smem + W::oP);  // [parts][C][C]
  auto gates = [&](int n) { return reinterpret_cast<float*>(smem + W::oG + (n & 1) * W::kG); };
  auto raw = [&](int n) { return reinterpret_cast<float*>(smem + W::oR) + (n % (W::NS + 1)) * 64; };

  // key channels 16 .. 31 of a 16-channel head are zero in LDS; the copies leave them alone
  if constexpr (DK < 32) {
    for (int i = tid * 4; i < (OUT ? 2 : 1) * W::NS * W::kK; i += W::NT * 4) *reinterpret_cast<uint32_t*>(smem + i) = 0u;
    __syncthreads();
  }

  if (wave >= NSW) {
    // ---- scores, gates and copies ----
    const int p = wave - NSW;
    const int64_t kst = int64_t(a.H) * DK, vst = int64_t(a.H) * DV;
    const T* kp = static_cast<const T*>(a.k) + (tok * a.H + head) * DK;
    const T* qp = OUT ? static_cast<const T*>(a.q) + (tok * a.H + head) * DK : nullptr;
    const T* vp = static_cast<const T*>(a.v) + (tok * a.H + head) * DV + slice * W::DVS;
    // A lane's byte offsets within a chunk's rows, per copy: the same for every chunk but a partial
    // one, whose rows at or past the sequence's end repeat its last row (their weights are zero).
    // The lane's chunk of 16 bytes is the one that belongs at its place in the tile.
    auto rows_of = [&](auto tile_tag, int i, int64_t stride, int last) -> uint32_t {
      using L = decltype(tile_tag);
      constexpr int PER = 64 / L::CH;
      const int r = (i * W::NPW + p) * PER + lane / L::CH, ch = (lane % L::CH) ^ L::swz(r);
      return uint32_t((r < last ? r : last) * stride * int64_t(sizeof(T))) + ch * 16;
    };
    constexpr int kPerK = C / (64 / TK::CH * W::NPW), kPerV = C / (64 / TV::CH * W::NPW);
    uint32_t offk[kPerK], offv[kPerV];
#pragma unroll
    for (int i = 0; i < kPerK; ++i) offk[i] = rows_of(TK{}, i, kst, C - 1);
#pragma unroll
    for (int i = 0; i < kPerV; ++i) offv[i] = rows_of(TV{}, i, vst, C - 1);
    const float* gp = a.g_head ? a.g + head : a.g + tok * a.H + head;
    const int64_t gst = a.g_head ? 0 : a.H;
    auto fetch_gate = [&](int n) {
      n = n < n1 ? n : n1 - 1;
      const int64_t t0 = int64_t(chunk_of(n)) * C;
      const int64_t t = t0 + lane < a.T ? lane : a.T - 1 - t0;
      lds_copy4(gp + t0 * gst, uint32_t(t * gst * 4), lds_offset(raw(n)));
    };
    // chunk n's rows and the next chunk's log-decays: W::kCopies copies of every wavefront, and nothing
    // else here reads memory, so that a count of copies is what to wait for
    auto fetch = [&](int n) {
      const int64_t t0 = int64_t(chunk_of(n)) * C;
      const T *kc = kp + t0 * kst, *qc = OUT ? qp + t0 * kst : nullptr, *vc = vp + t0 * vst;
      const uint32_t ks = lds_offset(Ks(n)) + p * 1024, qs = lds_offset(Qs(n)) + p * 1024, vs = lds_offset(Vs(n)) + p * 1024;
      // in a tile wider than the head, the lanes of the columns that do not exist copy nothing
      auto copy = [&](auto tile_tag, const T* from, uint32_t off, uint32_t to, int i, int cols) {
        using L = decltype(tile_tag);
        bool on = true;
        if (L::CH * L::EPC != cols) {
          const int r = (i * W::NPW + p) * (64 / L::CH) + lane / L::CH;
          on = ((lane % L::CH) ^ L::swz(r)) * L::EPC < cols;
        }
        if (on) lds_copy16(from, off, to + i * W::NPW * 1024);
      };
      if (a.T - t0 >= C) {
#pragma unroll
        for (int i = 0; i < kPerK; ++i) copy(TK{}, kc, offk[i], ks, i, DK);
        if constexpr (OUT > 0)
#pragma unroll
          for (int i = 0; i < kPerK; ++i) copy(TK{}, qc, offk[i], qs, i, DK);
#pragma unroll
        for (int i = 0; i < kPerV; ++i) copy(TV{}, vc, offv[i], vs, i, W::DVS);
      } else {
        const int last = int(a.T - t0) - 1;
#pragma unroll
        for (int i = 0; i < kPerK; ++i) {
          const uint32_t off = rows_of(TK{}, i, kst, last);
          copy(TK{}, kc, off, ks, i, DK);
          if constexpr (OUT > 0) copy(TK{}, qc, off, qs, i, DK);
        }
#pragma unroll
        for (int i = 0; i < kPerV; ++i) copy(TV{}, vc, rows_of(TV{}, i, vst, last), vs, i, W::DVS);
      }
      fetch_gate(n + 1);
    };
    // the gate wavefront has the fewest scores
    const bool gate = p == (REV ? W::NPW - 1 : 0);
    double total = 0.0;  // log2 of the walk's decay
    auto gate_sums = [&](int n) {
      const bool live = lane < C && int64_t(chunk_of(n)) * C + lane < a.T;
      float g = live ? raw(n)[lane] : 0.f;
      g = g < kLeastLog ? kLeastLog : g;
      const double G = wave_prefix(double(g) * 1.4426950408889634), Gc = lane_value(G, C - 1);
      total += Gc;
      if (lane < C) {
        float* ga = gates(n);
        const float hi = float(G), to_end = fast_exp2(float(Gc - G)), from_start = fast_exp2(float(G));
        ga[lane] = hi;
        ga[C + lane] = float(G - double(hi));
        ga[2 * C + lane] = REV ? to_end : from_start;
        ga[3 * C + lane] = live ? (REV ? a.scale * from_start : to_end) : 0.f;
        if (lane == C - 1) ga[4 * C] = from_start;
      }
    };
    const uint32_t brow = TK::b_row8_16(lane);
    // scores of 16 tokens (columns t) with the source tokens s that they take from, transposed: rows s
    auto scores = [&](int n) {
      if constexpr (OUT > 0) {
        const uint32_t kb = TK::at(Ks(n)) + brow, qb = TK::at(Qs(n)) + brow;
        const float* ga = gates(n);
        F qf[NKK];
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk) qf[kk] = TK::row8_16(qb + 16 * p * TK::ROWB, 0, kk);
        const int t = 16 * p + l16;
        const int64_t live = a.T - int64_t(chunk_of(n)) * C;
        const float thi = ga[t], tlo = ga[C + t];
#pragma unroll
        for (int si = 0; si < TT; ++si) {
          const bool on = REV ? si >= p : si <= p;
          if (!on && si / 2 != p / 2) continue;  // never read
          f32x4 c = {0, 0, 0, 0}, x = c;
          const int s = 16 * si + 4 * g4;
          if (on) {
#pragma unroll
            for (int kk = 0; kk < NKK; ++kk) c = O::mma16(TK::row8_16(kb, si, kk), qf[kk], c);
            const f32x4 shi = *reinterpret_cast<const f32x4*>(ga + s), slo = *reinterpret_cast<const f32x4*>(ga + C + s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float d = (thi - shi[j]) + (tlo - slo[j]);
              // backwards the sources lie behind t, and may lie behind the sequence
              if constexpr (REV) x[j] = s + j >= t && s + j < live ? a.scale * fast_exp2(-d) * c[j] : 0.f;
              else x[j] = s + j <= t ? fast_exp2(d) * c[j] : 0.f;
            }
          }
          if constexpr (kOut == 1) {
            TP::put4(P, t, s, x);
          } else {
            const Parts<T, kOut, 4> xp(x);
#pragma unroll
            for (int i = 0; i < kOut; ++i) *reinterpret_cast<u32x2v*>(P + i * C * C + TP::off(t, s)) = xp.p[i];
          }
        }
      }
    };
    if (n0 < n1) {
      fetch_gate(n0);
#pragma unroll
      for (int i = 0; i < W::NS - 1; ++i)
        if (n0 + i < n1) fetch(n0 + i);
      copies_landed();
      if (gate) gate_sums(n0);
      lds_barrier();
      for (int n = n0; n < n1; ++n) {
        const bool more = n + W::NS - 1 < n1;
        if (more) fetch(n + W::NS - 1);
        scores(n);
        if (gate && n + 1 < n1) gate_sums(n + 1);
        if constexpr (OUT > 0) lds_barrier();
        if (more) copies_landed<(W::NS - 2) * W::kCopies>();  // the next chunk is there
        else copies_landed();
        lds_barrier();
      }
    }
    if (a.seg_decay && gate && lane == 0 && slice == 0) a.seg_decay[bh * a.nseg + seg] = float(exp2(total));
    return;
  }

  // ---- the state ----
  const int col = slice * W::DVS + 16 * wave + l16;  // this lane's value column
  f32x4 S[NKT];
  {
    const float* Sin = a.S_in ? a.S_in + (a.S_in_seg ? bh * a.nseg + seg : bh) * DK * DV : nullptr;
    if (!a.S_in_seg && seg > 0) Sin = nullptr;  // a first walk's later segments start from zero
    const bool tr = a.state_tr && !a.S_in_seg;
#pragma unroll
    for (int i = 0; i < NKT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * g4 + r;
        S[i][r] = Sin ? Sin[tr ? col * DK + row : row * DV + col] : 0.f;
      }
  }
  // states kept for dg, in the accumulators' order
  const int nblk = (nch + kBlockChunks - 1) / kBlockChunks;
  const int part = slice * NSW + wave;
  auto kept = [&](int blk) {
    return reinterpret_cast<f32x4*>(a.ckpt) + (((bh * (nblk + 1) + blk) * W::NSL + slice) * NSW + wave) * NKT * 64 + lane;
  };
  auto keep = [&](int blk) {
    f32x4* c = kept(blk);
#pragma unroll
    for (int i = 0; i < NKT; ++i) c[i * 64] = S[i];
  };
  auto meet = [&](int blk) {  // <R, S> at the end of block blk - 1
    const f32x4* c = kept(blk);
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < NKT; ++i) {
      const f32x4 s = c[i * 64];
#pragma unroll
      for (int r = 0; r < 4; ++r) x += s[r] * S[i][r];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    if (lane == 0) a.bsum[(bh * nblk + blk - 1) * (W::NSL * NSW) + part] = x;
  };
  if constexpr (OUT == 2 && REV)
    if (seg == 0 && nch > 0) meet(nblk);

  if (n0 < n1) {
    lds_barrier();
    const uint32_t qrow = TK::b_row44_16(lane), kcol = TK::b_col8_16(lane), vcol = TV::b_col8_16(lane),
                   prow = TP::b_row8_16(lane);
    const int64_t ost = int64_t(a.H) * DV;
    const int64_t obase = (tok * a.H + head) * DV + slice * W::DVS + 16 * wave + 4 * g4;
    for (int n = n0; n < n1; ++n) {
      const int c = chunk_of(n);
      const int64_t t0 = int64_t(c) * C;
      const float* ga = gates(n);
      const uint32_t kb = TK::at(Ks(n)) + kcol, vb = TV::at(Vs(n)) + vcol;
      if constexpr (OUT == 2 && !REV)
        if (c % kBlockChunks == 0) keep(c / kBlockChunks);
      // the chunk's values in this wavefront's columns, tokens along k
      F vf[U];
#pragma unroll
      for (int u = 0; u < U; ++u) vf[u] = TV::col8_16(vb, u, wave);

      f32x4 acc[TT], dots[TT];  // dots: the tensor that the outputs meet, at the outputs' places
      if constexpr (OUT == 2)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const int64_t t = t0 + 16 * tt + l16;
          const T* dp = static_cast<const T*>(a.dot) + obase + (t < a.T ? t : a.T - 1) * ost;
          if constexpr (sizeof(T) == 2) dots[tt] = __builtin_convertvector(*reinterpret_cast<const bf16x4*>(dp), f32x4);
          else dots[tt] = *reinterpret_cast<const f32x4*>(dp);
        }
      if constexpr (OUT > 0) {
        const uint32_t qb = TK::at(Qs(n)) + qrow;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[tt] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk) {
          const f32x4 hi = 2 * kk + 1 < NKT ? S[(2 * kk + 1) % NKT] : f32x4{0, 0, 0, 0};
          const Parts<T, kOut, 8> sf(__builtin_shufflevector(S[2 * kk], hi, 0, 1, 2, 3, 4, 5, 6, 7));
          // a result's next addend waits for it: sums over different results in turn
          F qf[TT];
#pragma unroll
          for (int tt = 0; tt < TT; ++tt) qf[tt] = TK::row44_16(qb, tt, kk);
#pragma unroll
          for (int i = kOut - 1; i >= 0; --i)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) acc[tt] = O::mma16(part_of(sf, i), qf[tt], acc[tt]);
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[tt] *= ga[2 * C + 16 * tt + l16];
      }

      const float ec = ga[4 * C];
      const bool clean = fabsf(S[0][0]) < INFINITY;
#pragma unroll
      for (int i = 0; i < NKT; ++i) S[i] *= ec;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* w = ga + 3 * C + 32 * u + 8 * g4;
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(w), w1 = *reinterpret_cast<const f32x4*>(w + 4);
        const Parts<T, kExact, 8> x(O::unpack(vf[u]) * __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7));
        F kf[NKT];
#pragma unroll
        for (int i = 0; i < NKT; ++i) kf[i] = TK::col8_16(kb, u, i);
#pragma unroll
        for (int j = kExact - 1; j >= 0; --j)
#pragma unroll
          for (int i = 0; i < NKT; ++i) S[i] = O::mma16(kf[i], part_of(x, j), S[i]);
      }

      if constexpr (OUT > 0) {
        // Scores of tokens that do not see a value are zero, and zero times a NaN or infinity is not: such
        // values, which the updated state of their column shows, leave the product.
        const bool spoiled = __any(clean && !(fabsf(S[0][0]) < INFINITY));
        if (spoiled)
#pragma unroll
          for (int u = 0; u < U; ++u) vf[u] = Finite<T>::only(vf[u]);
        lds_barrier();  // the scores are there
        const uint32_t pb = TP::at(P) + prow;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = kOut - 1; i >= 0; --i)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
              if (REV ? u < tt / 2 : u > tt / 2) continue;
              acc[tt] = O::mma16(vf[u], TP::row8_16(pb + i * W::kP1, tt, u), acc[tt]);
            }
        if (spoiled) {  // and are added for the tokens that see them
          const int live = a.T - c * C < C ? a.T - c * C : C;
#pragma unroll 1
          for (int s = 0; s < live; ++s) {
            const f32x4 x = TV::get4(Vs(n), s, 16 * wave + 4 * g4);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
              const int t = 16 * tt + l16;
              const float p = io<T>::load(P, TP::off(t, s));
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[tt][r] += (REV ? s >= t : s <= t) && !(fabsf(x[r]) < INFINITY) ? p * x[r] : 0.f;
            }
          }
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const int64_t t = t0 + 16 * tt + l16;
          f32x4 x = acc[tt];
          if constexpr (!REV) x *= a.scale;
          if (t < a.T) store4(static_cast<TO*>(a.o) + obase + t * ost, x);
          if constexpr (OUT == 2) {
            x *= dots[tt];
            float d = (x[0] + x[1]) + (x[2] + x[3]);
            d += __shfl_xor(d, 16);
            d += __shfl_xor(d, 32);
            if (g4 == 0 && t < a.T) a.x[(int64_t(part) * a.B * a.H + bh) * a.T + t] = d;
          }
        }
      }
      if constexpr (OUT == 2 && REV)
        if (c % kBlockChunks == 0 && c > 0) meet(c / kBlockChunks);
      lds_barrier();
    }
  }

  if constexpr (OUT == 2 && !REV)
    if (seg == a.nseg - 1) keep(nblk);
  if (a.S_out && (a.S_out_seg || seg == a.nseg - 1)) {
    float* So = a.S_out + (a.S_out_seg ? bh * a.nseg + seg : bh) * DK * DV;
#pragma unroll
    for (int i = 0; i < NKT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) So[(16 * i + 4 * g4 + r) * DV + col] = S[i][r];
  }
}

template <typename T, typename TO, int DK, int DV, int OUT, bool REV>
hipError_t launch_walk(const LinearArgs& a, hipStream_t st) {
  using W = WalkShape<T, DK, DV, OUT>;
  auto kern = linear_walk_kernel<T, TO, DK, DV, OUT, REV>;
  static std::atomic<uint64_t> done{0};
  if constexpr (W::lds > 65536) {
    const hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kern), int(W::lds), done);
    if (e != hipSuccess) return e;
  }
  const int64_t grid = int64_t(a.B) * a.H * a.nseg * W::NSL;
  kern<<<dim3(uint32_t(grid)), W::NT, W::lds, st>>>(a);
  return hipGetLastError();
}

template <typename T, int DK, int DV, bool REV>
hipError_t launch_walk_d(const LinearArgs& a, hipStream_t st) {
  if (!a.o) return launch_walk<T, T, DK, DV, 0, REV>(a, st);
  if (a.dot) return a.out_bf16 ? launch_walk<T, bf16_t, DK, DV, 2, REV>(a, st) : launch_walk<T, float, DK, DV, 2, REV>(a, st);
  return a.out_bf16 ? launch_walk<T, bf16_t, DK, DV, 1, REV>(a, st) : launch_walk<T, float, DK, DV, 1, REV>(a, st);
}

template <typename T, int DK, bool REV>
hipError_t launch_walk_k(const LinearArgs& a, hipStream_t st) {
  switch (a.dv) {
    case 16: return launch_walk_d<T, DK, 16, REV>(a, st);
    case 32: return launch_walk_d<T, DK, 32, REV>(a, st);
    case 64: return launch_walk_d<T, DK, 64, REV>(a, st);
    default: return launch_walk_d<T, DK, 128, REV>(a, st);
  }
}

template <typename T, bool REV>
hipError_t launch_walk_t(const LinearArgs& a, hipStream_t st) {
  switch (a.dk) {
    case 16: return launch_walk_k<T, 16, REV>(a, st);
    case 32: return launch_walk_k<T, 32, REV>(a, st);
    case 64: return launch_walk_k<T, 64, REV>(a, st);
    default: return launch_walk_k<T, 128, REV>(a, st);
  }
}

}  // namespace

}  // namespace kda
