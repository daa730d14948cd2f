// kda_linear_fwd.hip -- linear attention with a decay per head, chunked.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// per (b, h), g_t <= 0 a scalar.  In a chunk of C tokens with entry state S and in-chunk
// sums G_t = g_1 + .. + g_t,
//   o_t   = scale (e^{G_t} S^T q_t + sum_{s <= t} e^{G_t - G_s} (q_t . k_s) v_s)
//   S_out = e^{G_C} S + sum_s e^{G_C - G_s} k_s v_s^T.
// Every exponent is a difference of sums over later tokens, so at most 0: nothing overflows,
// whatever the decays.  The sums are formed in 64 bits and kept as two fp32 parts, so a strong
// decay earlier in the chunk does not cost the later differences their low bits.
//
// One workgroup per (b, h, slice of up to 64 value columns, segment) walks its chunks in
// order.  The state slice stays in fp32 accumulators: wavefront w owns value columns
// 32 (w % NDV) .. + 31 and every second tile of 32 key channels.  Per chunk:
//   1  the chunk's rows go from registers to LDS, the next chunk's are fetched;
//   2  three wavefronts form the decayed scores P (32 x 32 tiles at or below the diagonal),
//      the last one the next chunk's gate sums; all put their part of S, rounded to the
//      element type, into LDS as operand fragments;
//   3  outputs o^T (value columns x tokens), one half of the tokens per wavefront, and the
//      state update.
// With bf16 elements P and the copy of S that the outputs read are rounded to bf16, half a
// unit of the last place that the outputs have anyway; the state itself takes its rows
// e^{G_C - G_s} v_s as a sum of two bf16 parts (relative error 2^-17), so it is good to fp32
// accumulation however long the sequence.
//
// Few, long sequences are cut into segments (the ABI layer's rule).  The decay being a scalar,
// a segment's transition is one number: a first walk leaves every segment's end state from
// zero, a scan joins them, a second walk from the true entry states writes the outputs.
//
// REV walks from the last chunk to the first with k = q, v = d_o and weights scale e^{G_t}:
// the gradient R of the state, R_in = e^{G_C} R + scale sum_t e^{G_t} q_t do_t^T.
#include "kda_mix_launch.hpp"
#include "kda_mma.hpp"

namespace kda {

namespace {

// A decay below this is zero in fp32 whatever follows; -inf (a reset) would make differences NaN.
constexpr float kLeastLog = -1.0e4f;

template <typename T, int DK, int DV, bool OUT>
struct WalkShape {
  static constexpr int C = linear_chunk(sizeof(T) == 2);
  static constexpr int DKP = DK < 32 ? 32 : DK;
  static constexpr int DVS = DV < 32 ? 32 : (DV < 64 ? DV : 64);  // value columns of a workgroup, padded
  static constexpr int DVC = DV < 64 ? DV : 64;                   // and those that exist
  static constexpr int NSL = (DV + 63) / 64;
  static constexpr int NDV = DVS / 32;
  static constexpr int NW = 2 * NDV, NT = 64 * NW;
  static constexpr int NKT = DKP / 32, NKW = (NKT + 1) / 2;
  static constexpr int TT = C / 32;
  static constexpr int kK = C * DKP, kV = C * DVS, kP = C * C, kS = DKP * DVS;
  static constexpr size_t elems = size_t(kK) + kV + (OUT ? size_t(kK) + kP + kS : 0);
  static constexpr size_t lds = elems * sizeof(T) + 2 * 4 * C * sizeof(float);
};

template <typename T, typename TO, int DK, int DV, bool OUT, bool REV>
__global__ __launch_bounds__((WalkShape<T, DK, DV, OUT>::NT)) void linear_walk_kernel(const LinearArgs a) {
  using W = WalkShape<T, DK, DV, OUT>;
  using O = Op<T>;
  using TK = Tile<T, W::DKP>;
  using TV = Tile<T, W::DVS>;
  using TP = Tile<T, W::C>;
  constexpr int C = W::C, NW = W::NW, NT = W::NT, NDV = W::NDV, NKT = W::NKT, NKW = W::NKW, TT = W::TT;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Ks = reinterpret_cast<T*>(smem);
  T* Vs = Ks + W::kK;
  T* Qs = Vs + W::kV;
  T* Ps = Qs + (OUT ? W::kK : 0);
  T* Sx = Ps + (OUT ? W::kP : 0);
  float* gates = reinterpret_cast<float*>(Sx + (OUT ? W::kS : 0));  // [2][4][C]: Ghi, Glo, weight, e^G

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h2 = lane >> 5, l32 = lane & 31;
  const int dvt = wave % NDV, hf = wave / NDV;
  int id = xcd_order(blockIdx.x, gridDim.x);
  const int slice = id % W::NSL;
  id /= W::NSL;
  const int seg = id % a.nseg;
  const int64_t bh = id / a.nseg;
  const int64_t b = bh / a.H, head = bh % a.H;
  const int dv0 = slice * 64;

  const int nch = (a.T + C - 1) / C;
  const int n0 = seg * a.seg_chunks;
  const int n1 = n0 + a.seg_chunks < nch ? n0 + a.seg_chunks : nch;
  const int64_t tok = b * a.T;  // the sequence's first row
  const int64_t kst = int64_t(a.H) * DK, vst = int64_t(a.H) * DV;
  const T* kp = static_cast<const T*>(a.k) + (tok * a.H + head) * DK;
  const T* qp = OUT ? static_cast<const T*>(a.q) + (tok * a.H + head) * DK : nullptr;
  const T* vp = static_cast<const T*>(a.v) + (tok * a.H + head) * DV + dv0;
  const float* gp = a.g_head ? a.g + head : a.g + tok * a.H + head;
  const int64_t gst = a.g_head ? 0 : a.H;

  // this wavefront's part of the state
  f32x16 S[NKW];
  const float* Sin = a.S_in ? a.S_in + (a.S_in_seg ? bh * a.nseg + seg : bh) * DK * DV : nullptr;
  // segments after the first of a walk without entry states start from zero
  if (!a.S_in_seg && seg > 0) Sin = nullptr;
  const int col = dv0 + 32 * dvt + l32;  // value column of this lane's state entries
#pragma unroll
  for (int i = 0; i < NKW; ++i) {
    const int kt = hf + 2 * i;
    S[i] = zero16();
    if (Sin && kt < NKT && col < DV)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * kt + crow(r, h2);
        if (row < DK) S[i][r] = Sin[row * DV + col];
      }
  }

  Stage<T, C, DK, W::DKP, NT> sk, sq;
  Stage<T, C, W::DVC, W::DVS, NT> sv;
  auto chunk_of = [&](int n) -> int64_t { return REV ? nch - 1 - n : n; };
  auto fetch = [&](int n) {
    const int64_t t0 = chunk_of(n) * C, valid = a.T - t0;
    sk.load(kp + t0 * kst, kst, valid, tid);
    sv.load(vp + t0 * vst, vst, valid, tid);
    if constexpr (OUT) sq.load(qp + t0 * kst, kst, valid, tid);
  };
  auto gate_of = [&](int n) -> float {
    const int64_t t = chunk_of(n) * C + lane;
    float g = (lane < C && t < a.T) ? gp[t * gst] : 0.f;
    return g < kLeastLog ? kLeastLog : g;
  };
  double total = 0.0;  // log2 of the walk's decay so far (the gate wavefront's lanes)
  auto gate_sums = [&](int n, float g) {
    double G = double(g) * 1.4426950408889634;
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
      const double up = __shfl_up(G, d);
      if (lane >= d) G += up;
    }
    const double Gc = __shfl(G, C - 1);
    total += Gc;
    if (lane < C) {
      float* ga = gates + (n & 1) * 4 * C;
      const float hi = float(G);
      ga[lane] = hi;
      ga[C + lane] = float(G - double(hi));
      ga[2 * C + lane] = REV ? a.scale * fast_exp2(float(G)) : fast_exp2(float(Gc - G));
      ga[3 * C + lane] = fast_exp2(float(G));
    }
  };

  const bool gate_wave = wave == NW - 1;
  float gnext = 0.f;
  if (n0 < n1) {
    if (gate_wave) {
      gate_sums(n0, gate_of(n0));
      if (n0 + 1 < n1) gnext = gate_of(n0 + 1);
    }
    fetch(n0);
  }

  for (int n = n0; n < n1; ++n) {
    const float* ga = gates + (n & 1) * 4 * C;
    const int64_t t0 = chunk_of(n) * C;
    sk.store(Ks, tid);
    sv.store(Vs, tid);
    if constexpr (OUT) sq.store(Qs, tid);
    __syncthreads();
    if (n + 1 < n1) fetch(n + 1);
    if (a.ckpt && col < DV) {
      float* cp = a.ckpt + (bh * nch + chunk_of(n)) * DK * DV;
#pragma unroll
      for (int i = 0; i < NKW; ++i) {
        const int kt = hf + 2 * i;
        if (kt < NKT)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int row = 32 * kt + crow(r, h2);
            if (row < DK) cp[row * DV + col] = S[i][r];
          }
      }
    }
    if constexpr (OUT) {
      typename O::frag* sx = reinterpret_cast<typename O::frag*>(Sx);
#pragma unroll
      for (int i = 0; i < NKW; ++i) {
        const int kt = hf + 2 * i;
        if (kt < NKT)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) sx[((dvt * NKT + kt) * 2 + ks) * 64 + lane] = frag_of<T>(S[i], ks);
      }
      // score tiles (s tile, t tile) at or below the diagonal, transposed: rows s, column t
      constexpr int NP = TT == 2 ? 3 : 1;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        if (p % (NW > 2 ? NW - 1 : NW) != wave) continue;
        const int si = p == 2 ? 1 : 0, ti = p == 0 ? 0 : 1;
        f32x16 c = zero16();
#pragma unroll
        for (int kk = 0; kk < W::DKP / 16; ++kk)
          c = O::mma32(TK::row8(Ks, 32 * si + l32, 16 * kk + 8 * h2), TK::row8(Qs, 32 * ti + l32, 16 * kk + 8 * h2), c);
        const int t = 32 * ti + l32;
        const float ghi = ga[t], glo = ga[C + t];
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int s = 32 * si + 8 * r4 + 4 * h2;
          const f32x4 shi = *reinterpret_cast<const f32x4*>(ga + s), slo = *reinterpret_cast<const f32x4*>(ga + C + s);
          f32x4 x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float d = fast_exp2((ghi - shi[j]) + (glo - slo[j]));
            x[j] = s + j <= t ? c[4 * r4 + j] * d : 0.f;
          }
          TP::put4(Ps, t, s, x);
        }
      }
    }
    if (gate_wave && n + 1 < n1) {
      gate_sums(n + 1, gnext);
      if (n + 2 < n1) gnext = gate_of(n + 2);
    }
    if constexpr (OUT) __syncthreads();

    // the chunk's values, tokens along k: C / 16 fragments of this wavefront's 32 columns
    typename O::frag vf[C / 16];
#pragma unroll
    for (int u = 0; u < C / 16; ++u) vf[u] = TV::col44(Vs, 16 * u + 8 * h2, 16 * u + 8 * h2 + 4, 32 * dvt, lane);

    if constexpr (OUT) {
      if (hf < TT) {
        const int t = 32 * hf + l32;
        const typename O::frag* sx = reinterpret_cast<const typename O::frag*>(Sx);
        f32x16 acc = zero16();
#pragma unroll
        for (int kk = 0; kk < 2 * NKT; ++kk)
          acc = O::mma32(sx[(dvt * NKT * 2 + kk) * 64 + lane], TK::row44(Qs, t, 16 * kk + 4 * h2, 16 * kk + 8 + 4 * h2), acc);
        const float eg = ga[3 * C + t];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] *= eg;
#pragma unroll
        for (int u = 0; u < C / 16; ++u)
          if (u < 2 * (hf + 1)) acc = O::mma32(vf[u], TP::row8(Ps, t, 16 * u + 8 * h2), acc);
        if (t0 + t < a.T) {
          TO* op = static_cast<TO*>(a.o) + ((tok + t0 + t) * a.H + head) * DV + dv0 + 32 * dvt;
#pragma unroll
          for (int r4 = 0; r4 < 4; ++r4) {
            const int c0 = 8 * r4 + 4 * h2;
            if (dv0 + 32 * dvt + c0 < DV) {
              f32x4 x;
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = a.scale * acc[4 * r4 + j];
              store4(op + c0, x);
            }
          }
        }
      }
    }

    const float ec = ga[3 * C + C - 1];
#pragma unroll
    for (int i = 0; i < NKW; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[i][r] *= ec;
#pragma unroll
    for (int u = 0; u < C / 16; ++u) {
      const float* w = ga + 2 * C + 16 * u + 8 * h2;
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(w), w1 = *reinterpret_cast<const f32x4*>(w + 4);
      const f32x8 x = O::unpack(vf[u]) * __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7);
      const typename O::frag hi = O::pack(x);
#pragma unroll
      for (int i = 0; i < NKW; ++i) {
        const int kt = hf + 2 * i;
        if (kt < NKT) {
          const typename O::frag kf = TK::col44(Ks, 16 * u + 8 * h2, 16 * u + 8 * h2 + 4, 32 * kt, lane);
          S[i] = O::mma32(kf, hi, S[i]);
          if constexpr (sizeof(T) == 2) S[i] = O::mma32(kf, O::pack(x - O::unpack(hi)), S[i]);
        }
      }
    }
    __syncthreads();
  }

  if (a.S_out && (a.S_out_seg || seg == a.nseg - 1) && col < DV) {
    float* So = a.S_out + (a.S_out_seg ? bh * a.nseg + seg : bh) * DK * DV;
#pragma unroll
    for (int i = 0; i < NKW; ++i) {
      const int kt = hf + 2 * i;
      if (kt < NKT)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = 32 * kt + crow(r, h2);
          if (row < DK) So[row * DV + col] = S[i][r];
        }
    }
  }
  if (a.seg_decay && gate_wave && lane == 0 && slice == 0) a.seg_decay[bh * a.nseg + seg] = float(exp2(total));
}

// One thread per four state elements: the segments' entry states in order.
__global__ __launch_bounds__(256) void linear_scan_kernel(const LinearScanArgs a) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int n4 = a.n / 4;
  if (i >= a.BH * n4) return;
  const int64_t bh = i / n4, e = i % n4;
  f32x4 x = a.S_in ? reinterpret_cast<const f32x4*>(a.S_in)[bh * n4 + e] : f32x4{0, 0, 0, 0};
  for (int p = 0; p < a.nseg; ++p) {
    reinterpret_cast<f32x4*>(a.E)[(bh * a.nseg + p) * n4 + e] = x;
    x = x * a.decay[bh * a.nseg + p] + reinterpret_cast<const f32x4*>(a.St)[(bh * a.nseg + p) * n4 + e];
  }
}

template <typename T, typename TO, int DK, int DV, bool OUT, bool REV>
hipError_t launch(const LinearArgs& a, hipStream_t st) {
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

template <typename T, int DK, int DV>
hipError_t launch_d(const LinearArgs& a, hipStream_t st) {
  if (a.reverse) return launch<T, T, DK, DV, false, true>(a, st);
  if (!a.o) return launch<T, T, DK, DV, false, false>(a, st);
  return a.out_bf16 ? launch<T, bf16_t, DK, DV, true, false>(a, st) : launch<T, float, DK, DV, true, false>(a, st);
}

template <typename T, int DK>
hipError_t launch_k(const LinearArgs& a, hipStream_t st) {
  switch (a.dv) {
    case 16: return launch_d<T, DK, 16>(a, st);
    case 32: return launch_d<T, DK, 32>(a, st);
    case 64: return launch_d<T, DK, 64>(a, st);
    default: return launch_d<T, DK, 128>(a, st);
  }
}

template <typename T>
hipError_t launch_t(const LinearArgs& a, hipStream_t st) {
  switch (a.dk) {
    case 16: return launch_k<T, 16>(a, st);
    case 32: return launch_k<T, 32>(a, st);
    case 64: return launch_k<T, 64>(a, st);
    default: return launch_k<T, 128>(a, st);
  }
}

}  // namespace

hipError_t launch_linear_walk(const LinearArgs& a, hipStream_t st) {
  return a.in_bf16 ? launch_t<bf16_t>(a, st) : launch_t<float>(a, st);
}

hipError_t launch_linear_scan(const LinearScanArgs& a, hipStream_t st) {
  const int64_t n = (a.BH * (a.n / 4) + 255) / 256;
  linear_scan_kernel<<<dim3(uint32_t(n)), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace kda
