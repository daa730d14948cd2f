// kda_linear_bwd.hip -- gradients of linear attention with a decay per head.
//
// With A_ts = e^{G_t - G_s} (s <= t, G the log-decays summed inside a chunk), S the state that
// enters the chunk and R = dL/dS after it,
//   dq_t = scale (e^{G_t} S do_t + sum_s A_ts (do_t . v_s) k_s)
//   dk_s = scale sum_t A_ts (do_t . v_s) q_t + e^{G_C - G_s} R v_s
//   dv_s = scale sum_t A_ts (q_t . k_s) do_t + e^{G_C - G_s} R^T k_s
// and a log-decay scales all that crosses it: with M_us = scale A_us (q_u . k_s)(do_u . v_s),
//   dg_t = e^{G_C} <R, S> + sum_{s < t} k_s . dk'_s + sum_{u >= t} q_u . dq'_u
//          + sum_{u >= t} (sum_{s < u} M_us - sum_{w > u} M_wu),
// dk', dq' being the parts that come through R and S.  The pairs s = u are left out of both inner
// sums (they cancel exactly), and the crossing terms are sums in one direction, so a chunk's dg is
// as exact as its products.
//
// Two walks over the chunks (kda_linear_fwd.hip) have left S and R of every chunk in memory; this
// kernel then takes one workgroup per (chunk, b, h), with no order between chunks.  Four
// wavefronts (fewer where the head sizes are small); wavefront w forms key channels 32 w .. + 31 of
// dq and dk and value channels 32 w .. + 31 of dv, all transposed (channels x tokens).
// Its rows of S and R come straight from memory into fragments.  With bf16 elements S v and R v
// products take S and R as two bf16 parts each: dg is fp32 and needs them.  The scores and the
// copy of R behind dv are rounded to bf16, as the gradients themselves may be.
#include "kda_mix_launch.hpp"
#include "kda_mma.hpp"

namespace kda {

namespace {

constexpr float kLeastLog = -1.0e4f;  // as in the forward

template <typename T, int DK, int DV>
struct GradShape {
  static constexpr int C = linear_chunk(sizeof(T) == 2);
  static constexpr int DKP = DK < 32 ? 32 : DK, DVP = DV < 32 ? 32 : DV;
  static constexpr int NKT = DKP / 32, NVT = DVP / 32;
  static constexpr int NW0 = NKT > NVT ? NKT : NVT;
  static constexpr int NW = NW0 < 2 ? 2 : NW0, NT = 64 * NW;
  static constexpr int TT = C / 32;
  static constexpr size_t elems = size_t(2) * C * DKP + size_t(2) * C * DVP + size_t(3) * C * C;
  // G hi, G lo, e^{G_C - G}, e^G, rows of M, columns of M (per score tile), k . dk', q . dq' (per wavefront)
  static constexpr int kFloats = 4 * C + 2 * 3 * C + 2 * NW * C + NW;
  static constexpr size_t lds = elems * sizeof(T) + kFloats * sizeof(float);
};

template <typename T, typename TG, int DK, int DV>
__global__ __launch_bounds__((GradShape<T, DK, DV>::NT)) void linear_grad_kernel(const LinearBwdArgs a, int nch) {
  using W = GradShape<T, DK, DV>;
  using O = Op<T>;
  using F = typename O::frag;
  using TK = Tile<T, W::DKP>;
  using TV = Tile<T, W::DVP>;
  using TP = Tile<T, W::C>;
  constexpr int C = W::C, NW = W::NW, NT = W::NT, TT = W::TT;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Qs = reinterpret_cast<T*>(smem);
  T* Ks = Qs + C * W::DKP;
  T* Vs = Ks + C * W::DKP;
  T* Os = Vs + C * W::DVP;  // do
  T* Pt = Os + C * W::DVP;  // [s][t] scale A (q.k)
  T* dA = Pt + C * C;       // [t][s] scale A (do.v)
  T* dAt = dA + C * C;      // [s][t]
  float* ghi = reinterpret_cast<float*>(dAt + C * C);
  float* glo = ghi + C;
  float* wk = glo + C;      // e^{G_C - G}
  float* eg = wk + C;       // e^G
  float* mrow = eg + C;     // [3][C]
  float* mcol = mrow + 3 * C;
  float* kdk = mcol + 3 * C;  // [NW][C]
  float* qdq = kdk + NW * C;
  float* rs = qdq + NW * C;  // [NW]

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h2 = lane >> 5, l32 = lane & 31;
  const int64_t item = xcd_order(blockIdx.x, gridDim.x);
  const int64_t bh = item / nch, c = item % nch;
  const int64_t b = bh / a.H, head = bh % a.H;
  const int64_t t0 = c * C, valid = a.T - t0 < C ? a.T - t0 : C;
  const int64_t row0 = (b * a.T + t0) * a.H + head;  // in rows of a head
  const int64_t kst = int64_t(a.H) * DK, vst = int64_t(a.H) * DV;

  {
    Stage<T, C, DK, W::DKP, NT> s0, s1;
    Stage<T, C, DV, W::DVP, NT> s2, s3;
    s0.load(static_cast<const T*>(a.q) + row0 * DK, kst, valid, tid);
    s1.load(static_cast<const T*>(a.k) + row0 * DK, kst, valid, tid);
    s2.load(static_cast<const T*>(a.v) + row0 * DV, vst, valid, tid);
    s3.load(static_cast<const T*>(a.d_o) + row0 * DV, vst, valid, tid);
    if (wave == 0) {
      float g = 0.f;
      if (lane < valid) g = a.g_head ? a.g[head] : a.g[row0 + int64_t(lane) * a.H];
      g = g < kLeastLog ? kLeastLog : g;
      double G = double(g) * 1.4426950408889634;
#pragma unroll
      for (int d = 1; d < C; d <<= 1) {
        const double up = __shfl_up(G, d);
        if (lane >= d) G += up;
      }
      const double Gc = __shfl(G, C - 1);
      if (lane < C) {
        const float hi = float(G);
        ghi[lane] = hi;
        glo[lane] = float(G - double(hi));
        wk[lane] = fast_exp2(float(Gc - G));
        eg[lane] = fast_exp2(float(G));
      }
    }
    s0.store(Qs, tid);
    s1.store(Ks, tid);
    s2.store(Vs, tid);
    s3.store(Os, tid);
  }
  for (int i = tid; i < 6 * C; i += NT) mrow[i] = 0.f;  // mrow and mcol
  __syncthreads();

  // score tiles (s tile, t tile) at or below the diagonal, in both orientations
  constexpr int NP = TT == 2 ? 3 : 1;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (p % NW != wave) continue;
    const int si = p == 2 ? 1 : 0, ti = p == 0 ? 0 : 1;  // TT == 1: only (0, 0)
    {  // rows t, column s
      f32x16 x = zero16(), y = zero16();
#pragma unroll
      for (int kk = 0; kk < W::DKP / 16; ++kk)
        x = O::mma32(TK::row8(Qs, 32 * ti + l32, 16 * kk + 8 * h2), TK::row8(Ks, 32 * si + l32, 16 * kk + 8 * h2), x);
#pragma unroll
      for (int kk = 0; kk < W::DVP / 16; ++kk)
        y = O::mma32(TV::row8(Os, 32 * ti + l32, 16 * kk + 8 * h2), TV::row8(Vs, 32 * si + l32, 16 * kk + 8 * h2), y);
      const int s = 32 * si + l32;
      const float shi = ghi[s], slo = glo[s];
      float col = 0.f;
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int t = 32 * ti + 8 * r4 + 4 * h2;
        const f32x4 thi = *reinterpret_cast<const f32x4*>(ghi + t), tlo = *reinterpret_cast<const f32x4*>(glo + t);
        f32x4 px, py;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float d = a.scale * fast_exp2((thi[j] - shi) + (tlo[j] - slo));
          px[j] = s <= t + j ? x[4 * r4 + j] * d : 0.f;
          py[j] = s <= t + j ? y[4 * r4 + j] * d : 0.f;
          col += s < t + j ? px[j] * y[4 * r4 + j] : 0.f;
        }
        TP::put4(Pt, s, t, px);
        TP::put4(dAt, s, t, py);
      }
      col = sum_halves(col);
      if (h2 == 0) mcol[p * C + s] = col;
    }
    {  // rows s, column t
      f32x16 x = zero16(), y = zero16();
#pragma unroll
      for (int kk = 0; kk < W::DKP / 16; ++kk)
        x = O::mma32(TK::row8(Ks, 32 * si + l32, 16 * kk + 8 * h2), TK::row8(Qs, 32 * ti + l32, 16 * kk + 8 * h2), x);
#pragma unroll
      for (int kk = 0; kk < W::DVP / 16; ++kk)
        y = O::mma32(TV::row8(Vs, 32 * si + l32, 16 * kk + 8 * h2), TV::row8(Os, 32 * ti + l32, 16 * kk + 8 * h2), y);
      const int t = 32 * ti + l32;
      const float thi = ghi[t], tlo = glo[t];
      float row = 0.f;
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int s = 32 * si + 8 * r4 + 4 * h2;
        const f32x4 shi = *reinterpret_cast<const f32x4*>(ghi + s), slo = *reinterpret_cast<const f32x4*>(glo + s);
        f32x4 py;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float d = a.scale * fast_exp2((thi - shi[j]) + (tlo - slo[j]));
          py[j] = s + j <= t ? y[4 * r4 + j] * d : 0.f;
          row += s + j < t ? py[j] * x[4 * r4 + j] : 0.f;
        }
        TP::put4(dA, t, s, py);
      }
      row = sum_halves(row);
      if (h2 == 0) mrow[p * C + t] = row;
    }
  }
  __syncthreads();

  const float* Sp = a.S + (bh * nch + c) * DK * DV;
  const float* Rp = a.R + (bh * nch + c) * DK * DV;
  TG* const dqp = static_cast<TG*>(a.dq) + row0 * DK;
  TG* const dkp = static_cast<TG*>(a.dk_) + row0 * DK;
  TG* const dvp = static_cast<TG*>(a.dv_) + row0 * DV;

  float dot = 0.f;
  if (wave < W::NKT) {
    // rows 32 wave .. + 31 of S do and R v
    f32x16 xq[TT], xk[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) xq[i] = xk[i] = zero16();
    const int row = 32 * wave + l32;
#pragma unroll 2
    for (int kk = 0; kk < W::DVP / 16; ++kk) {
      const int cc = 16 * kk + 8 * h2;
      f32x8 s = {0, 0, 0, 0, 0, 0, 0, 0}, r = s;
      if (row < DK && cc < DV) {
        s = *reinterpret_cast<const f32x8*>(Sp + row * DV + cc);
        r = *reinterpret_cast<const f32x8*>(Rp + row * DV + cc);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) dot += s[j] * r[j];
      const F sh = O::pack(s), rh = O::pack(r);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const F od = TV::row8(Os, 32 * i + l32, cc), vv = TV::row8(Vs, 32 * i + l32, cc);
        xq[i] = O::mma32(sh, od, xq[i]);
        xk[i] = O::mma32(rh, vv, xk[i]);
        if constexpr (sizeof(T) == 2) {
          xq[i] = O::mma32(O::pack(s - O::unpack(sh)), od, xq[i]);
          xk[i] = O::mma32(O::pack(r - O::unpack(rh)), vv, xk[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int t = 32 * i + l32;
      const float eq = a.scale * eg[t], ek = wk[t];
      float sq = 0.f, sk = 0.f;
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const f32x4 q4 = TK::get4(Qs, t, 32 * wave + 8 * r4 + 4 * h2), k4 = TK::get4(Ks, t, 32 * wave + 8 * r4 + 4 * h2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xq[i][4 * r4 + j] *= eq;
          xk[i][4 * r4 + j] *= ek;
          sq += q4[j] * xq[i][4 * r4 + j];
          sk += k4[j] * xk[i][4 * r4 + j];
        }
      }
      sq = sum_halves(sq);
      sk = sum_halves(sk);
      if (h2 == 0) {
        qdq[wave * C + t] = sq;
        kdk[wave * C + t] = sk;
      }
    }
#pragma unroll
    for (int u = 0; u < C / 16; ++u) {
      const F kf = TK::col44(Ks, 16 * u + 8 * h2, 16 * u + 8 * h2 + 4, 32 * wave, lane);
      const F qf = TK::col44(Qs, 16 * u + 8 * h2, 16 * u + 8 * h2 + 4, 32 * wave, lane);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        if (u < 2 * (i + 1)) xq[i] = O::mma32(kf, TP::row8(dA, 32 * i + l32, 16 * u + 8 * h2), xq[i]);   // s <= t
        if (u >= 2 * i) xk[i] = O::mma32(qf, TP::row8(dAt, 32 * i + l32, 16 * u + 8 * h2), xk[i]);       // t >= s
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int t = 32 * i + l32;
      if (t < valid)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int cc = 32 * wave + 8 * r4 + 4 * h2;
          if (cc < DK) {
            store4(dqp + t * kst + cc, f32x4{xq[i][4 * r4], xq[i][4 * r4 + 1], xq[i][4 * r4 + 2], xq[i][4 * r4 + 3]});
            store4(dkp + t * kst + cc, f32x4{xk[i][4 * r4], xk[i][4 * r4 + 1], xk[i][4 * r4 + 2], xk[i][4 * r4 + 3]});
          }
        }
    }
  } else {
    for (int i = lane; i < C; i += 64) qdq[wave * C + i] = kdk[wave * C + i] = 0.f;
  }
  if (wave < W::NVT) {
    // rows 32 wave .. + 31 of R^T k, then the chunk's own pairs
    f32x16 x[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) x[i] = zero16();
    const int col = 32 * wave + l32;
#pragma unroll 2
    for (int kk = 0; kk < W::DKP / 16; ++kk) {
      f32x8 r = {0, 0, 0, 0, 0, 0, 0, 0};
      const int cc = 16 * kk + 8 * h2;
      if (col < DV && cc < DK)
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = Rp[(cc + j) * DV + col];
      const F rh = O::pack(r);
#pragma unroll
      for (int i = 0; i < TT; ++i) x[i] = O::mma32(rh, TK::row8(Ks, 32 * i + l32, cc), x[i]);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const float ek = wk[32 * i + l32];
#pragma unroll
      for (int r = 0; r < 16; ++r) x[i][r] *= ek;
    }
#pragma unroll
    for (int u = 0; u < C / 16; ++u) {
      const F of = TV::col44(Os, 16 * u + 8 * h2, 16 * u + 8 * h2 + 4, 32 * wave, lane);
#pragma unroll
      for (int i = 0; i < TT; ++i)
        if (u >= 2 * i) x[i] = O::mma32(of, TP::row8(Pt, 32 * i + l32, 16 * u + 8 * h2), x[i]);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int t = 32 * i + l32;
      if (t < valid)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int cc = 32 * wave + 8 * r4 + 4 * h2;
          if (cc < DV)
            store4(dvp + t * vst + cc, f32x4{x[i][4 * r4], x[i][4 * r4 + 1], x[i][4 * r4 + 2], x[i][4 * r4 + 3]});
        }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
  if (lane == 0) rs[wave] = dot;
  __syncthreads();

  if (wave == 0) {
    // before t: k . dk' of earlier tokens; from t on: q . dq' and the in-chunk pairs
    float before = 0.f, from = 0.f, rsum = 0.f;
    for (int w = 0; w < NW; ++w) rsum += rs[w];
    if (lane < C) {
      for (int w = 0; w < NW; ++w) {
        before += kdk[w * C + lane];
        from += qdq[w * C + lane];
      }
      for (int p = 0; p < 3; ++p) from += mrow[p * C + lane] - mcol[p * C + lane];
    }
    const float own = before;
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
      const float up = __shfl_up(before, d), dn = __shfl_down(from, d);
      if (lane >= d) before += up;
      if (lane + d < C) from += dn;
    }
    if (lane < valid) a.dg[row0 + int64_t(lane) * a.H] = eg[C - 1] * rsum + (before - own) + from;
  }
}

// dg [H] from x [rows, H]: one workgroup per head, sums in 64 bits, in a fixed order.
__global__ __launch_bounds__(256) void linear_dg_sum_kernel(const float* x, float* dg, int64_t rows, int H) {
  __shared__ double part[256];
  double s = 0.0;
  for (int64_t r = threadIdx.x; r < rows; r += 256) s += double(x[r * H + blockIdx.x]);
  part[threadIdx.x] = s;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if (int(threadIdx.x) < d) part[threadIdx.x] += part[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[blockIdx.x] = float(part[0]);
}

template <typename T, typename TG, int DK, int DV>
hipError_t launch(const LinearBwdArgs& a, hipStream_t st) {
  using W = GradShape<T, DK, DV>;
  auto kern = linear_grad_kernel<T, TG, DK, DV>;
  static_assert(W::lds <= 160 * 1024, "LDS of a compute unit");
  static std::atomic<uint64_t> done{0};
  if constexpr (W::lds > 65536) {
    const hipError_t e = set_lds_limit(reinterpret_cast<const void*>(kern), int(W::lds), done);
    if (e != hipSuccess) return e;
  }
  const int nch = (a.T + W::C - 1) / W::C;
  const int64_t grid = int64_t(a.B) * a.H * nch;
  kern<<<dim3(uint32_t(grid)), W::NT, W::lds, st>>>(a, nch);
  return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t launch_g(const LinearBwdArgs& a, hipStream_t st) {
  return a.grad_bf16 ? launch<T, bf16_t, DK, DV>(a, st) : launch<T, float, DK, DV>(a, st);
}

template <typename T, int DK>
hipError_t launch_k(const LinearBwdArgs& a, hipStream_t st) {
  switch (a.dv) {
    case 16: return launch_g<T, DK, 16>(a, st);
    case 32: return launch_g<T, DK, 32>(a, st);
    case 64: return launch_g<T, DK, 64>(a, st);
    default: return launch_g<T, DK, 128>(a, st);
  }
}

template <typename T>
hipError_t launch_t(const LinearBwdArgs& a, hipStream_t st) {
  switch (a.dk) {
    case 16: return launch_k<T, 16>(a, st);
    case 32: return launch_k<T, 32>(a, st);
    case 64: return launch_k<T, 64>(a, st);
    default: return launch_k<T, 128>(a, st);
  }
}

}  // namespace

hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t st) {
  return a.in_bf16 ? launch_t<bf16_t>(a, st) : launch_t<float>(a, st);
}

hipError_t launch_linear_dg_sum(const float* x, float* dg, int64_t rows, int H, hipStream_t st) {
  linear_dg_sum_kernel<<<dim3(uint32_t(H)), 256, 0, st>>>(x, dg, rows, H);
  return hipGetLastError();
}

}  // namespace kda
