// kda_linear_step.hip -- one token of linear attention with a decay per head:
//   S' = e^g S + k v^T,   o = scale S'^T q = scale (e^g S^T q + (q . k) v).
// The call moves the fp32 state once in and once out and does two multiply-adds per element on
// the way: bound by memory.  One workgroup per (n, h) in the single-token layout of
// kda_launch.hpp (thread (rg, j4): four value columns of rows rg + NR i), 16-byte streaming
// accesses, the output's sum over rows through LDS.  Measured (256 sequences, 32 heads, 128 x 128): 179
// us, 6.0 TB/s, where a large copy reaches 5.05.
#include "kda_common.hpp"
#include "kda_mix_launch.hpp"

namespace kda {

namespace {

template <int DK, int DV, typename T, typename TO>
__global__ __launch_bounds__(decode_threads(DK, DV)) void linear_step_kernel(const LinearStepArgs a) {
  using Sh = DecodeShape<DK, DV>;
  __shared__ f32x4 part[Sh::NR][Sh::NJ];
  __shared__ float ks[DK], qs[DK];
  const int tid = threadIdx.x, j4 = tid % Sh::NJ, rg = tid / Sh::NJ;
  const int64_t nh = blockIdx.x;
  const T* kp = static_cast<const T*>(a.k) + nh * DK;
  const T* qp = static_cast<const T*>(a.q) + nh * DK;
  const f32x4* Si = reinterpret_cast<const f32x4*>(a.S_in + nh * DK * DV);
  f32x4* So = reinterpret_cast<f32x4*>(a.S_out + nh * DK * DV);
  f32x4 s[Sh::RPT];
#pragma unroll
  for (int i = 0; i < Sh::RPT; ++i) s[i] = __builtin_nontemporal_load(Si + (rg + Sh::NR * i) * Sh::NJ + j4);
  for (int i = tid; i < DK; i += Sh::NTHREADS) {
    ks[i] = io<T>::load(kp, i);
    qs[i] = io<T>::load(qp, i);
  }
  f32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = io<T>::load(static_cast<const T*>(a.v) + nh * DV, 4 * j4 + j);
  const float decay = fast_exp2(kLog2e * a.g[a.g_head ? nh % a.H : nh]);
  __syncthreads();
  f32x4 acc = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < Sh::RPT; ++i) {
    const int row = rg + Sh::NR * i;
    s[i] = s[i] * decay + v * ks[row];
    acc += s[i] * qs[row];
    __builtin_nontemporal_store(s[i], So + row * Sh::NJ + j4);
  }
  part[rg][j4] = acc;
  __syncthreads();
  if (tid < DV) {
    float o = 0.f;
#pragma unroll
    for (int r = 0; r < Sh::NR; ++r) o += part[r][tid / 4][tid % 4];
    io<TO>::store(static_cast<TO*>(a.o) + nh * DV, tid, a.scale * o);
  }
}

template <int DK, int DV>
hipError_t launch(const LinearStepArgs& a, hipStream_t st) {
  const dim3 grid(uint32_t(int64_t(a.N) * a.H));
  constexpr int nt = decode_threads(DK, DV);
  if (a.in_bf16) {
    if (a.out_bf16) linear_step_kernel<DK, DV, bf16_t, bf16_t><<<grid, nt, 0, st>>>(a);
    else linear_step_kernel<DK, DV, bf16_t, float><<<grid, nt, 0, st>>>(a);
  } else {
    if (a.out_bf16) linear_step_kernel<DK, DV, float, bf16_t><<<grid, nt, 0, st>>>(a);
    else linear_step_kernel<DK, DV, float, float><<<grid, nt, 0, st>>>(a);
  }
  return hipGetLastError();
}

template <int DK>
hipError_t launch_k(const LinearStepArgs& a, hipStream_t st) {
  switch (a.dv) {
    case 16: return launch<DK, 16>(a, st);
    case 32: return launch<DK, 32>(a, st);
    case 64: return launch<DK, 64>(a, st);
    default: return launch<DK, 128>(a, st);
  }
}

}  // namespace

hipError_t launch_linear_step(const LinearStepArgs& a, hipStream_t st) {
  switch (a.dk) {
    case 16: return launch_k<16>(a, st);
    case 32: return launch_k<32>(a, st);
    case 64: return launch_k<64>(a, st);
    default: return launch_k<128>(a, st);
  }
}

}  // namespace kda
