// kda_linear.hip -- linear attention with a decay per head: what lies between the walks of
// kda_linear_walk.hpp.
#include "kda_common.hpp"
#include "kda_mix_launch.hpp"

namespace kda {

namespace {

// The segments' entry states in order, E_0 = S_in (or 0), E_{p+1} = decay_p E_p + St_p.  One thread per
// state element; S_in may lie transposed.  Segments are few, and loads of later ones do not wait for
// earlier sums.
__global__ __launch_bounds__(256) void linear_scan_kernel(const LinearScanArgs a) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int n = a.dk * a.dv;
  if (i >= a.BH * n) return;
  const int64_t bh = i / n, e = i % n;
  float x = 0.f;
  if (a.S_in) x = a.S_in[bh * n + (a.state_tr ? (e % a.dv) * a.dk + e / a.dv : e)];
#pragma unroll 8
  for (int p = 0; p < a.nseg; ++p) {
    const float s = a.St[(bh * a.nseg + p) * n + e], d = a.decay[bh * a.nseg + p];
    a.E[(bh * a.nseg + p) * n + e] = x;
    x = x * d + s;
  }
}

// dg of one block of chunks (kBlockChunks of C tokens, one token a thread): the block's boundary
// term and the sum from each token to the block's end, in 64 bits.
__global__ __launch_bounds__(512) void linear_dg_kernel(const LinearDgArgs a) {
  __shared__ double sums[8];
  const int nblk = (a.T + a.block - 1) / a.block;
  const int64_t bh = blockIdx.x / nblk;
  const int blk = blockIdx.x % nblk, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t = int64_t(blk) * a.block + tid, rows = a.BH * a.T;
  double v = 0.0;
  if (tid < a.block && t < a.T)
    for (int p = 0; p < a.parts; ++p) v += double(a.xq[p * rows + bh * a.T + t]) - double(a.xk[p * rows + bh * a.T + t]);
  double edge = 0.0;
  for (int p = 0; p < a.parts; ++p) edge += double(a.bsum[(bh * nblk + blk) * a.parts + p]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double x = __shfl_down(v, d);
    if (lane + d < 64) v += x;
  }
  if (lane == 0) sums[wave] = v;
  __syncthreads();
  for (int w = wave + 1; w < 8; ++w) v += sums[w];
  if (tid < a.block && t < a.T) a.dg[((bh / a.H) * a.T + t) * a.H + bh % a.H] = float(v + edge);
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

}  // namespace

hipError_t launch_linear_walk(const LinearArgs& a, hipStream_t st) {
  if (a.reverse) return a.in_bf16 ? launch_linear_rev_bf16(a, st) : launch_linear_rev_f32(a, st);
  return a.in_bf16 ? launch_linear_fwd_bf16(a, st) : launch_linear_fwd_f32(a, st);
}

hipError_t launch_linear_scan(const LinearScanArgs& a, hipStream_t st) {
  const int64_t n = (a.BH * a.dk * a.dv + 255) / 256;
  linear_scan_kernel<<<dim3(uint32_t(n)), 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_linear_dg(const LinearDgArgs& a, hipStream_t st) {
  const int64_t nblk = (a.T + a.block - 1) / a.block;
  linear_dg_kernel<<<dim3(uint32_t(a.BH * nblk)), 512, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_linear_dg_sum(const float* x, float* dg, int64_t rows, int H, hipStream_t st) {
  linear_dg_sum_kernel<<<dim3(uint32_t(H)), 256, 0, st>>>(x, dg, rows, H);
  return hipGetLastError();
}

}  // namespace kda
