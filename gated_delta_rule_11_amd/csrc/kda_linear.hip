// kda_linear.hip -- linear attention with a decay per head: what lies between the walks of
// kda_linear_walk.hpp.  Measured: the scan of 16 segments of 8 heads 6 us; dg of 4 x 4001 tokens and
// 32 heads 10 us; both small beside the walks.
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

// The sum over a workgroup of 256, in 64 bits and a fixed order, in every thread.
__device__ __forceinline__ double sum_256(double v, double* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// dg of one block of chunks (kBlockChunks of C tokens, one token a thread): the block's boundary
// term and the sum from each token to the block's end, in 64 bits.  For a decay per head only
// their sum over the block is kept.
__global__ __launch_bounds__(256) void linear_dg_kernel(const LinearDgArgs a) {
  __shared__ double sums[4], total[4];
  const int nblk = (a.T + a.block - 1) / a.block;
  const int64_t bh = blockIdx.x / nblk;
  const int blk = blockIdx.x % nblk, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t = int64_t(blk) * a.block + tid, rows = a.BH * a.T;
  const bool live = tid < a.block && t < a.T;
  double v = 0.0;
  if (live)
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
  for (int w = wave + 1; w < 4; ++w) v += sums[w];
  v += edge;
  if (a.block_sum) {
    v = sum_256(live ? v : 0.0, total);
    if (tid == 0) a.block_sum[bh * nblk + blk] = v;
  } else if (live) {
    a.dg[((bh / a.H) * a.T + t) * a.H + bh % a.H] = float(v);
  }
}

// dg [H] from the blocks' sums [B, H, nblk]: one workgroup per head.
__global__ __launch_bounds__(256) void linear_dg_sum_kernel(const double* x, float* dg, int64_t B, int H, int64_t nblk) {
  __shared__ double lds[4];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < B * nblk; i += 256) s += x[((i / nblk) * H + blockIdx.x) * nblk + i % nblk];
  s = sum_256(s, lds);
  if (threadIdx.x == 0) dg[blockIdx.x] = float(s);
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
  linear_dg_kernel<<<dim3(uint32_t(a.BH * nblk)), 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_linear_dg_sum(const double* x, float* dg, int64_t B, int H, int64_t nblk, hipStream_t st) {
  linear_dg_sum_kernel<<<dim3(uint32_t(H)), 256, 0, st>>>(x, dg, B, H, nblk);
  return hipGetLastError();
}

}  // namespace kda
