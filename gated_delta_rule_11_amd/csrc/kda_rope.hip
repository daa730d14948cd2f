// kda_rope.hip -- rotary positions over rows of heads, and their gradient (the turn backwards).
//
// Bound by the bytes of x and y.  One wavefront takes one row and some of its heads: its lanes form the
// row's sines and cosines once, one pair (two where half > 64) each, and hand them round through the
// LDS; then each lane turns one unit of 16 channels for head after head, so the row's sines cost a
// few instructions a head and neighbouring lanes read neighbouring memory.
#include "kda_mix_launch.hpp"
#include "kda_rotary.hpp"

namespace kda {

namespace {

template <typename T, typename TO>
__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs a) {
  __shared__ float sc[4][2][128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t item = int64_t(blockIdx.x) * 4 + wave;
  const int parts = (a.H + a.heads - 1) / a.heads;
  const int64_t row = item / parts;
  if (row >= a.n) return;  // (no barrier follows: a wavefront only reads what it wrote itself)
  rotate_row<T, TO>(a, row, 0, int(item % parts) * a.heads, sc[wave], lane);
}

template <typename T, typename TO>
hipError_t launch(const RopeArgs& a, hipStream_t st) {
  const int64_t items = int64_t(a.n) * ((a.H + a.heads - 1) / a.heads);
  rope_kernel<T, TO><<<dim3(uint32_t((items + 3) / 4)), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t st) {
  if (a.in_bf16) return a.out_bf16 ? launch<bf16_t, bf16_t>(a, st) : launch<bf16_t, float>(a, st);
  return a.out_bf16 ? launch<float, bf16_t>(a, st) : launch<float, float>(a, st);
}

}  // namespace kda
