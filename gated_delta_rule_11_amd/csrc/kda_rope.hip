// kda_rope.hip -- rotary positions over rows of heads, and their gradient (the turn backwards).
//
// Bound by the bytes of x and y.  A wavefront's lanes form the sines and cosines of its rows once, one pair after
// another, and hand them round through the LDS; then each lane turns one unit of 16 channels for head after head, so
// the sines cost a few instructions a head and neighbouring lanes read neighbouring memory.  A table of sines would be
// read again for every row; formed in 64 bits they need none, and are right at any position.
//
// Measured: 16270 bf16 rows of 40 heads of 128 (333 MB) in 65 us, 5.1 TB/s; 9001 fp32 rows of 24 heads of 64 with three
// axes (111 MB) in 29, forwards or backwards; 8 rows of 32 heads in 3.7.
#include "kda_mix_launch.hpp"
#include "kda_rotary.hpp"

namespace kda {

namespace {

template <typename T, typename TO>
__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs a) {
  __shared__ float sc[4][2][kSines];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t item = int64_t(blockIdx.x) * 4 + wave;
  const int parts = (a.H + a.heads - 1) / a.heads;
  const int64_t row0 = item / parts * a.rows;
  if (row0 >= a.n) return;  // (no barrier follows: a wavefront only reads what it wrote itself)
  rotate_rows<T, TO>(a, row0, 0, int(item % parts) * a.heads, sc[wave], lane);
}

template <typename T, typename TO>
hipError_t launch(const RopeArgs& a, hipStream_t st) {
  rope_kernel<T, TO><<<dim3(uint32_t((rope_items(a) + 3) / 4)), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t st) {
  if (a.in_bf16) return a.out_bf16 ? launch<bf16_t, bf16_t>(a, st) : launch<bf16_t, float>(a, st);
  return a.out_bf16 ? launch<float, bf16_t>(a, st) : launch<float, float>(a, st);
}

}  // namespace kda
