// kda_prompt.hpp -- what the forward and backward kernels of the packed prompts' attention
// share: the sequence a row belongs to, and tiles of rows staged into LDS.
#pragma once

#include "kda_mix_launch.hpp"
#include "kda_mma.hpp"

namespace kda {

// First row of the sequence that holds row r, and the row behind its last: the last entry of cu
// that is at most r, and the next one.  Entries outside [0, n] or out of order (which a caller
// must not pass) still give 0 <= start <= r and end <= n.
struct Span {
  int start, end;
};
__device__ __forceinline__ Span span_of(const int* cu, int nseq, int n, int r) {
  int lo = 0, hi = nseq;  // cu[lo] <= r (taken as given for lo = 0), cu[hi] > r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  int s = cu[lo], e = cu[hi];
  s = s < 0 ? 0 : (s > r ? r : s);
  e = e > n ? n : e;
  return {s, e};
}

// Rows in use: cu's last entry, within the buffer.
__device__ __forceinline__ int rows_used(const int* cu, int nseq, int n) {
  const int e = cu[nseq];
  return e < 0 ? 0 : (e > n ? n : e);
}

// Zeroes rows [first, last) of one head, by all threads of a workgroup of 256.
template <typename T, int D>
__device__ __forceinline__ void zero_rows(T* out, int64_t stride, int first, int last, int tid) {
  for (int e = tid; e < (last - first) * (D / 4); e += 256)
    store4(out + (first + e / (D / 4)) * stride + 4 * (e % (D / 4)), f32x4{0, 0, 0, 0});
}

// ROWS rows of D elements copied from memory into a Tile, without registers in between.  The LDS
// side of such a copy is one run of 1024 bytes per wavefront, so each lane picks the source chunk
// that belongs at its place.  Rows at or past `last` repeat row `last - 1`: no row outside
// [0, last) is read.
template <typename T, int ROWS, int D, int NW>
__device__ __forceinline__ void copy_rows(T* tile, const T* base, int64_t stride, int row0, int last, int wave,
                                          int lane) {
  typedef Tile<T, D> L;
  constexpr int PER = 64 / L::CH;  // rows of one wavefront's copy
  static_assert(64 % L::CH == 0 && ROWS % (PER * NW) == 0, "whole copies");
  // the addresses are formed again at every call: held over a loop they would cost more than they save
  int lr = wave * PER + lane / L::CH;
  asm volatile("" : "+v"(lr));
#pragma unroll
  for (int i = 0; i < ROWS / (PER * NW); ++i) {
    const int r = i * NW * PER + lr;
    int g = row0 + r;
    g = g < last ? g : last - 1;
    lds_copy16(base + g * stride + ((lane % L::CH) ^ L::swz(r)) * L::EPC, lds_offset(tile + (i * NW + wave) * PER * D));
  }
}

// Waits for this wavefront's copies; behind the barrier every wavefront's are there.
__device__ __forceinline__ void copies_done() {
  copies_landed();
  lds_barrier();
}

}  // namespace kda
