// kda_checks.hpp -- host-side argument checks shared by the entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/kda.h"

namespace kda {

constexpr int64_t kMaxElems = int64_t(1) << 62;

inline bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool dtype_ok(int t) { return t == KDA_F32 || t == KDA_BF16; }
inline size_t esize(int t) { return t == KDA_BF16 ? 2 : 4; }

struct Range {
  const void* p;
  int64_t bytes;
};

// True when two non-empty byte ranges overlap.
inline bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

// Checks B, T, H, dk, dv and returns false when a size is out of range (negative
// B or T; H, dk or dv below 1) or any product overflows the supported index range.
// The head dims are checked here, before the products below divide by them.  T is
// kept 64 below INT_MAX so that token offsets rounded up to a whole chunk (T + 63,
// a chunk start + 64) stay within 32 bits in the kernels.
constexpr int64_t kMaxT = 0x7fffffffLL - 64;
inline bool sizes_ok(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv) {
  if (B < 0 || T < 0 || H < 1 || dk < 1 || dv < 1 || T > kMaxT) return false;
  if (B * H > 0x7fffffffLL) return false;
  if (H * dk > 0x7fffffffLL || H * dv > 0x7fffffffLL) return false;
  if (B > 0 && T > 0 && B * T > kMaxElems / (H * (dk > dv ? dk : dv))) return false;
  if (B * H > kMaxElems / (dk * dv)) return false;
  return true;
}

inline kda_status from_hip(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Tensor bases 16-byte aligned, beta to its element size (NULL passes).
inline bool all_aligned(std::initializer_list<const void*> vec16, const void* beta, size_t beta_size) {
  for (const void* p : vec16)
    if (!aligned(p, 16)) return false;
  return aligned(beta, beta_size);
}

// A launch holds fewer than 2^32 threads.  In workgroups of 256, which all kernels of the mixers have but
// the linear walks (linear_threads; see walk_grid_ok):
constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

// ---- prompts and cache ------------------------------------------------------------------

inline bool attn_dim_ok(int d) { return d == 64 || d == 128; }
inline bool page_ok(int p) { return p == 16 || p == 32 || p == 64; }

// n rows (or N sequences) of Hq heads in groups over Hkv, d wide.
inline kda_status heads_ok(int64_t n, int64_t Hq, int64_t Hkv, int64_t d) {
  // the last tile of rows ends within 32 bits
  if (!sizes_ok(n, 1, Hq, d, d) || Hkv < 1 || n > 0x7fffffffLL - 256) return KDA_ERR_SHAPE;
  if (!attn_dim_ok(int(d)) || Hq % Hkv != 0) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace kda
