// kda_cache.hpp -- what the kernels over the paged 8-bit cache share: scales, codes, pages.
#pragma once

#include "kda_mix_launch.hpp"
#include "kda_mma.hpp"

namespace kda {

constexpr float kE4m3Max = 448.f;
constexpr int kLeastExp = -100;  // of a scale: an all-zero page's

// The smallest power of two s with amax <= 448 s, from amax's fp32 pattern: amax = 1.f 2^(E - 127),
// 448 = 1.75 2^8.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int k = int(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = k < kLeastExp ? kLeastExp : k;
  return __uint_as_float(uint32_t(k + 127) << 23);
}

// x / s for s a power of two (its reciprocal is exact), infinities held as the largest value.
__device__ __forceinline__ float to_range(float x, float inv) {
  x *= inv;
  return x > kE4m3Max ? kE4m3Max : (x < -kE4m3Max ? -kE4m3Max : x);
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true));
}
// four codes rounded again at a scale 1 / f times theirs
__device__ __forceinline__ uint32_t recode4(uint32_t w, float f) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
  return encode4(a[0] * f, a[1] * f, b[0] * f, b[1] * f);
}

__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

__device__ __forceinline__ int page_shift(int page) { return page == 64 ? 6 : (page == 32 ? 5 : 4); }

// A page's new V codes, tokens off .. off + cnt - 1 of `image` ([d][P + 4] in LDS), into its rows of
// tokens, sixteen at a time where they are whole sixteens (most pages of a prompt; 14300 turned tokens of 8 heads of 128
// take 40 us so, 42 by words), else by words where those are whole; `grown`: the earlier codes are rounded again at a scale
// 1 / f times theirs.
template <int D, int NT = 256>
__device__ __forceinline__ void store_v_image(uint8_t* vc, const uint8_t* image, int P, int off, int cnt, bool grown, float f,
                                              int tid) {
  if (!grown && ((off | cnt) & 15) == 0) {
    for (int e = tid; e < D * (cnt / 16); e += NT) {
      const int d = e / (cnt / 16), t = off + 16 * (e % (cnt / 16));
      const uint32_t* im = reinterpret_cast<const uint32_t*>(image + d * (P + 4) + t);
      *reinterpret_cast<u32x4*>(vc + d * P + t) = u32x4{im[0], im[1], im[2], im[3]};
    }
    return;
  }
  const int t_lo = grown ? 0 : off / 4, t_hi = (off + cnt + 3) / 4, nd = t_hi - t_lo;  // words of a row
  for (int e = tid; e < D * nd; e += NT) {
    const int d = e / nd, t = 4 * (t_lo + e % nd);
    uint8_t* p = vc + d * P + t;
    const uint8_t* im = image + d * (P + 4) + t;
    if (t >= off && t + 4 <= off + cnt) {
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(im);
    } else if (t + 4 <= off) {
      *reinterpret_cast<uint32_t*>(p) = recode4(*reinterpret_cast<uint32_t*>(p), f);
    } else {
      for (int j = 0; j < 4; ++j) {
        if (t + j < off) {
          if (grown) p[j] = uint8_t(recode4(p[j], f));
        } else if (t + j < off + cnt) {
          p[j] = im[j];
        }
      }
    }
  }
}

// Rows of the new tokens in use: cu's last entry, within the buffer.
__device__ __forceinline__ int rows_in_use(const int* cu, int N, int n) {
  const int e = cu[N];
  return e < 0 ? 0 : (e > n ? n : e);
}

// Eight codes (two words) as a fragment, times a power of two.  Every e4m3 value is a bf16 value.
__device__ __forceinline__ bf16x8 codes(uint32_t a, uint32_t b, float scale = 1.0f) {
  const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false),
               q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true),
               r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false),
               s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
  return __builtin_shufflevector(__builtin_shufflevector(p, q, 0, 1, 2, 3), __builtin_shufflevector(r, s, 0, 1, 2, 3), 0, 1,
                                 2, 3, 4, 5, 6, 7);
}

// The maximum and sum over the four 16-lane groups.
__device__ __forceinline__ float max_groups(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_groups(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

}  // namespace kda
