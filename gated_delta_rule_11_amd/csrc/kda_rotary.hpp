// kda_rotary.hpp -- rotary positions, as the kernel that only rotates and the one that appends to
// the cache share them.
//
// Pair j of a row's channels turns by the angle pos[axis(j)] inv_freq[j]:
//   y_a = x_a cos t - x_b sin t,   y_b = x_b cos t + x_a sin t
// with (a, b) = (j, j + half) or, interleaved, (2 j, 2 j + 1).  The angle is formed and reduced in 64
// bits: a far position's angle has few fraction bits left in 32 (2^17 turns leave 2^-7 of a turn).  From a position of
// 2^29 on the product has more than 53 bits, and what its rounding loses (up to 2^-23) is kept beside it.
#pragma once

#include "kda_mix_launch.hpp"
#include "kda_mma.hpp"

namespace kda {

// The product of a place and a frequency, up to 55 bits: rounded, and what the rounding lost.
struct Angle {
  double a, rest;
};

// Sine and cosine: a = k pi/2 + r with |r| <= pi/4 (pi/2 in two parts, so that r keeps 53 bits after the
// point), then the Taylor sums, whose first terms left out are below 2^-49, and a quarter turn k mod 4.
// The vector unit runs 64-bit multiply-adds at the rate of 32-bit ones.
__device__ __forceinline__ void sine_cosine(const Angle& t, double& s, double& c) {
  const double k = __builtin_rint(t.a * 0.63661977236758134308);
  double r = __builtin_fma(-k, 1.57079632679489655800, t.a) + t.rest;
  r = __builtin_fma(-k, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double p = 1.0 / 1307674368000.0, q = 1.0 / 87178291200.0;
  p = __builtin_fma(-p, z, 1.0 / 6227020800.0);
  q = __builtin_fma(-q, z, 1.0 / 479001600.0);
  p = __builtin_fma(-p, z, 1.0 / 39916800.0);
  q = __builtin_fma(-q, z, 1.0 / 3628800.0);
  p = __builtin_fma(-p, z, 1.0 / 362880.0);
  q = __builtin_fma(-q, z, 1.0 / 40320.0);
  p = __builtin_fma(-p, z, 1.0 / 5040.0);
  q = __builtin_fma(-q, z, 1.0 / 720.0);
  p = __builtin_fma(-p, z, 1.0 / 120.0);
  q = __builtin_fma(-q, z, 1.0 / 24.0);
  p = __builtin_fma(-p, z, 1.0 / 6.0);
  q = __builtin_fma(-q, z, 0.5);
  const double sr = __builtin_fma(-p * z, r, r), cr = __builtin_fma(-q, z, 1.0);
  const int quarter = int(k - 4.0 * __builtin_rint(k * 0.25)) & 3;
  s = quarter & 1 ? cr : sr;
  c = quarter & 1 ? sr : cr;
  s = quarter & 2 ? -s : s;
  c = (quarter + 1) & 2 ? -c : c;
}

__device__ __forceinline__ Angle angle_of(const Rotation& t, int64_t row, int64_t place, int j) {
  double p = double(place);
  if (t.pos) {
    int x = 0;
    if (t.axis) {
      x = t.axis[j];
      x = x < 0 ? 0 : (x < t.axes ? x : t.axes - 1);
    }
    p = double(t.pos[row * t.axes + x]);
  }
  const double f = double(t.inv[j]), a = p * f;
  return {a, __builtin_fma(p, f, -a)};
}

// A row is handled in units of two chunks of eight channels: u below half / 8 holds chunks u and
// u + half / 8, which with halves are eight whole pairs; behind them come chunks that do not turn.
struct Unit {
  int c0, c1;
  bool turns;
};
__device__ __forceinline__ Unit unit_of(int u, int half) {
  const int m = half / 8;
  if (u < m) return {u, u + m, true};
  return {2 * u, 2 * u + 1, false};
}
// The pair that element e of a unit's eight sines stands for.
__device__ __forceinline__ int pair_of(int u, int e, int half, bool interleaved) {
  if (!interleaved) return 8 * u + e;
  return e < 4 ? 4 * u + e : half / 2 + 4 * u + e - 4;
}

__device__ __forceinline__ float mul_add(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double mul_add(double a, double b, double c) { return __builtin_fma(a, b, c); }

// A turned channel as fp32.  From 64 bits it is rounded to odd (cut, and the last bit set where that lost
// something): a later rounding to fewer bits then gives what it would give from the 64 bits.
__device__ __forceinline__ float to_fp32(float y) { return y; }
__device__ __forceinline__ float to_fp32(double y) {
  const uint64_t u = __builtin_bit_cast(uint64_t, y);
  uint32_t lo = uint32_t(u);
  lo = (lo & 0xe0000000u) | (lo & 0x1fffffffu ? 0x20000000u : 0u);
  return float(__builtin_bit_cast(double, (u & 0xffffffff00000000ull) | lo));
}

// x0 and x1 (a unit's chunks) turned.
template <typename V>
__device__ __forceinline__ void turn(f32x8& x0, f32x8& x1, const V* c, const V* s, bool interleaved) {
  f32x8 y0, y1;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const V a0 = x0[2 * i], b0 = x0[2 * i + 1], a1 = x1[2 * i], b1 = x1[2 * i + 1];
      y0[2 * i] = to_fp32(mul_add(a0, c[i], -b0 * s[i]));
      y0[2 * i + 1] = to_fp32(mul_add(b0, c[i], a0 * s[i]));
      y1[2 * i] = to_fp32(mul_add(a1, c[4 + i], -b1 * s[4 + i]));
      y1[2 * i + 1] = to_fp32(mul_add(b1, c[4 + i], a1 * s[4 + i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const V a = x0[i], b = x1[i];
      y0[i] = to_fp32(mul_add(a, c[i], -b * s[i]));
      y1[i] = to_fp32(mul_add(b, c[i], a * s[i]));
    }
  }
  x0 = y0;
  x1 = y1;
}

// The last sequence that starts at or before `row` of all wavefronts' lanes alike, 64 candidates at a time.
__device__ __forceinline__ int sequence_of(const int* cu, int N, int64_t row, int lane) {
  int lo = 0, up = N;
  while (up - lo > 1) {
    const int step = (up - lo + 63) / 64;
    const int64_t mid = lo + int64_t(step) * (lane + 1);
    lo += step * __popcll(__ballot(mid < up && cu[mid] <= row));
    up = lo + step < up ? lo + step : up;
  }
  return lo;
}

// Heads h0 .. h0 + heads - 1 of rows row0 .. row0 + rows - 1 turned by one wavefront, `side` heads at a time; `sc` is
// its own LDS.  (`place` is for one row.)
constexpr int kSines = 512;  // of a wavefront: rows * half, at most 64 / (d / 16) * d / 2
template <typename T, typename TO>
__device__ __forceinline__ void rotate_rows(const RopeArgs& a, int64_t row0, int64_t place, int h0, float (*sc)[kSines], int lane) {
  const int half = a.turn.half, units = a.d / 16;
  const bool inter = a.turn.interleaved;
  for (int j = lane; j < a.rows * half; j += 64) {
    const int64_t row = row0 + j / half;
    double s = 0.0, c = 1.0;
    if (row < a.n) sine_cosine(angle_of(a.turn, row, place, j % half), s, c);
    sc[0][j] = float(c);
    sc[1][j] = float(a.inverse ? -s : s);
  }
  __builtin_amdgcn_wave_barrier();
  const int u = lane % units, g = lane / units, r = g / a.side;
  const int64_t row = row0 + r;
  if (r >= a.rows || row >= a.n) return;
  const Unit w = unit_of(u, half);
  float c[8], s[8];
  if (w.turns)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = sc[0][r * half + pair_of(u, e, half, inter)];
      s[e] = sc[1][r * half + pair_of(u, e, half, inter)];
    }
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  TO* y = static_cast<TO*>(a.y) + row * a.y_stride;
  const int end = h0 + a.heads < a.H ? h0 + a.heads : a.H;
#pragma unroll 4
  for (int h = h0 + g % a.side; h < end; h += a.side) {
    f32x8 x0 = Op<T>::unpack(Op<T>::load(x + int64_t(h) * a.d + 8 * w.c0));
    f32x8 x1 = Op<T>::unpack(Op<T>::load(x + int64_t(h) * a.d + 8 * w.c1));
    if (w.turns) turn(x0, x1, c, s, inter);
    store8(y + int64_t(h) * a.d + 8 * w.c0, x0);
    store8(y + int64_t(h) * a.d + 8 * w.c1, x1);
  }
}

}  // namespace kda
