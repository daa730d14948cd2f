// kda_mma.hpp -- matrix-core operands shared by the linear-attention, prompt-attention
// and cache-attention kernels, for bf16 and fp32 elements alike.
//
// A fragment is the eight k-elements one lane feeds a product with: lane l holds row
// (A) or column (B) l % 32 and k = 8 (l / 32) .. + 7 of a 32x32x16 product, or l % 16
// and k = 8 (l / 16) .. + 7 of a 16x16x32 product.  With bf16 that is one
// v_mfma_f32_32x32x16_bf16 (16x16x32); with fp32 the same fragment feeds eight
// v_mfma_f32_32x32x2_f32 (16x16x4), product j taking element j of every lane, so both
// element types share one data layout.  A product's k order does not matter as long as A
// and B agree on it.  Results (fp32): lane l holds column l % 32, rows
// 8 (i / 4) + 4 (l / 32) + i % 4 in register i (32x32), or column l % 16, rows
// 4 (l / 16) + i (16x16).  Hence a result's registers 8 s .. 8 s + 7 are again a fragment:
// k-step s of a product over its rows, element j standing for row
// 16 s + 4 (l / 32) + j (j < 4) or 16 s + 8 + 4 (l / 32) + j - 4 (`perm` below).
#pragma once

#include "kda_common.hpp"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

// Row of a 32x32 result held by register i in lane half h.
__device__ __forceinline__ constexpr int crow(int i, int h) { return 8 * (i / 4) + 4 * h + i % 4; }

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

template <typename T> struct Op;

template <> struct Op<bf16_t> {
  typedef bf16x8 frag;
  __device__ __forceinline__ static frag load(const bf16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }
  __device__ __forceinline__ static frag join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  // round to nearest even (v_cvt_pk_bf16_f32)
  __device__ __forceinline__ static frag pack(const f32x8 f) { return __builtin_convertvector(f, bf16x8); }
  __device__ __forceinline__ static f32x8 unpack(const frag a) { return __builtin_convertvector(a, f32x8); }
  __device__ __forceinline__ static frag neg(const frag a) { return -a; }
  __device__ __forceinline__ static f32x16 mma32(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  __device__ __forceinline__ static f32x4 mma16(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

template <> struct Op<float> {
  typedef f32x8 frag;
  __device__ __forceinline__ static frag load(const float* p) {
    return join(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4));
  }
  __device__ __forceinline__ static frag join(f32x4 a, f32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ __forceinline__ static frag pack(const f32x8 f) { return f; }
  __device__ __forceinline__ static f32x8 unpack(const frag a) { return a; }
  __device__ __forceinline__ static frag neg(const frag a) { return -a; }
  __device__ __forceinline__ static f32x16 mma32(frag a, frag b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  __device__ __forceinline__ static f32x4 mma16(frag a, frag b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
};

// Non-finite elements of fragments: 16 (32) bit lanes that reach zero where an exponent is all
// ones, over any number of fragments, and a fragment with those elements set to zero.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <typename T> struct Finite;
template <> struct Finite<bf16_t> {
  u16x2 low = {0xffff, 0xffff};
  __device__ __forceinline__ void see(bf16x8 a) {
    const u32x4 w = __builtin_bit_cast(u32x4, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) low = __builtin_elementwise_min(low, __builtin_bit_cast(u16x2, ~w[i] & 0x7f807f80u));
  }
  __device__ __forceinline__ bool all() const { return low[0] != 0 && low[1] != 0; }
  __device__ __forceinline__ static bf16x8 only(bf16x8 a) {
    u32x4 w = __builtin_bit_cast(u32x4, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u16x2 e = __builtin_elementwise_min(__builtin_bit_cast(u16x2, ~w[i] & 0x7f807f80u), u16x2{1, 1});
      w[i] &= __builtin_bit_cast(uint32_t, u16x2{0, 0} - e);
    }
    return __builtin_bit_cast(bf16x8, w);
  }
};
template <> struct Finite<float> {
  uint32_t low = 0xffffffffu;
  __device__ __forceinline__ void see(f32x8 a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = ~__float_as_uint(a[i]) & 0x7f800000u;
      low = x < low ? x : low;
    }
  }
  __device__ __forceinline__ bool all() const { return low != 0; }
  __device__ __forceinline__ static f32x8 only(f32x8 a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (~__float_as_uint(a[i]) & 0x7f800000u) == 0 ? 0.f : a[i];
    return a;
  }
};

// Two fp32 values' upper halves as a pair of bf16.
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// x as parts of the element type: one, rounded, or three bf16 whose sum is x (each takes the upper
// half of what is left, 8 bits of significand at a time, and the rest is exact).
template <typename T, int N, int W>
struct Parts {
  typedef uint32_t words __attribute__((ext_vector_type(W / 2)));
  words p[N];
  template <typename V>
  __device__ __forceinline__ explicit Parts(V x) {
    static_assert(N == 3 && sizeof(T) == 2, "the exact form");
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < W; j += 2) {
        p[i][j / 2] = upper_halves(x[j], x[j + 1]);
        if (i + 1 < N) {
          x[j] -= __uint_as_float(__float_as_uint(x[j]) & 0xffff0000u);
          x[j + 1] -= __uint_as_float(__float_as_uint(x[j + 1]) & 0xffff0000u);
        }
      }
  }
};
template <typename T>
struct Parts<T, 1, 8> {
  typename Op<T>::frag p[1];
  __device__ __forceinline__ explicit Parts(f32x8 x) { p[0] = Op<T>::pack(x); }
};
template <typename T, int N>
__device__ __forceinline__ typename Op<T>::frag part_of(const Parts<T, N, 8>& x, int i) {
  return __builtin_bit_cast(typename Op<T>::frag, x.p[i]);
}

// Registers 8 s .. 8 s + 7 of a result as a fragment.
template <typename T>
__device__ __forceinline__ typename Op<T>::frag frag_of(const f32x16& c, int s) {
  f32x8 f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = c[8 * s + j];
  return Op<T>::pack(f);
}

// A tile of rows of COLS elements in LDS, aligned to its rows.  Each row's 16-byte chunks are
// permuted by the row's number, so that reads of one chunk from 8 or 16 consecutive rows, and
// transposing reads of 4 rows by 16 columns, spread over the banks.
//
// The permutation is an exclusive or, and so are the steps from one fragment of a lane to the next:
// a lane keeps one byte offset per kind of read (the b_* functions), and a fragment's address is
// that, plus the tile's, xor a constant, plus a constant that fits the instruction.  (Written
// as offsets of (row, column) the compiler kept an address register for every fragment.)
template <typename T, int COLS>
struct Tile {
  static constexpr int EPC = 16 / int(sizeof(T));   // elements of a chunk
  static constexpr int CH = COLS / EPC;             // chunks of a row
  static constexpr int ROWB = COLS * int(sizeof(T));  // bytes of a row
  static constexpr bool B16 = sizeof(T) == 2;
  static_assert(COLS % EPC == 0 && (CH & (CH - 1)) == 0 && CH >= 4, "rows of a power of two of chunks");
  typedef typename Op<T>::frag F;
  // The permutation, linear over the row's bits, from the LDS' 64 banks and the lanes that it serves
  // together (16 of a 16-byte read: 0-3, 12-15, 20-23 and 24-27, and those + 4, + 32, + 36; 32 of an
  // 8-byte one): with these images of bits 0 .. 3 every kind of read below is free of conflicts.
  // Rows of 64 (128) bytes share 256 bytes of banks with three (one) neighbours, which stands in for
  // the images of bits 0 and 1 (0).  Measured per read of a wavefront: 4 and 2 cycles, the width's own.
  __device__ __forceinline__ static constexpr int swz(int row) {
    return (CH >= 16 ? (row << 2) & 12 : (CH == 8 ? (row << 1) & 4 : 0)) ^ ((row >> 2) & 1) * 3 ^ ((row >> 3) & 1) * 2;
  }
  // element offset of (row, col); `col` a multiple of 4 keeps 4 elements together
  __device__ __forceinline__ static int off(int row, int col) {
    return row * COLS + (((col / EPC) ^ swz(row)) * EPC) + col % EPC;
  }
  template <typename V>
  __device__ __forceinline__ static V rd(uint32_t a) {
    return *(const __attribute__((address_space(3))) V*)(uintptr_t)a;
  }
  __device__ __forceinline__ static uint32_t at(const T* t) {
    return uint32_t(uintptr_t(t));  // the low half of a generic pointer into LDS is the LDS offset
  }
  __device__ __forceinline__ static bf16x4 tr(uint32_t a) {
    typedef s16x4 __attribute__((address_space(3)))* lds_ptr;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uintptr_t)a));
  }

  // 32x32: row 32 j + lane % 32, columns 16 kk + 8 (lane / 32) .. + 7
  __device__ __forceinline__ static uint32_t b_row8_32(int lane) {
    const int r = lane & 31, h = lane >> 5;
    return r * ROWB + (((B16 ? h : 2 * h) ^ swz(r)) << 4);
  }
  __device__ __forceinline__ static F row8_32(uint32_t b, int j, int kk) {
    if constexpr (B16) {
      return rd<bf16x8>((b ^ (kk << 5)) + 32 * j * ROWB);
    } else {
      return Op<T>::join(rd<f32x4>((b ^ (kk << 6)) + 32 * j * ROWB), rd<f32x4>((b ^ ((kk << 6) | 16)) + 32 * j * ROWB));
    }
  }
  // 32x32, summing over rows in a result's order: rows r0 + 4 (lane / 32) .. + 3 and those + 8
  // (r0 a multiple of 16), column 32 i + lane % 32.  With bf16 by two transposing reads
  // (ds_read_b64_tr_b16): 16 lanes fetch 4 rows of 16 columns, 4 columns each, and lane i of
  // them receives column i.
  __device__ __forceinline__ static uint32_t b_col44_32(int lane) {
    const int h = lane >> 5;
    if constexpr (B16) {
      const int r = 4 * h + ((lane & 15) >> 2), c = (lane & 16) + 4 * (lane & 3);
      return r * ROWB + (((c >> 3) ^ swz(r)) << 4) + 2 * (c & 7);
    } else {
      const int c = lane & 31;
      return 4 * h * ROWB + (((c >> 2) ^ swz(4 * h)) << 4) + 4 * (c & 3);
    }
  }
  __device__ __forceinline__ static F col44_32(uint32_t b, int r0, int i) {
    if constexpr (B16) {
      return Op<T>::join(tr((b ^ (i << 6)) + r0 * ROWB), tr((b ^ ((i << 6) ^ (swz(8) << 4))) + (r0 + 8) * ROWB));
    } else {
      F f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = (j & 3) + 8 * (j >> 2);
        f[j] = rd<float>((b ^ ((i << 7) ^ (swz(x) << 4))) + (r0 + x) * ROWB);
      }
      return f;
    }
  }

  // 16x16: row 16 t + lane % 16, columns 32 kk + 8 (lane / 16) .. + 7
  __device__ __forceinline__ static uint32_t b_row8_16(int lane) {
    const int r = lane & 15, g = lane >> 4;
    return r * ROWB + (((B16 ? g : 2 * g) ^ swz(r)) << 4);
  }
  __device__ __forceinline__ static F row8_16(uint32_t b, int t, int kk) {
    if constexpr (B16) {
      return rd<bf16x8>((b ^ (kk << 6)) + 16 * t * ROWB);
    } else {
      return Op<T>::join(rd<f32x4>((b ^ (kk << 7)) + 16 * t * ROWB), rd<f32x4>((b ^ ((kk << 7) | 16)) + 16 * t * ROWB));
    }
  }
  // 16x16, the columns in the order of two results' rows: 32 kk + 4 (lane / 16) .. + 3 and those + 16
  __device__ __forceinline__ static uint32_t b_row44_16(int lane) {
    const int r = lane & 15, g = lane >> 4;
    return r * ROWB + (B16 ? ((((g >> 1) ^ swz(r)) << 4) + 8 * (g & 1)) : ((g ^ swz(r)) << 4));
  }
  // (volatile: merged into strided pairs, the two halves would have to be moved next to each other)
  __device__ __forceinline__ static F row44_16(uint32_t b, int t, int kk) {
    if constexpr (B16) {
      typedef const volatile __attribute__((address_space(3))) bf16x4* half;
      return Op<T>::join(*(half)(uintptr_t)((b ^ (kk << 6)) + 16 * t * ROWB), *(half)(uintptr_t)((b ^ ((kk << 6) | 32)) + 16 * t * ROWB));
    } else {
      return Op<T>::join(rd<f32x4>((b ^ (kk << 7)) + 16 * t * ROWB), rd<f32x4>((b ^ ((kk << 7) | 64)) + 16 * t * ROWB));
    }
  }
  // 16x16, summing over rows: rows 32 u + 8 (lane / 16) .. + 7, column 16 t + lane % 16
  __device__ __forceinline__ static uint32_t b_col8_16(int lane) {
    const int g = lane >> 4;
    if constexpr (B16) {
      const int r = 8 * g + ((lane & 15) >> 2), c = 4 * (lane & 3);
      return r * ROWB + (((c >> 3) ^ swz(r)) << 4) + 2 * (c & 7);
    } else {
      const int c = lane & 15;
      return 8 * g * ROWB + (((c >> 2) ^ swz(8 * g)) << 4) + 4 * (c & 3);
    }
  }
  __device__ __forceinline__ static F col8_16(uint32_t b, int u, int t) {
    if constexpr (B16) {
      return Op<T>::join(tr((b ^ (t << 5)) + 32 * u * ROWB), tr((b ^ ((t << 5) ^ (swz(4) << 4))) + (32 * u + 4) * ROWB));
    } else {
      F f;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = rd<float>((b ^ ((t << 6) ^ (swz(j) << 4))) + (32 * u + j) * ROWB);
      return f;
    }
  }

  // four consecutive columns of a row as fp32
  __device__ __forceinline__ static f32x4 get4(const T* t, int row, int col) {
    if constexpr (B16) return __builtin_convertvector(*reinterpret_cast<const bf16x4*>(t + off(row, col)), f32x4);
    else return *reinterpret_cast<const f32x4*>(t + off(row, col));
  }
  __device__ __forceinline__ static void put4(T* t, int row, int col, f32x4 x) {
    if constexpr (B16) *reinterpret_cast<bf16x4*>(t + off(row, col)) = __builtin_convertvector(x, bf16x4);
    else *reinterpret_cast<f32x4*>(t + off(row, col)) = x;
  }
};

// Four consecutive elements to global memory, rounded to the output type.
template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 x) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(x, bf16x4);
  else
    *reinterpret_cast<f32x4*>(p) = x;
}

// The sum and maximum of a value and the other half-wavefront's (lane ^ 32).
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Dispatch of workgroups to consecutive work items per XCD: the hardware deals workgroups to
// the eight XCDs in turn; the returned index gives each XCD one contiguous run of items, so that
// neighbours share an L2.
__device__ __forceinline__ int xcd_order(int id, int n) {
  const int x = id & 7, per = n >> 3, rem = n & 7;
  return x * per + (x < rem ? x : rem) + (id >> 3);
}

// The item of a launch of `n` tiles for each of `heads` heads: tiles in the outer order, so that
// the longest, given first, start first on every XCD; where the heads divide by eight, each XCD
// keeps to its own consecutive heads.
struct HeadTile {
  int head, tile;
};
__device__ __forceinline__ HeadTile head_tile(int id, int heads) {
  const int h = id % heads;
  return {(heads & 7) == 0 ? (h & 7) * (heads >> 3) + (h >> 3) : h, id / heads};
}

// Copies from memory straight into LDS, 16 (4) bytes a lane: the wavefront's lanes land behind one
// another at `lds`, whatever their source addresses (inactive lanes write nothing).  Written as
// assembly without outputs, since the compiler, which cannot tell which LDS reads such a copy may
// meet, would wait for it before the next one; copies_landed() is the wait that they need.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return uint32_t(uintptr_t(p));  // the low half of a generic pointer into LDS
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_copy4(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
               : "memory", "m0");
}
// The same from one base for the wavefront plus 32 bits of byte offset per lane.
__device__ __forceinline__ void lds_copy16(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(offset), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_copy4(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :
               : "s"(lds), "v"(offset), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop
template <int LATER = 0>  // all but the last LATER copies of this wavefront
__device__ __forceinline__ void copies_landed() {
  static_assert(LATER < 64, "the counter's range");
  // the builtin, so that the compiler knows that its own earlier loads are there too and does not
  // wait for them, and the copies with them, inside the loop
  __builtin_amdgcn_s_waitcnt((LATER & 15) | (LATER >> 4) << 14 | 0x0f70);
  asm volatile("" ::: "memory");
}
// A barrier for LDS contents: waits for this wavefront's LDS accesses, not for its stores to memory.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The sum over lanes 0 .. l in lane l, in 64 bits, by lane shifts within the register file (rows of
// 16 lanes, then the rows' last lanes broadcast).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_shifted(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(u)), CTRL, ROWS, 15, false));
  const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(u >> 32)), CTRL, ROWS, 15, false));
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ double wave_prefix(double x) {
  x += dpp_shifted<0x111, 15>(x);  // row_shr by 1, 2, 4, 8
  x += dpp_shifted<0x112, 15>(x);
  x += dpp_shifted<0x114, 15>(x);
  x += dpp_shifted<0x118, 15>(x);
  x += dpp_shifted<0x142, 10>(x);  // row_bcast:15 into rows 1 and 3
  x += dpp_shifted<0x143, 12>(x);  // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(u), lane), hi = __builtin_amdgcn_readlane(uint32_t(u >> 32), lane);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

}  // namespace kda
