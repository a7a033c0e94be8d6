// mp_units.cuh — eight columns a lane of rows at any alignment, and rows in 8
// bits (e4m3 values with scales), for the operators of a block between its
// matrix products.
//
// A run of `run` neighbouring lanes (a warp; of wide rows also half or a quarter of
// one) takes 8 * run neighbouring columns of a row from `base` on; lane l of the
// run has eight of them, in slots 0 to 7:
//  Wide rows (on the 16-byte grid): columns base + 8 l to base + 8 l + 7, one
//    16-byte access (two for fp32). Four lanes share a scale of 32 columns.
//  Other rows, 16-bit: pairs of columns, pair i at base + 64 i + 2 l, so that a
//    warp's lanes touch neighbouring 4-byte words whatever the row's place; only
//    on an odd one is a pair two accesses. 16 lanes share a scale.
//  Other rows, fp32: slot i is column base + 32 i + l. A warp shares a scale.
// (Cutting eight neighbours out of the two or three 16-byte pieces that they lie in,
// and handing pieces to the neighbour for the stores, takes more instructions than
// these narrow accesses: gated forward of 32768 x 2731, fp32 229 us so and 151 this way.)
#pragma once

#include "mp_block.h"
#include "mp_rows.cuh"

namespace mpk {

constexpr int64_t kMaxUnitD = int64_t{1} << 24;

inline bool unit_shape_ok(int64_t rows, int64_t d) { return rows_ok(rows) && d >= 1 && d <= kMaxUnitD; }
inline bool scale8_ok(int32_t kind) { return kind == MP_SCALE_ROW || kind == MP_SCALE_BLOCK; }
inline bool scale8_aligned(const void* p, int32_t kind) { return kind != MP_SCALE_ROW || aligned4(p); }

// Whether 8-bit rows can be read and written as 8-B units.
inline bool wide_rows8(const void* p, int64_t length, int64_t stride, int64_t rows) {
  return aligned_to(p, 8) && length % 8 == 0 && (rows <= 1 || stride % 8 == 0);
}

// An output that is an input has to be the same matrix.
inline bool alias_ok(const void* out, int64_t out_stride, const void* in, int64_t in_stride) {
  return !out || out != in || out_stride == in_stride;
}

// ---- eight floats -----------------------------------------------------------------
// Four pairs for the two-wide fp32 instructions: each lane's result is that of the
// scalar instruction, for half the issue slots, which is what bounds these
// kernels next to HBM (packing 16384 x 4096 bf16: 41 us at 83 % of the issue slots with
// scalar arithmetic).
struct F8 {
  float2 p[4];
};

__device__ __forceinline__ uint64_t as_u64(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 as_f2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

__device__ __forceinline__ F8 mul8(const F8& a, const F8& b) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = mul2(a.p[i], b.p[i]);
  return r;
}
__device__ __forceinline__ F8 mul8(const F8& a, float b) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = mul2(a.p[i], both(b));
  return r;
}
__device__ __forceinline__ F8 add8(const F8& a, const F8& b) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = add2(a.p[i], b.p[i]);
  return r;
}
__device__ __forceinline__ F8 zero8() {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = make_float2(0.0f, 0.0f);
  return r;
}

template <int T>
__device__ __forceinline__ F8 get8(const Pack8<T>& u) {
  float f[8];
  u.get(f);
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = make_float2(f[2 * i], f[2 * i + 1]);
  return r;
}
template <int T>
__device__ __forceinline__ void put8(Pack8<T>& u, const F8& a) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = a.p[i].x;
    f[2 * i + 1] = a.p[i].y;
  }
  u.put(f);
}

// Sums rounded to the type. Of 16-bit types in one instruction a pair, whose single
// rounding is that of the fp32 sum's: two of them whose sum lies on both sides of
// a midpoint are less than 16 bits apart, and such a sum is exact in fp32.
template <int T>
__device__ __forceinline__ Pack8<T> sum_of(const Pack8<T>& a, const Pack8<T>& b) {
  Pack8<T> r;
  if constexpr (T == MP_FP32) {
    put8(r, add8(get8(a), get8(b)));
  } else {
    const uint32_t x[4] = {a.v.x, a.v.y, a.v.z, a.v.w}, y[4] = {b.v.x, b.v.y, b.v.z, b.v.w};
    uint32_t z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (T == MP_BF16)
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(z[i]) : "r"(x[i]), "r"(y[i]));
      else
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(z[i]) : "r"(x[i]), "r"(y[i]));
    }
    r.v = make_uint4(z[0], z[1], z[2], z[3]);
  }
  return r;
}

// The largest of m and the magnitudes of a, NaN if one is NaN.
__device__ __forceinline__ float amax2(float m, float2 a) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float amax8(float m, const F8& a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = amax2(m, a.p[i]);
  return m;
}

// ---- units ----------------------------------------------------------------------

// The column of slot i.
template <int T, bool Wide>
__device__ __forceinline__ int slot_column(int base, int l, int i) {
  if (Wide) return base + 8 * l + i;
  return T == MP_FP32 ? base + 32 * i + l : base + 64 * (i / 2) + 2 * l + i % 2;
}

// A lane's columns of a row of n as they come in, zeros from n on; unit() puts them
// together, so that a wait for the loads comes there and not between them.
template <int T, bool Wide>
struct Raw {  // 16-bit, not wide
  uint32_t a[4], b[4];  // a pair, or its first and second column

  __device__ __forceinline__ void load(const uint16_t* row, int base, int l, int n) {
    const uint16_t* p = row + base + 2 * l;
    const bool even = reinterpret_cast<uintptr_t>(row) % 4 == 0;
    if (base + 256 <= n) {
      if (even) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = *reinterpret_cast<const uint32_t*>(p + 64 * i);
          b[i] = 0u;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = p[64 * i];
          b[i] = p[64 * i + 1];
        }
      }
    } else {
      const int left = n - base - 2 * l;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = 64 * i < left ? p[64 * i] : 0u;
        b[i] = 64 * i + 1 < left ? p[64 * i + 1] : 0u;
      }
    }
  }
  __device__ __forceinline__ Pack8<T> unit() const {
    Pack8<T> u;
    u.v = make_uint4(a[0] | b[0] << 16, a[1] | b[1] << 16, a[2] | b[2] << 16, a[3] | b[3] << 16);
    return u;
  }
};

template <>
struct Raw<MP_FP32, false> {
  float f[8];

  __device__ __forceinline__ void load(const float* row, int base, int l, int n) {
    const float* p = row + base + l;
    if (base + 256 <= n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = p[32 * i];
    } else {
      const int left = n - base - l;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 32 * i < left ? p[32 * i] : 0.0f;
    }
  }
  __device__ __forceinline__ Pack8<MP_FP32> unit() const {
    Pack8<MP_FP32> u;
    u.put(f);
    return u;
  }
};

template <int T>
struct Raw<T, true> {
  Pack8<T> u;

  __device__ __forceinline__ void load(const typename Elem<T>::type* row, int base, int l, int n) {
    const int c = base + 8 * l;
    if (c < n)
      u.load(row + c);
    else
      u.zero();
  }
  __device__ __forceinline__ Pack8<T> unit() const { return u; }
};

template <>
struct Raw<MP_FP32, true> {
  Pack8<MP_FP32> u;

  __device__ __forceinline__ void load(const float* row, int base, int l, int n) {
    const int c = base + 8 * l;
    if (c < n)
      u.load(row + c);
    else
      u.zero();
  }
  __device__ __forceinline__ Pack8<MP_FP32> unit() const { return u; }
};

template <int T, bool Wide>
__device__ __forceinline__ void store_unit(const Pack8<T>& u, typename Elem<T>::type* row, int base, int l, int n) {
  if constexpr (Wide) {
    const int c = base + 8 * l;
    if (c < n) u.store(row + c);
  } else if constexpr (T == MP_FP32) {
    float* p = row + base + l;
    float f[8];
    u.get(f);
    if (base + 256 <= n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[32 * i] = f[i];
    } else {
      const int left = n - base - l;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (32 * i < left) p[32 * i] = f[i];
    }
  } else {
    uint16_t* p = row + base + 2 * l;
    const uint32_t w[4] = {u.v.x, u.v.y, u.v.z, u.v.w};
    if (base + 256 <= n && reinterpret_cast<uintptr_t>(row) % 4 == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(p + 64 * i) = w[i];
    } else {
      const int left = n - base - 2 * l;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (64 * i < left) p[64 * i] = static_cast<uint16_t>(w[i]);
        if (64 * i + 1 < left) p[64 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
      }
    }
  }
}

// The same of bytes, in the slots that elements of type T have.
template <int T, bool Wide>
struct Raw8 {  // 16-bit, not wide
  uint32_t a[4], b[4];

  __device__ __forceinline__ void load(const uint8_t* row, int base, int l, int n) {
    const uint8_t* p = row + base + 2 * l;
    const bool even = reinterpret_cast<uintptr_t>(row) % 2 == 0;
    if (base + 256 <= n) {
      if (even) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = *reinterpret_cast<const uint16_t*>(p + 64 * i);
          b[i] = 0u;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = p[64 * i];
          b[i] = p[64 * i + 1];
        }
      }
    } else {
      const int left = n - base - 2 * l;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = 64 * i < left ? p[64 * i] : 0u;
        b[i] = 64 * i + 1 < left ? p[64 * i + 1] : 0u;
      }
    }
  }
  __device__ __forceinline__ uint2 unit() const {
    return make_uint2(a[0] | b[0] << 8 | a[1] << 16 | b[1] << 24, a[2] | b[2] << 8 | a[3] << 16 | b[3] << 24);
  }
};

template <>
struct Raw8<MP_FP32, false> {
  uint32_t b[8];

  __device__ __forceinline__ void load(const uint8_t* row, int base, int l, int n) {
    const uint8_t* p = row + base + l;
    const int left = n - base - l;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 32 * i < left ? p[32 * i] : 0u;
  }
  __device__ __forceinline__ uint2 unit() const {
    return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
  }
};

struct Raw8Wide {
  uint2 q;

  __device__ __forceinline__ void load(const uint8_t* row, int base, int l, int n) {
    const int c = base + 8 * l;
    q = c < n ? *reinterpret_cast<const uint2*>(row + c) : make_uint2(0u, 0u);
  }
  __device__ __forceinline__ uint2 unit() const { return q; }
};

template <int T>
struct Raw8<T, true> : Raw8Wide {};
template <>
struct Raw8<MP_FP32, true> : Raw8Wide {};

template <int T, bool Wide>
__device__ __forceinline__ void store_unit8(uint2 q, uint8_t* row, int base, int l, int n) {
  if constexpr (Wide) {
    const int c = base + 8 * l;
    if (c < n) *reinterpret_cast<uint2*>(row + c) = q;
  } else if constexpr (T == MP_FP32) {
    uint8_t* p = row + base + l;
    const int left = n - base - l;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < left) p[32 * i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i % 4)));
  } else {
    uint8_t* p = row + base + 2 * l;
    const uint32_t w[4] = {q.x, q.x >> 16, q.y, q.y >> 16};
    if (base + 256 <= n && reinterpret_cast<uintptr_t>(row) % 2 == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint16_t*>(p + 64 * i) = static_cast<uint16_t>(w[i]);
    } else {
      const int left = n - base - 2 * l;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (64 * i < left) p[64 * i] = static_cast<uint8_t>(w[i]);
        if (64 * i + 1 < left) p[64 * i + 1] = static_cast<uint8_t>(w[i] >> 8);
      }
    }
  }
}

// ---- rows staged through shared memory ---------------------------------------------
// The TMA engine copies the whole 16-byte pieces that a row lies in (bytes of
// its neighbours that share one come along and are not used), so that loads stay
// in flight without registers or resident warps to hold them.
struct Pieces {
  const void* src;
  uint32_t bytes;
  uint32_t offset;  // of the row in them

  __device__ __forceinline__ Pieces(const void* row, uint32_t length) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row);
    offset = at % 16;
    src = reinterpret_cast<const void*>(at - offset);
    bytes = (offset + length + 15u) / 16u * 16u;
  }
};

// Bytes of the buffer of a row of `length` bytes at any place.
inline uint32_t pieces_pitch(int64_t length) { return static_cast<uint32_t>((length + 30) / 16 * 16); }

// ---- e4m3 -----------------------------------------------------------------------

// Nearest e4m3 values (ties to even), magnitudes above 448 as 448, NaN as NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 e4m3_pack(const F8& a) {
  return make_uint2(e4m3_pair(a.p[0].x, a.p[0].y) | (e4m3_pair(a.p[1].x, a.p[1].y) << 16),
                    e4m3_pair(a.p[2].x, a.p[2].y) | (e4m3_pair(a.p[3].x, a.p[3].y) << 16));
}

__device__ __forceinline__ F8 e4m3_unpack(uint2 q) {
  const uint32_t w[2] = {q.x, q.y};
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
    r.p[i] = __half22float2(*reinterpret_cast<const __half2*>(&h));
  }
  return r;
}

// ---- scales of 32 columns --------------------------------------------------------

constexpr uint32_t kScaleNan = 255u;

// The byte of the least power of two s >= 2^-127 with amax <= 448 s: with amax =
// m 2^k, 1 <= m < 2, and 448 = 1.75 * 2^8, that is 2^(k - 8) for m <= 1.75 and
// 2^(k - 7) above.
__device__ __forceinline__ uint32_t block_scale(float amax) {
  if (!(amax < kInf)) return kScaleNan;
  const int b = static_cast<int>((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(max(b, 0));
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float block_scale_value(uint32_t byte) {
  return byte == kScaleNan ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Slots whose columns share a scale: all eight, a pair, one.
template <int T, bool Wide>
constexpr int kShare = Wide ? 8 : T == MP_FP32 ? 1 : 2;

// The inverse of a scale, itself a power of two, so that products with it are exact.
__device__ __forceinline__ float block_inverse(uint32_t byte) {
  return __uint_as_float(byte == kScaleNan ? 0x7FC00000u : (254u - byte) << 23);
}

// Where the block's scale is that of the largest exponent of the element type V,
// values up to 255.9 of it would round to 256, above what the type holds.
template <int V>
__device__ __forceinline__ bool block_top(uint32_t byte) {
  return byte == (V == MP_FP16 ? 127u + 15u - 7u : 127u + 127u - 7u);
}
__device__ __forceinline__ float below_256(float f) { return fminf(fmaxf(f, -240.0f), 240.0f); }

// The largest magnitudes of the blocks that a lane's slots are in, NaN if one is NaN
// (all lanes of the warp call): of values in fp32, and of 16-bit ones as
// integers, two at a time: without the sign, patterns rise with the magnitude, infinities
// next and NaN last.
template <int T, bool Wide>
__device__ __forceinline__ void blocks_amax(float (&m)[8 / kShare<T, Wide>], const F8& f) {
  if constexpr (Wide) {
    m[0] = amax8(0.0f, f);
    m[0] = max_nan(m[0], __shfl_xor_sync(kAll, m[0], 1));
    m[0] = max_nan(m[0], __shfl_xor_sync(kAll, m[0], 2));
  } else if constexpr (T == MP_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[2 * i] = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(f.p[i].x) & 0x7FFFFFFFu));
      m[2 * i + 1] = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(f.p[i].y) & 0x7FFFFFFFu));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = amax2(0.0f, f.p[i]);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m[i] = max_nan(m[i], __shfl_xor_sync(kAll, m[i], o));
    }
  }
}

template <int T, bool Wide>
__device__ __forceinline__ void blocks_amax(float (&m)[8 / kShare<T, Wide>], const Pack8<T>& u) {
  if constexpr (T == MP_FP32) {
    blocks_amax<T, Wide>(m, get8(u));
  } else {
    constexpr uint32_t kMask = 0x7FFF7FFFu;
    if constexpr (Wide) {
      uint32_t w = __vimax3_u16x2(u.v.x & kMask, u.v.y & kMask, u.v.z & kMask);
      w = __vmaxu2(w, u.v.w & kMask);
      w = __vmaxu2(w, __shfl_xor_sync(kAll, w, 1));
      w = __vmaxu2(w, __shfl_xor_sync(kAll, w, 2));
      m[0] = Elem<T>::get(static_cast<uint16_t>(max(w & 0xFFFFu, w >> 16)));
    } else {
      // pairs 0 and 1, 2 and 3 side by side
      const auto side = [](uint32_t a, uint32_t b) {
        return __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)) & kMask;
      };
      uint32_t a = side(u.v.x & kMask, u.v.y & kMask), b = side(u.v.z & kMask, u.v.w & kMask);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        a = __vmaxu2(a, __shfl_xor_sync(kAll, a, o));
        b = __vmaxu2(b, __shfl_xor_sync(kAll, b, o));
      }
      m[0] = Elem<T>::get(static_cast<uint16_t>(a));
      m[1] = Elem<T>::get(static_cast<uint16_t>(a >> 16));
      m[2] = Elem<T>::get(static_cast<uint16_t>(b));
      m[3] = Elem<T>::get(static_cast<uint16_t>(b >> 16));
    }
  }
}

// Puts a lane's eight values f (of element type V, whose blocks' largest magnitudes
// are m) away in 8 bits with the blocks' scales. Slots past the row are zeros;
// where `live` is false nothing is written.
template <int T, int V, bool Wide>
__device__ __forceinline__ void put_block8(const F8& f, const float (&m)[8 / kShare<T, Wide>], uint8_t* row,
                                           uint8_t* scales, int base, int l, int n, bool live) {
  constexpr int kS = kShare<T, Wide>;
  uint32_t byte[8 / kS];
  float inverse[8 / kS];
  bool top = false;
#pragma unroll
  for (int i = 0; i < 8 / kS; ++i) {
    byte[i] = block_scale(m[i]);
    inverse[i] = block_inverse(byte[i]);
    top = top || block_top<V>(byte[i]);
  }
  F8 g;
#pragma unroll
  for (int i = 0; i < 4; ++i) g.p[i] = mul2(f.p[i], make_float2(inverse[2 * i / kS], inverse[(2 * i + 1) / kS]));
  if (top) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (block_top<V>(byte[2 * i / kS])) g.p[i].x = below_256(g.p[i].x);
      if (block_top<V>(byte[(2 * i + 1) / kS])) g.p[i].y = below_256(g.p[i].y);
    }
  }
  if (!live) return;
  store_unit8<T, Wide>(e4m3_pack(g), row, base, l, n);
  if (l % (32 / kS) == 0) {
    const int c = slot_column<T, Wide>(base, l, 0);
    uint8_t* p = scales + static_cast<uint32_t>(c) / 32;
#pragma unroll
    for (int i = 0; i < 8 / kS; ++i)
      if (c + 32 * kS * i < n) p[kS * i] = static_cast<uint8_t>(byte[i]);
  }
}

// The scales of a lane's slots, a byte for each share, and the values that its 8 bits
// stand for, times `factor`.
template <int T, bool Wide>
struct RawScales {
  static constexpr int kS = kShare<T, Wide>;
  uint32_t b[8 / kS];

  __device__ __forceinline__ void load(const uint8_t* scales, int base, int l, int n) {
    const int c = slot_column<T, Wide>(base, l, 0);
    const uint8_t* p = scales + static_cast<uint32_t>(c) / 32;
#pragma unroll
    for (int i = 0; i < 8 / kS; ++i) b[i] = c + 32 * kS * i < n ? p[kS * i] : 0u;
  }
  __device__ __forceinline__ F8 values(uint2 q, float factor) const {
    float s[8 / kS];
#pragma unroll
    for (int i = 0; i < 8 / kS; ++i) s[i] = __fmul_rn(block_scale_value(b[i]), factor);
    F8 r = e4m3_unpack(q);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = mul2(r.p[i], make_float2(s[2 * i / kS], s[(2 * i + 1) / kS]));
    return r;
  }
};

// ---- a scale for each row -----------------------------------------------------------

__device__ __forceinline__ float row_scale(float amax) {
  const float s = fmaxf(__fmul_rn(amax, 1.0f / 448.0f), 0x1p-126f);
  return amax < kInf ? s : __uint_as_float(0x7FC00000u);
}

}  // namespace mpk
