// mp_units.cuh — eight-column units of rows at any alignment, and rows in 8
// bits (e4m3 values with scales), for the operators of a block between its
// matrix products.
//
// A thread's unit is eight neighbouring columns that start at a multiple of
// eight, so the 32 columns that share a power-of-two scale are four
// neighbouring lanes'. Rows on the 16-byte grid (Wide) are read and written in
// 16-byte pieces. Of other rows a unit is cut out of the pieces that it lies
// in: each is read once more by a neighbouring lane, out of L1.
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

// ---- units ----------------------------------------------------------------------

// Columns c to c + 7 of a row of n, zeros from n on.
template <int T>
__device__ __forceinline__ void load_across(Pack8<T>& u, const typename Elem<T>::type* row, int64_t c, int64_t n) {
  using E = typename Elem<T>::type;
  constexpr int kPiece = 16 / sizeof(E);
  const E* p = row + c;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const int off = static_cast<int>(at % 16 / sizeof(E));
  const uint4* base = reinterpret_cast<const uint4*>(at - at % 16);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // a piece is read if it holds a column of the row
  const uint4 a = c < n ? base[0] : zero;
  if constexpr (T == MP_FP32) {
    const uint4 b = c + kPiece - off < n ? base[1] : zero;
    const uint4 d = off && c + 2 * kPiece - off < n ? base[2] : zero;
    const uint32_t w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, d.x, d.y, d.z, d.w};
    uint32_t t[10];
    float f[8];
#pragma unroll
    for (int i = 0; i < 10; ++i) t[i] = off & 2 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(off & 1 ? t[i + 1] : t[i]);
    if (c + 8 > n)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i >= n) f[i] = 0.0f;
    u.put(f);
  } else {
    const uint4 b = off && c + kPiece - off < n ? base[1] : zero;
    u.across(p, a, b);
    if (c + 8 > n) {
      const int left = c < n ? static_cast<int>(n - c) : 0;
      uint32_t w[4] = {u.v.x, u.v.y, u.v.z, u.v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < left ? w[i] : 2 * i < left ? w[i] & 0xFFFFu : 0u;
      u.v = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int T, bool Wide>
__device__ __forceinline__ void load_unit(Pack8<T>& u, const typename Elem<T>::type* row, int64_t c, int64_t n) {
  if (!Wide)
    load_across(u, row, c, n);
  else if (c < n)
    u.load(row + c);
  else
    u.zero();
}

template <int T, bool Wide>
__device__ __forceinline__ void store_unit(const Pack8<T>& u, typename Elem<T>::type* row, int64_t c, int64_t n) {
  if (!Wide) {
    if (c < n) u.store_stepped(row + c, 0, 1, static_cast<int>(n - c < 8 ? n - c : 8));
  } else if (c < n) {
    u.store(row + c);
  }
}

// The same of eight bytes.
template <bool Wide>
__device__ __forceinline__ uint2 load_unit8(const uint8_t* row, int64_t c, int64_t n) {
  const uint2 zero = make_uint2(0u, 0u);
  if constexpr (Wide) {
    return c < n ? *reinterpret_cast<const uint2*>(row + c) : zero;
  } else {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
    const int off = static_cast<int>(at % 8);
    const uint2* base = reinterpret_cast<const uint2*>(at - off);
    const uint2 a = c < n ? base[0] : zero;
    const uint2 b = off && c + 8 - off < n ? base[1] : zero;
    const uint32_t t[4] = {a.x, a.y, b.x, b.y};
    const bool one = off & 4;
    const uint32_t w[3] = {one ? t[1] : t[0], one ? t[2] : t[1], one ? t[3] : t[2]};
    const uint32_t shift = 8 * (off & 3);
    uint2 q = make_uint2(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift));
    if (c + 8 > n) {
      const int left = c < n ? static_cast<int>(n - c) : 0;
      q.x = left >= 4 ? q.x : q.x & ((1u << (8 * left)) - 1u);
      q.y = left <= 4 ? 0u : q.y & ((1u << (8 * (left - 4))) - 1u);
    }
    return q;
  }
}

template <bool Wide>
__device__ __forceinline__ void store_unit8(uint2 q, uint8_t* row, int64_t c, int64_t n) {
  if constexpr (Wide) {
    if (c < n) *reinterpret_cast<uint2*>(row + c) = q;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = static_cast<uint8_t>((e < 4 ? q.x : q.y) >> (8 * (e % 4)));
  }
}

// ---- e4m3 -----------------------------------------------------------------------

// Nearest e4m3 values (ties to even), magnitudes above 448 as 448, NaN as NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 e4m3_pack(const float (&f)[8]) {
  return make_uint2(e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16),
                    e4m3_pair(f[4], f[5]) | (e4m3_pair(f[6], f[7]) << 16));
}

__device__ __forceinline__ void e4m3_unpack(uint2 q, float (&f)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = g.x;
    f[2 * i + 1] = g.y;
  }
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

// Eight values of an element type T over their block's scale, in 8 bits. Where
// the block's scale is the type's largest exponent's, values up to 255.9 of it
// would round to 256, above what the type holds.
template <int T>
__device__ __forceinline__ uint2 block_pack(const float (&f)[8], uint32_t byte) {
  constexpr uint32_t kTop = T == MP_FP16 ? 127u + 15u - 7u : 127u + 127u - 7u;
  float g[8];
  // an exact product: the inverse is a power of two as well
  const float inverse = byte == kScaleNan ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
#pragma unroll
  for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(f[e], inverse);
  if (byte == kTop) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = fminf(fmaxf(g[e], -240.0f), 240.0f);
  }
  return e4m3_pack(g);
}

// The largest magnitude of eight values, NaN if one is NaN.
__device__ __forceinline__ float amax_of(const float (&f)[8]) {
  float m[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = max_nan(fabsf(f[e]), fabsf(f[e + 4]));
  return max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
}

// The largest of four neighbouring lanes' values (all lanes of the warp call).
__device__ __forceinline__ float quad_max(float v) {
  v = max_nan(v, __shfl_xor_sync(kAll, v, 1));
  return max_nan(v, __shfl_xor_sync(kAll, v, 2));
}

// Puts the unit at column c of a row away in 8 bits with its block's scale. All
// lanes of a warp call, four neighbouring lanes with a block's four units; units past
// the row are zeros and write nothing.
template <int T, bool Wide>
__device__ __forceinline__ void put_block8(const float (&f)[8], uint8_t* row, uint8_t* scales, int64_t c, int64_t n,
                                           bool live) {
  const uint32_t byte = block_scale(quad_max(amax_of(f)));
  if (!live || c >= n) return;
  store_unit8<Wide>(block_pack<T>(f, byte), row, c, n);
  if (c % 32 == 0) scales[c / 32] = static_cast<uint8_t>(byte);
}

// Reads it back.
template <bool Wide>
__device__ __forceinline__ void get_block8(float (&f)[8], const uint8_t* row, const uint8_t* scales, int64_t c,
                                           int64_t n) {
  e4m3_unpack(load_unit8<Wide>(row, c, n), f);
  const float s = c < n ? block_scale_value(scales[c / 32]) : 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], s);
}

// ---- a scale for each row -----------------------------------------------------------

__device__ __forceinline__ float row_scale(float amax) {
  const float s = fmaxf(__fmul_rn(amax, 1.0f / 448.0f), 0x1p-126f);
  return amax < kInf ? s : __uint_as_float(0x7FC00000u);
}

}  // namespace mpk
