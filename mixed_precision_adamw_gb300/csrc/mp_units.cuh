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

// Columns c to c + 7 of a row of n, zeros from n on.
template <int T>
__device__ __forceinline__ void load_across(Pack8<T>& u, const typename Elem<T>::type* row, int c, int n) {
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
      const int left = c < n ? n - c : 0;
      uint32_t w[4] = {u.v.x, u.v.y, u.v.z, u.v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < left ? w[i] : 2 * i < left ? w[i] & 0xFFFFu : 0u;
      u.v = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int T, bool Wide>
__device__ __forceinline__ void load_unit(Pack8<T>& u, const typename Elem<T>::type* row, int c, int n) {
  if (!Wide)
    load_across(u, row, c, n);
  else if (c < n)
    u.load(row + c);
  else
    u.zero();
}

// Writes the units of a warp. All lanes call; runs of `run` neighbouring lanes hold
// neighbouring units of one row (the lanes whose `live` is false, whole runs,
// write nothing). Rows off the 16-byte grid: a lane gets the end of its neighbour's
// unit by shuffles and writes the 16-byte piece that its own first columns lie
// in; what no whole piece holds (a run's ends, a row's end) is written by elements. Written by
// elements throughout, each of eight stores of a warp touches all its sectors:
// 1021 x 2731 fp16 backward 21.9 us that way.
template <int T, bool Wide>
__device__ __forceinline__ void store_unit(const Pack8<T>& u, typename Elem<T>::type* row, int c, int n,
                                           bool live, int run) {
  using E = typename Elem<T>::type;
  if constexpr (Wide) {
    if (live && c < n) u.store(row + c);
  } else {
    constexpr int kPiece = 16 / sizeof(E);
    const int lane = threadIdx.x % 32;
    const bool first = lane % run == 0, last = (lane + 1) % run == 0;
    E* at = row + c;
    const int p = static_cast<int>(reinterpret_cast<uintptr_t>(at) % 16 / sizeof(E));
    // whether the piece that column c (or the next unit's) lies in is in the row and in the warp
    const bool whole = (p == 0 || !first) && c - p + kPiece <= n;
    const bool next = p == 0 || (!last && c + 8 - p + kPiece <= n);
    uint32_t own = 0;  // elements to be written one by one
    if constexpr (T == MP_FP32) {
      float f[8], w[11];
      u.get(f);
#pragma unroll
      for (int i = 0; i < 3; ++i) w[i] = __shfl_up_sync(kAll, f[5 + i], 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[3 + i] = f[i];
      float t[9], o[8];  // o: columns c - p to c - p + 7
#pragma unroll
      for (int i = 0; i < 9; ++i) t[i] = p & 2 ? w[i] : w[i + 2];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = p & 1 ? t[i] : t[i + 1];
      const bool second = c - p + 8 <= n;  // all of it the lane's own
      if (live && whole) *reinterpret_cast<float4*>(at - p) = make_float4(o[0], o[1], o[2], o[3]);
      if (live && second) *reinterpret_cast<float4*>(at - p + 4) = make_float4(o[4], o[5], o[6], o[7]);
      own = (whole ? 0u : (1u << (4 - p)) - 1u) | (second ? 0u : 0xF0u >> p & 0xFFu) |
            (next ? 0u : 0xFF00u >> p & 0xFFu);
      if (live && own)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((own >> e & 1) && c + e < n) at[e] = f[e];
    } else {
      uint4 before;
      before.x = __shfl_up_sync(kAll, u.v.x, 1);
      before.y = __shfl_up_sync(kAll, u.v.y, 1);
      before.z = __shfl_up_sync(kAll, u.v.z, 1);
      before.w = __shfl_up_sync(kAll, u.v.w, 1);
      Pack8<T> o = u;
      // eight elements, 8 - p into the neighbour's unit
      if (p) o.across(reinterpret_cast<const E*>(static_cast<uintptr_t>(16 - 2 * p)), before, u.v);
      if (live && whole) o.store(at - p);
      own = (whole ? 0u : (1u << (8 - p)) - 1u) | (next ? 0u : 0xFF00u >> p & 0xFFu);
      if (live && own) {
        const uint32_t w[4] = {u.v.x, u.v.y, u.v.z, u.v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((own >> e & 1) && c + e < n)
            at[e] = static_cast<uint16_t>(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
      }
    }
  }
}

// The same of eight bytes.
template <bool Wide>
__device__ __forceinline__ uint2 load_unit8(const uint8_t* row, int c, int n) {
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
      const int left = c < n ? n - c : 0;
      q.x = left >= 4 ? q.x : q.x & ((1u << (8 * left)) - 1u);
      q.y = left <= 4 ? 0u : q.y & ((1u << (8 * (left - 4))) - 1u);
    }
    return q;
  }
}

template <bool Wide>
__device__ __forceinline__ void store_unit8(uint2 q, uint8_t* row, int c, int n, bool live, int run) {
  if constexpr (Wide) {
    if (live && c < n) *reinterpret_cast<uint2*>(row + c) = q;
  } else {
    const int lane = threadIdx.x % 32;
    const bool first = lane % run == 0, last = (lane + 1) % run == 0;
    uint8_t* at = row + c;
    const int p = static_cast<int>(reinterpret_cast<uintptr_t>(at) % 8);
    const bool whole = (p == 0 || !first) && c - p + 8 <= n;
    const bool next = p == 0 || (!last && c + 16 - p <= n);
    const uint2 before = make_uint2(__shfl_up_sync(kAll, q.x, 1), __shfl_up_sync(kAll, q.y, 1));
    if (live && whole) {
      uint2 o = q;
      if (p) {
        const uint32_t w[3] = {p > 4 ? before.x : before.y, p > 4 ? before.y : q.x, p > 4 ? q.x : q.y};
        // the last p bytes of the neighbour's unit, then the lane's own
        const uint32_t shift = 8 * ((8 - p) & 3);
        o = make_uint2(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift));
      }
      *reinterpret_cast<uint2*>(at - p) = o;
    }
    const uint32_t own = (whole ? 0u : (1u << (8 - p)) - 1u) | (next ? 0u : 0xFF00u >> p & 0xFFu);
    if (live && own)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((own >> e & 1) && c + e < n) at[e] = static_cast<uint8_t>((e < 4 ? q.x : q.y) >> (8 * (e % 4)));
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

// Eight values of an element type T over their block's scale, in 8 bits. Where
// the block's scale is the type's largest exponent's, values up to 255.9 of it
// would round to 256, above what the type holds.
template <int T>
__device__ __forceinline__ uint2 block_pack(const F8& f, uint32_t byte) {
  constexpr uint32_t kTop = T == MP_FP16 ? 127u + 15u - 7u : 127u + 127u - 7u;
  // an exact product: the inverse is a power of two as well
  const float inverse = byte == kScaleNan ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
  F8 g = mul8(f, inverse);
  if (byte == kTop) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      g.p[i] = make_float2(fminf(fmaxf(g.p[i].x, -240.0f), 240.0f), fminf(fmaxf(g.p[i].y, -240.0f), 240.0f));
  }
  return e4m3_pack(g);
}

// The largest magnitude of four neighbouring lanes' units, NaN if one is NaN (all
// lanes of the warp call). Of 16-bit types as integers, two at a time: without
// the sign, patterns rise with the magnitude, infinities next and NaN last.
__device__ __forceinline__ float quad_amax(const F8& f) {
  float m = amax8(0.0f, f);
  m = max_nan(m, __shfl_xor_sync(kAll, m, 1));
  return max_nan(m, __shfl_xor_sync(kAll, m, 2));
}

template <int T>
__device__ __forceinline__ float quad_amax(const Pack8<T>& u) {
  if constexpr (T == MP_FP32) {
    return quad_amax(get8(u));
  } else {
    constexpr uint32_t kMask = 0x7FFF7FFFu;
    uint32_t m = __vimax3_u16x2(u.v.x & kMask, u.v.y & kMask, u.v.z & kMask);
    m = __vmaxu2(m, u.v.w & kMask);
    m = __vmaxu2(m, __shfl_xor_sync(kAll, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(kAll, m, 2));
    return Elem<T>::get(static_cast<uint16_t>(max(m & 0xFFFFu, m >> 16)));
  }
}

// Puts the unit at column c of a row, eight values f whose block's largest
// magnitude is amax, away in 8 bits with the block's scale. Four neighbouring lanes hold
// a block's four units; units past the row are zeros and write nothing. live, run: as
// store_unit.
template <int T, bool Wide>
__device__ __forceinline__ void put_block8(const F8& f, float amax, uint8_t* row, uint8_t* scales, int c, int n,
                                           bool live, int run) {
  const uint32_t byte = block_scale(amax);
  store_unit8<Wide>(block_pack<T>(f, byte), row, c, n, live, run);
  if (live && c < n && c % 32 == 0) scales[c / 32] = static_cast<uint8_t>(byte);
}

// ---- a scale for each row -----------------------------------------------------------

__device__ __forceinline__ float row_scale(float amax) {
  const float s = fmaxf(__fmul_rn(amax, 1.0f / 448.0f), 0x1p-126f);
  return amax < kInf ? s : __uint_as_float(0x7FC00000u);
}

}  // namespace mpk
