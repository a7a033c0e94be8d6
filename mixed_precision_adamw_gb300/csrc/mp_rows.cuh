// mp_rows.cuh — element types and reductions of the row-wise operators
// (layer norm, token log probabilities, distillation).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mp_train.h"

namespace mpk {

// ---- argument checks shared by the entry points ---------------------------
constexpr int64_t kMaxRows = int64_t{1} << 40;  // also of a row stride

inline bool type_ok(int32_t t) { return t == MP_BF16 || t == MP_FP16 || t == MP_FP32; }
inline bool index_type_ok(int32_t t) { return t == MP_INT32 || t == MP_INT64; }
inline bool rows_ok(int64_t rows) { return rows >= 0 && rows < kMaxRows; }
inline bool vocab_ok(int64_t vocab) { return vocab >= 1 && vocab <= INT32_MAX; }
inline bool stride_ok(int64_t stride, int64_t length) { return stride >= length && stride < kMaxRows; }
inline bool scale_ok(float scale) { return scale > 0.0f && scale <= 0x1p126f; }  // scale * log2(e) is finite
inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool aligned4(const void* p) { return aligned_to(p, 4); }
inline bool type_aligned(const void* p, int32_t t) { return aligned_to(p, t == MP_FP32 ? 4 : 2); }
inline bool index_aligned(const void* p, int32_t t) { return aligned_to(p, t == MP_INT64 ? 8 : 4); }

// ---- elements ---------------------------------------------------------------

constexpr float kInf = INFINITY;
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// A matrix element of mp_dtype_t `T` as stored, widened to fp32 exactly and
// rounded back to nearest even.
template <int T>
struct Elem;

template <>
struct Elem<MP_BF16> {
  using type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }
  static __device__ __forceinline__ uint16_t put(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
  static constexpr uint16_t kMinusInf = 0xFF80;
};

template <>
struct Elem<MP_FP16> {
  using type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t h) { return __half2float(__ushort_as_half(h)); }
  static __device__ __forceinline__ uint16_t put(float x) { return __half_as_ushort(__float2half_rn(x)); }
  static constexpr uint16_t kMinusInf = 0xFC00;
};

template <>
struct Elem<MP_FP32> {
  using type = float;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
  static constexpr float kMinusInf = -kInf;
};

// One element of a vector whose type is known at run time only (weights:
// read or written once per block or launch).
__device__ __forceinline__ float load_as(const void* p, int64_t i, int type) {
  if (type == MP_FP32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return type == MP_BF16 ? Elem<MP_BF16>::get(h) : Elem<MP_FP16>::get(h);
}

__device__ __forceinline__ void store_as(void* p, int64_t i, int type, float x) {
  if (type == MP_FP32)
    static_cast<float*>(p)[i] = x;
  else
    static_cast<uint16_t*>(p)[i] = type == MP_BF16 ? Elem<MP_BF16>::put(x) : Elem<MP_FP16>::put(x);
}

__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, int type) {
  return type == MP_INT64 ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

// 2^x, to 2 ulp of fp32; results below 2^-126 are 0. NaN stays NaN.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Order of the alternatives as unsigned integers: rising value, -0 equal to
// +0, NaN (of any kind) last.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  if (x != x) return 0xFFFFFFFFu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The value that order_of maps to `key` (NaN for the NaN key).
__device__ __forceinline__ float value_of_order(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// ---- eight elements of a row ------------------------------------------------
// A thread's unit of a row is eight elements, kept as stored until used. With
// Wide they are consecutive (16-B loads and stores; the row must start on a
// 16-B boundary and hold a multiple of eight elements), otherwise `step`
// apart, so that neighbouring threads read neighbouring elements.
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack2_fp16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int T>
struct Pack8 {  // bf16, fp16
  uint4 v;

  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void fill(uint16_t h) {
    const uint32_t w = h | (static_cast<uint32_t>(h) << 16);
    v = make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
  // The elements at p, from the two 16-B pieces a and b that they lie in.
  __device__ __forceinline__ void across(const uint16_t* p, uint4 a, uint4 b) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const bool two = at & 8, one = at & 4;
    const uint32_t shift = at & 2 ? 16 : 0;
    const uint32_t t[6] = {two ? a.z : a.x, two ? a.w : a.y, two ? b.x : a.z,
                           two ? b.y : a.w, two ? b.z : b.x, two ? b.w : b.y};
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = one ? t[i + 1] : t[i];
    v = make_uint4(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift),
                   __funnelshift_r(w[2], w[3], shift), __funnelshift_r(w[3], w[4], shift));
  }
  __device__ __forceinline__ void load_stepped(const uint16_t* p, int j, int step, int n) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = j + e * step < n ? p[j + e * step] : 0u;
    v = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
  }
  __device__ __forceinline__ void store_stepped(uint16_t* p, int j, int step, int n) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e * step < n) p[j + e * step] = static_cast<uint16_t>(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (T == MP_BF16) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = g.x;
        f[2 * i + 1] = g.y;
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = T == MP_BF16 ? pack2_bf16(f[2 * i], f[2 * i + 1]) : pack2_fp16(f[2 * i], f[2 * i + 1]);
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Pack8<MP_FP32> {
  float4 a, b;

  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void fill(float f) { a = b = make_float4(f, f, f, f); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void load_stepped(const float* p, int j, int step, int n) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = j + e * step < n ? p[j + e * step] : 0.0f;
    put(h);
  }
  __device__ __forceinline__ void store_stepped(float* p, int j, int step, int n) const {
    float h[8];
    get(h);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e * step < n) p[j + e * step] = h[e];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Sixteen bytes of a row in shared memory.
template <int T>
struct Vec16 {
  static constexpr int N = T == MP_FP32 ? 4 : 8;
  uint4 v;

  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (T == MP_FP32) {
      f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
      f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    } else {
      Pack8<T> p;
      p.v = v;
      p.get(f);
    }
  }
  __device__ __forceinline__ void put(const float (&f)[N]) {
    if constexpr (T == MP_FP32) {
      v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
      Pack8<T> p;
      p.put(f);
      v = p.v;
    }
  }
  __device__ __forceinline__ void fill_minus_inf() {
    constexpr uint32_t w = T == MP_BF16 ? 0xFF80FF80u : T == MP_FP16 ? 0xFC00FC00u : 0xFF800000u;
    v = make_uint4(w, w, w, w);
  }
  // the largest of n vectors' elements, NaN if one is NaN
  template <int n>
  static __device__ __forceinline__ float max_of(const Vec16 (&x)[n]) {
    if constexpr (T == MP_FP32) {
      float m = -kInf;
#pragma unroll
      for (int q = 0; q < n; ++q) {
        float f[4];
        x[q].get(f);
        m = max_nan(m, max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3])));
      }
      return m;
    } else {
      uint32_t a = x[0].v.x;
      auto take = [&](uint32_t w) {
        if (T == MP_BF16)
          asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(w));
        else
          asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(w));
      };
#pragma unroll
      for (int q = 0; q < n; ++q) {
        if (q) take(x[q].v.x);
        take(x[q].v.y);
        take(x[q].v.z);
        take(x[q].v.w);
      }
      return max_nan(Elem<T>::get(static_cast<uint16_t>(a)), Elem<T>::get(static_cast<uint16_t>(a >> 16)));
    }
  }
};

// The largest of U units' elements, NaN if one is NaN.
template <int T, int U>
__device__ __forceinline__ float max_of(const Pack8<T> (&x)[U]) {
  if constexpr (T == MP_FP32) {
    float m = x[0].a.x;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      float f[8];
      x[q].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, f[e]);
    }
    return m;
  } else {
    uint32_t w[4 * U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      w[4 * q] = x[q].v.x;
      w[4 * q + 1] = x[q].v.y;
      w[4 * q + 2] = x[q].v.z;
      w[4 * q + 3] = x[q].v.w;
    }
#pragma unroll
    for (int n = 4 * U; n > 1; n /= 2)
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        if (T == MP_BF16)
          asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(w[i + n / 2]));
        else
          asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(w[i + n / 2]));
      }
    const uint16_t lo = static_cast<uint16_t>(w[0]), hi = static_cast<uint16_t>(w[0] >> 16);
    return max_nan(Elem<T>::get(lo), Elem<T>::get(hi));
  }
}

// Whether rows of `length` elements, `stride` apart from p on, can be read
// and written as 16-B vectors of whole units.
inline bool wide_rows(const void* p, int64_t length, int64_t stride, int64_t rows, int32_t type) {
  const int64_t unit = type == MP_FP32 ? 4 : 8;
  return aligned_to(p, 16) && length % 8 == 0 && (rows <= 1 || stride % unit == 0);
}

}  // namespace mpk
