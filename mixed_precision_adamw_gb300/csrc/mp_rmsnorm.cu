// mp_rmsnorm.cu — RMS norm with the residual's addition, forward and backward,
// with outputs and kept activations in 8 bits, and rows put away in 8 bits
// with a scale for each.
//
// A row is read once and stays in registers from the sum of its squares to its
// outputs. All sums are fp32. Everything is bound by HBM: 8 B an element forward
// with a residual and 16-bit types (7 with the output in 8 bits), 8 B backward
// (7 with h kept in 8 bits).
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_units.cuh"

namespace mpk {
namespace {

constexpr int64_t kRowD = 8192;  // longest row that registers hold
constexpr int kMaxThreads = 512;
constexpr int kLongThreads = 512;
constexpr int64_t kSms = 152;

struct RmsArgs {
  void* y;  // dx in the backward pass
  void* h;
  float* rstd;
  uint8_t* y8;
  void* y8_scale;
  uint8_t* h8;
  uint8_t* h8_scale;
  const void* x;  // h in the backward pass (8-bit values with x_scale)
  const uint8_t* x_scale;
  const void* residual;  // dh in the backward pass
  const void* dy;
  const void* weight;
  const float* rstd_in;
  int64_t rows, d, y_stride, h_stride, y8_stride, h8_stride, x_stride, residual_stride, dy_stride;
  float eps;
  int weight_type;
  int y8_kind;
  int plain;  // y8 alone, of x itself (no norm)
};

// Sum and largest over the threads of a row: L lanes of a warp, or G warps that
// meet at a barrier of their own. `red` holds two floats a warp, of alternate rows.
template <int L>
__device__ __forceinline__ void row_join(float& s, float& m, bool want_m, float2 (*red)[kMaxThreads / 32], int G,
                                         int group, int parity) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(kAll, s, o));
  if (want_m)
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, o));
  if (L < 32 || G == 1) return;
  if (threadIdx.x % 32 == 0) red[parity][threadIdx.x / 32] = make_float2(s, m);
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * G) : "memory");
  s = 0.0f;
  for (int w = 0; w < G; ++w) {
    const float2 v = red[parity][group * G + w];
    s = __fadd_rn(s, v.x);
    m = w ? max_nan(m, v.y) : v.y;
  }
}

// Rows of up to 8 * NV * (threads of a row) elements. The next row is on its way
// while a row is summed and written.
template <int T, bool Wide, int NV, int L>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_kernel(RmsArgs a, int G) {
  pdl_enter();
  using E = typename Elem<T>::type;
  __shared__ float2 red[2][kMaxThreads / 32];
  const int per_row = L < 32 ? L : 32 * G, t = threadIdx.x % per_row, group = threadIdx.x / per_row;
  const int groups = blockDim.x / per_row;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(a.d));
  const E* x = static_cast<const E*>(a.x);
  const E* res = static_cast<const E*>(a.residual);
  float w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t j = 8 * (t + static_cast<int64_t>(v) * per_row) + e;
      w[v][e] = j < a.d ? (a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f) : 0.0f;
    }
  const bool row8 = a.y8 && a.y8_kind == MP_SCALE_ROW;
  Pack8<T> xn[NV], rn[NV];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = 8 * (t + static_cast<int64_t>(v) * per_row);
      load_unit<T, Wide>(xn[v], x + r * a.x_stride, r < a.rows ? c : a.d, a.d);
      if (res) load_unit<T, Wide>(rn[v], res + r * a.residual_stride, r < a.rows ? c : a.d, a.d);
    }
  };
  // every lane of a warp runs the same number of rounds (the shuffles are whole-warp)
  int64_t r = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t ahead = L < 32 ? threadIdx.x % 32 / L : 0;
  fetch(r);
  int parity = 0;
#pragma unroll 1
  for (; r - ahead < a.rows; r += step, parity ^= 1) {
    const bool live = r < a.rows;
    Pack8<T> u[NV];
    float s = 0.0f, m = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      u[v] = xn[v];
      float f[8];
      u[v].get(f);
      if (res) {
        float g[8];
        rn[v].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fadd_rn(f[e], g[e]);
        u[v].put(f);
        u[v].get(f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __fmaf_rn(f[e], f[e], s);
      if (row8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(__fmul_rn(f[e], w[v][e])));
      }
    }
    fetch(r + step);
    row_join<L>(s, m, row8, red, G, group, parity);
    const float rstd = a.plain ? 1.0f : rsqrtf(__fmaf_rn(s, inv_d, a.eps));
    float inverse = 0.0f;
    if (row8) {
      const float scale = row_scale(__fmul_rn(m, rstd));
      inverse = __frcp_rn(scale);
      if (t == 0 && live) static_cast<float*>(a.y8_scale)[r] = scale;
    }
    if (t == 0 && live && a.rstd) a.rstd[r] = rstd;
    const int64_t blocks = (a.d + 31) / 32;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = 8 * (t + static_cast<int64_t>(v) * per_row);
      float f[8];
      u[v].get(f);
      if (a.h && live) store_unit<T, Wide>(u[v], static_cast<E*>(a.h) + r * a.h_stride, c, a.d);
      if (a.h8) put_block8<T, Wide>(f, a.h8 + r * a.h8_stride, a.h8_scale + r * blocks, c, a.d, live);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(__fmul_rn(f[e], rstd), w[v][e]);
      if (a.y && live) {
        Pack8<T> o;
        o.put(f);
        store_unit<T, Wide>(o, static_cast<E*>(a.y) + r * a.y_stride, c, a.d);
      }
      if (row8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], inverse);
        if (live) store_unit8<Wide>(e4m3_pack(f), a.y8 + r * a.y8_stride, c, a.d);
      } else if (a.y8) {
        put_block8<MP_FP32, Wide>(f, a.y8 + r * a.y8_stride, static_cast<uint8_t*>(a.y8_scale) + r * blocks, c, a.d,
                                  live);
      }
    }
  }
}

// ---- longer rows --------------------------------------------------------------
// A block a row, a lane a column and a warp 32 neighbouring ones, so that a
// warp's columns share a scale; the row is read again for the outputs.

__device__ __forceinline__ float long_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < kLongThreads / 32; ++w) s = __fadd_rn(s, red[w]);
  return s;
}

__device__ __forceinline__ float long_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < kLongThreads / 32; ++w) s = max_nan(s, red[w]);
  return s;
}

template <int T>
__device__ __forceinline__ void long_block8(float f, uint8_t* row, uint8_t* scales, int64_t j, int64_t d) {
  const uint32_t byte = block_scale(warp_max(fabsf(f)));
  if (j >= d) return;
  const float g[8] = {f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  row[j] = static_cast<uint8_t>(block_pack<T>(g, byte).x);
  if (j % 32 == 0) scales[j / 32] = static_cast<uint8_t>(byte);
}

template <int T>
__global__ void __launch_bounds__(kLongThreads) rms_forward_long_kernel(RmsArgs a) {
  pdl_enter();
  using E = Elem<T>;
  using S = typename E::type;
  __shared__ float red[kLongThreads / 32];
  const bool row8 = a.y8 && a.y8_kind == MP_SCALE_ROW;
  const int64_t blocks = (a.d + 31) / 32;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const S* x = static_cast<const S*>(a.x) + r * a.x_stride;
    const S* res = a.residual ? static_cast<const S*>(a.residual) + r * a.residual_stride : nullptr;
    S* h = a.h ? static_cast<S*>(a.h) + r * a.h_stride : nullptr;
    S* y = a.y ? static_cast<S*>(a.y) + r * a.y_stride : nullptr;
    auto weight = [&](int64_t j) { return a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f; };
    auto sum_of = [&](int64_t j) {
      return res ? E::get(E::put(__fadd_rn(E::get(x[j]), E::get(res[j])))) : E::get(x[j]);
    };
    float s = 0.0f, m = 0.0f;
    for (int64_t j = threadIdx.x; j < a.d; j += kLongThreads) {
      const float f = sum_of(j);
      if (h) h[j] = E::put(f);
      s = __fmaf_rn(f, f, s);
      if (row8) m = max_nan(m, fabsf(__fmul_rn(f, weight(j))));
    }
    const float rstd =
        a.plain ? 1.0f : rsqrtf(__fmaf_rn(long_sum(s, red), __fdiv_rn(1.0f, static_cast<float>(a.d)), a.eps));
    float inverse = 0.0f;
    if (row8) {
      const float scale = row_scale(__fmul_rn(long_max(m, red), rstd));
      inverse = __frcp_rn(scale);
      if (threadIdx.x == 0) static_cast<float*>(a.y8_scale)[r] = scale;
    }
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    // whole warps, for the scales of 32 columns; h may lie over x, and a thread reads what it wrote itself
    for (int64_t j = threadIdx.x; j < blocks * 32; j += kLongThreads) {
      const bool in = j < a.d;
      float f = in ? (h ? E::get(h[j]) : sum_of(j)) : 0.0f;
      if (a.h8) long_block8<T>(f, a.h8 + r * a.h8_stride, a.h8_scale + r * blocks, j, a.d);
      f = __fmul_rn(__fmul_rn(f, rstd), in ? weight(j) : 0.0f);
      if (y && in) y[j] = E::put(f);
      if (row8) {
        if (in) a.y8[r * a.y8_stride + j] = static_cast<uint8_t>(e4m3_pair(__fmul_rn(f, inverse), 0.0f));
      } else if (a.y8) {
        long_block8<MP_FP32>(f, a.y8 + r * a.y8_stride, static_cast<uint8_t*>(a.y8_scale) + r * blocks, j, a.d);
      }
    }
  }
}

// ---- backward -----------------------------------------------------------------
// A thread owns the same columns in every row it sees and adds their dy xh in
// registers; a block writes its sums once, part[block][d], and a second, small
// launch adds the blocks' sums in block order.
template <int T, bool Wide, bool H8, int NV, int L>
__global__ void __launch_bounds__(kMaxThreads) rms_backward_kernel(RmsArgs a, float* part, int G) {
  pdl_enter();
  using E = typename Elem<T>::type;
  __shared__ float2 red[2][kMaxThreads / 32];
  extern __shared__ __align__(16) float joined[];  // a block's groups' sums
  const int per_row = L < 32 ? L : 32 * G, t = threadIdx.x % per_row, group = threadIdx.x / per_row;
  const int groups = blockDim.x / per_row;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(a.d));
  const int64_t blocks = (a.d + 31) / 32;
  const E* dy = static_cast<const E*>(a.dy);
  const E* dh = static_cast<const E*>(a.residual);
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t j = 8 * (t + static_cast<int64_t>(v) * per_row) + e;
      w[v][e] = j < a.d ? (a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f) : 0.0f;
      dw[v][e] = 0.0f;
    }
  Pack8<T> yn[NV], gn[NV], hn[H8 ? 1 : NV];
  uint2 qn[H8 ? NV : 1];
  uint32_t bn[H8 ? NV : 1];
  float rstd_n = 0.0f;
  auto fetch = [&](int64_t r) {
    const bool live = r < a.rows;
    rstd_n = live ? a.rstd_in[r] : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = live ? 8 * (t + static_cast<int64_t>(v) * per_row) : a.d;
      load_unit<T, Wide>(yn[v], dy + r * a.dy_stride, c, a.d);
      if constexpr (H8) {
        qn[v] = load_unit8<Wide>(static_cast<const uint8_t*>(a.x) + r * a.x_stride, c, a.d);
        bn[v] = c < a.d ? a.x_scale[r * blocks + c / 32] : 127u;
      } else {
        load_unit<T, Wide>(hn[v], static_cast<const E*>(a.x) + r * a.x_stride, c, a.d);
      }
      if (dh) load_unit<T, Wide>(gn[v], dh + r * a.residual_stride, c, a.d);
    }
  };
  int64_t r = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t ahead = L < 32 ? threadIdx.x % 32 / L : 0;
  fetch(r);
  int parity = 0;
#pragma unroll 1
  for (; r - ahead < a.rows; r += step, parity ^= 1) {
    const bool live = r < a.rows;
    const float rstd = rstd_n;
    Pack8<T> g[NV], dhp[NV];
    float xh[NV][8], s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      g[v] = yn[v];
      if (dh) dhp[v] = gn[v];
      if constexpr (H8) {
        e4m3_unpack(qn[v], xh[v]);
        const float k = __fmul_rn(block_scale_value(bn[v]), rstd);
#pragma unroll
        for (int e = 0; e < 8; ++e) xh[v][e] = __fmul_rn(xh[v][e], k);
      } else {
        hn[v].get(xh[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) xh[v][e] = __fmul_rn(xh[v][e], rstd);
      }
      float f[8];
      g[v].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = __fmaf_rn(__fmul_rn(f[e], w[v][e]), xh[v][e], s);
        dw[v][e] = __fmaf_rn(f[e], xh[v][e], dw[v][e]);
      }
    }
    fetch(r + step);
    float none = 0.0f;
    row_join<L>(s, none, false, red, G, group, parity);
    if (!a.y || !live) continue;
    const float c = -__fmul_rn(__fmul_rn(s, inv_d), rstd);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float f[8], o[8];
      g[v].get(f);
      if (dh)
        dhp[v].get(o);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = __fmaf_rn(__fmul_rn(f[e], w[v][e]), rstd, __fmaf_rn(xh[v][e], c, dh ? o[e] : 0.0f));
      Pack8<T> u;
      u.put(o);
      store_unit<T, Wide>(u, static_cast<E*>(a.y) + r * a.y_stride, 8 * (t + static_cast<int64_t>(v) * per_row), a.d);
    }
  }
  if (!part) return;
  float* to = part + static_cast<int64_t>(blockIdx.x) * a.d;
  if (groups == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t j = 8 * (t + static_cast<int64_t>(v) * per_row) + e;
        if (j < a.d) to[j] = dw[v][e];
      }
    return;
  }
  const int width = 8 * NV * per_row;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) joined[group * width + 8 * (t + v * per_row) + e] = dw[v][e];
  __syncthreads();
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    float s = 0.0f;
    for (int q = 0; q < groups; ++q) s = __fadd_rn(s, joined[q * width + j]);
    to[j] = s;
  }
}

// Rows longer than the registers hold: dx row by row, in two passes.
template <int T, bool H8>
__device__ __forceinline__ float long_h(const RmsArgs& a, int64_t r, int64_t j) {
  if constexpr (H8) {
    float f[8];
    e4m3_unpack(make_uint2(static_cast<const uint8_t*>(a.x)[r * a.x_stride + j], 0u), f);
    return __fmul_rn(f[0], block_scale_value(a.x_scale[r * ((a.d + 31) / 32) + j / 32]));
  } else {
    return Elem<T>::get(static_cast<const typename Elem<T>::type*>(a.x)[r * a.x_stride + j]);
  }
}

template <int T, bool H8>
__global__ void __launch_bounds__(kLongThreads) rms_dx_long_kernel(RmsArgs a) {
  pdl_enter();
  using E = Elem<T>;
  using S = typename E::type;
  __shared__ float red[kLongThreads / 32];
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(a.d));
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const S* dy = static_cast<const S*>(a.dy) + r * a.dy_stride;
    const S* dh = a.residual ? static_cast<const S*>(a.residual) + r * a.residual_stride : nullptr;
    S* dx = static_cast<S*>(a.y) + r * a.y_stride;
    const float rstd = a.rstd_in[r];
    auto g = [&](int64_t j) {
      return __fmul_rn(E::get(dy[j]), a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f);
    };
    float s = 0.0f;
    for (int64_t j = threadIdx.x; j < a.d; j += kLongThreads)
      s = __fmaf_rn(g(j), __fmul_rn(long_h<T, H8>(a, r, j), rstd), s);
    const float c = -__fmul_rn(__fmul_rn(long_sum(s, red), inv_d), rstd);
    for (int64_t j = threadIdx.x; j < a.d; j += kLongThreads)
      dx[j] = E::put(__fmaf_rn(g(j), rstd,
                               __fmaf_rn(__fmul_rn(long_h<T, H8>(a, r, j), rstd), c, dh ? E::get(dh[j]) : 0.0f)));
  }
}

// ... and the weight gradient column by column: block (i, c) adds 512 columns over
// the c-th chunk of rows.
template <int T, bool H8>
__global__ void __launch_bounds__(kLongThreads) rms_dw_long_kernel(RmsArgs a, float* part) {
  pdl_enter();
  using E = Elem<T>;
  const int64_t strips = (a.d + kLongThreads - 1) / kLongThreads;
  const int64_t c = blockIdx.x / strips, chunks = gridDim.x / strips;
  const int64_t j = (blockIdx.x % strips) * kLongThreads + threadIdx.x;
  if (j >= a.d) return;
  const int64_t r1 = a.rows * (c + 1) / chunks;
  float s = 0.0f;
#pragma unroll 4
  for (int64_t r = a.rows * c / chunks; r < r1; ++r) {
    const float g = E::get(static_cast<const typename E::type*>(a.dy)[r * a.dy_stride + j]);
    s = __fmaf_rn(g, __fmul_rn(long_h<T, H8>(a, r, j), a.rstd_in[r]), s);
  }
  part[c * a.d + j] = s;
}

// dweight from `parts` blocks' sums: 32 columns a block, 32 threads a column,
// each adding every 32nd block's sum.
constexpr int kFinishSlices = 32;

__global__ void __launch_bounds__(32 * kFinishSlices) rms_finish_kernel(void* dweight, const float* part, int64_t d,
                                                                        int parts, int weight_type) {
  pdl_enter();
  __shared__ float red[kFinishSlices][33];
  const int c = threadIdx.x % 32, slice = threadIdx.x / 32;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float s = 0.0f;
  if (j < d) {
#pragma unroll 8
    for (int p = slice; p < parts; p += kFinishSlices) s = __fadd_rn(s, part[static_cast<int64_t>(p) * d + j]);
  }
  red[slice][c] = s;
  __syncthreads();
  if (slice || j >= d) return;
  s = 0.0f;
#pragma unroll
  for (int q = 0; q < kFinishSlices; ++q) s = __fadd_rn(s, red[q][c]);
  store_as(dweight, j, weight_type, s);
}

// ---- launches -------------------------------------------------------------------

// How the threads of a block share rows of d elements.
struct RowPlan {
  int lanes, units, warps, threads;  // lanes of a row if under a warp; units a thread; warps of a row; of a block
};

RowPlan row_plan(int64_t d, int64_t most_units) {
  const int64_t units = (d + 7) / 8;
  RowPlan p = {32, 1, 1, 256};
  if (units <= 16) {
    p.lanes = units <= 8 ? 8 : 16;
    return p;
  }
  p.units = units > most_units ? 2 : 1;
  p.warps = static_cast<int>((units + 32 * p.units - 1) / (32 * p.units));
  p.threads = 32 * p.warps * std::max(1, 8 / p.warps);
  return p;
}

template <int T, bool Wide, int NV, int L>
cudaError_t forward_rows(const RmsArgs& a, const RowPlan& p, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t groups = p.threads / (L < 32 ? L : 32 * p.warps);
  const int64_t per_sm = std::max<int64_t>(1, 1024 / p.threads);
  const int64_t blocks = std::min((a.rows + groups - 1) / groups, per_sm * dev.sms);
  return launch_pdl(rms_forward_kernel<T, Wide, NV, L>, static_cast<unsigned>(blocks),
                    static_cast<unsigned>(p.threads), s, a, p.warps);
}

template <int T, bool Wide>
cudaError_t forward_wide(const RmsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const RowPlan p = row_plan(a.d, 64);
  if (p.lanes == 8) return forward_rows<T, Wide, 1, 8>(a, p, dev, s);
  if (p.lanes == 16) return forward_rows<T, Wide, 1, 16>(a, p, dev, s);
  if (p.units == 1) return forward_rows<T, Wide, 1, 32>(a, p, dev, s);
  return forward_rows<T, Wide, 2, 32>(a, p, dev, s);
}

template <int T>
cudaError_t forward(const RmsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.d > kRowD)
    return launch_pdl(rms_forward_long_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 4 * dev.sms)),
                      kLongThreads, s, a);
  const bool wide = wide_rows(a.x, a.d, a.x_stride, a.rows, T) &&
                    (!a.residual || wide_rows(a.residual, a.d, a.residual_stride, a.rows, T)) &&
                    (!a.y || wide_rows(a.y, a.d, a.y_stride, a.rows, T)) &&
                    (!a.h || wide_rows(a.h, a.d, a.h_stride, a.rows, T)) &&
                    (!a.y8 || wide_rows8(a.y8, a.d, a.y8_stride, a.rows)) &&
                    (!a.h8 || wide_rows8(a.h8, a.d, a.h8_stride, a.rows));
  return wide ? forward_wide<T, true>(a, dev, s) : forward_wide<T, false>(a, dev, s);
}

cudaError_t forward_of(int32_t type, const RmsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  return type == MP_BF16 ? forward<MP_BF16>(a, dev, s)
                         : type == MP_FP16 ? forward<MP_FP16>(a, dev, s) : forward<MP_FP32>(a, dev, s);
}

// Blocks of the backward pass, from rows and d alone: they fix the order of the
// sums over rows and the workspace.
int backward_parts(int64_t rows, int64_t d) {
  int64_t cap, per_block;  // blocks; rows that make a further block worth its partial sum
  if (d > kRowD) {
    cap = 64;
    per_block = 32;
  } else {
    const RowPlan p = row_plan(d, 512);
    const int64_t groups = p.threads / (p.lanes < 32 ? p.lanes : 32 * p.warps);
    cap = std::max<int64_t>(1, 1024 / p.threads) * kSms;
    per_block = 2 * groups;
  }
  return static_cast<int>(std::max<int64_t>(1, std::min(cap, (rows + per_block - 1) / per_block)));
}

template <int T, bool Wide, bool H8, int NV, int L>
cudaError_t backward_rows(const RmsArgs& a, const RowPlan& p, int parts, float* part, cudaStream_t s) {
  const int per_row = L < 32 ? L : 32 * p.warps;
  const size_t smem = p.threads > per_row ? static_cast<size_t>(p.threads) * NV * 8 * sizeof(float) : 0;
  return launch_pdl_smem(rms_backward_kernel<T, Wide, H8, NV, L>, static_cast<unsigned>(parts),
                         static_cast<unsigned>(p.threads), smem, s, a, part, p.warps);
}

template <int T, bool Wide, bool H8>
cudaError_t backward_wide(const RmsArgs& a, int parts, float* part, cudaStream_t s) {
  const RowPlan p = row_plan(a.d, 512);
  if (p.lanes == 8) return backward_rows<T, Wide, H8, 1, 8>(a, p, parts, part, s);
  if (p.lanes == 16) return backward_rows<T, Wide, H8, 1, 16>(a, p, parts, part, s);
  if (p.units == 1) return backward_rows<T, Wide, H8, 1, 32>(a, p, parts, part, s);
  return backward_rows<T, Wide, H8, 2, 32>(a, p, parts, part, s);
}

template <int T, bool H8>
cudaError_t backward(const RmsArgs& a, void* dweight, float* part, const DeviceInfo& dev, cudaStream_t s) {
  const int parts = backward_parts(a.rows, a.d);
  cudaError_t e = cudaSuccess;
  if (a.d <= kRowD) {
    const bool wide = wide_rows(a.dy, a.d, a.dy_stride, a.rows, T) &&
                      (!a.residual || wide_rows(a.residual, a.d, a.residual_stride, a.rows, T)) &&
                      (!a.y || wide_rows(a.y, a.d, a.y_stride, a.rows, T)) &&
                      (H8 ? wide_rows8(a.x, a.d, a.x_stride, a.rows) : wide_rows(a.x, a.d, a.x_stride, a.rows, T));
    float* to = dweight ? part : nullptr;
    e = wide ? backward_wide<T, true, H8>(a, parts, to, s) : backward_wide<T, false, H8>(a, parts, to, s);
  } else {
    const int64_t strips = (a.d + kLongThreads - 1) / kLongThreads;
    if (dweight)  // before dx, which may be written over dy or h
      e = launch_pdl(rms_dw_long_kernel<T, H8>, static_cast<unsigned>(strips * parts), kLongThreads, s, a, part);
    if (e == cudaSuccess && a.y && a.rows)
      e = launch_pdl(rms_dx_long_kernel<T, H8>, static_cast<unsigned>(std::min<int64_t>(a.rows, 4 * dev.sms)),
                     kLongThreads, s, a);
  }
  if (e == cudaSuccess && dweight)
    e = launch_pdl(rms_finish_kernel, static_cast<unsigned>((a.d + 31) / 32), 32 * kFinishSlices, s, dweight,
                   static_cast<const float*>(part), a.d, parts, a.weight_type);
  return e;
}

template <int T>
cudaError_t backward_h(const RmsArgs& a, void* dweight, float* part, const DeviceInfo& dev, cudaStream_t s) {
  return a.x_scale ? backward<T, true>(a, dweight, part, dev, s) : backward<T, false>(a, dweight, part, dev, s);
}

}  // namespace

cudaError_t launch_pack8_rows(uint8_t* q, float* scale, const void* x, int64_t rows, int64_t d, int64_t q_stride,
                              int64_t x_stride, int32_t type, const DeviceInfo& dev, cudaStream_t s) {
  RmsArgs a = {};
  a.y8 = q;
  a.y8_scale = scale;
  a.y8_kind = MP_SCALE_ROW;
  a.x = x;
  a.rows = rows;
  a.d = d;
  a.y8_stride = q_stride;
  a.x_stride = x_stride;
  a.plain = 1;
  return forward_of(type, a, dev, s);
}

}  // namespace mpk

extern "C" int mp_rmsnorm_forward(void* y, void* h, float* rstd, void* y8, void* y8_scale, void* h8, void* h8_scale,
                                  const void* x, const void* residual, const void* weight, int64_t rows, int64_t d,
                                  int64_t y_stride, int64_t h_stride, int64_t y8_stride, int64_t h8_stride,
                                  int64_t x_stride, int64_t residual_stride, float eps, int32_t type,
                                  int32_t weight_type, int32_t y8_kind, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !type_ok(weight_type) || !unit_shape_ok(rows, d) || (y && !stride_ok(y_stride, d)) ||
      (h && !stride_ok(h_stride, d)) || (y8 && (!stride_ok(y8_stride, d) || !scale8_ok(y8_kind))) ||
      (h8 && !stride_ok(h8_stride, d)) || !stride_ok(x_stride, d) || (residual && !stride_ok(residual_stride, d)) ||
      !(eps >= 0.0f) || !std::isfinite(eps))
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!x || (!y && !h && !rstd && !y8 && !h8) || (y8 && !y8_scale) || (h8 && !h8_scale) || (h && !residual))
    return MP_ERR_NULL;
  if (!alias_ok(y, y_stride, x, x_stride) || !alias_ok(y, y_stride, residual, residual_stride) ||
      !alias_ok(h, h_stride, x, x_stride) || !alias_ok(h, h_stride, residual, residual_stride) || (y && y == h) ||
      (y8 && (y8 == h8 || y8 == x || y8 == residual || y8 == y || y8 == h)) ||
      (h8 && (h8 == x || h8 == residual || h8 == y || h8 == h)))
    return MP_ERR_RANGE;
  if (!type_aligned(y, type) || !type_aligned(h, type) || !type_aligned(x, type) || !type_aligned(residual, type) ||
      !type_aligned(weight, weight_type) || !aligned4(rstd) || (y8 && !scale8_aligned(y8_scale, y8_kind)))
    return MP_ERR_ALIGN;
  DeviceInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return record_cuda_error(e);
  RmsArgs a = {};
  a.y = y;
  a.h = h;
  a.rstd = rstd;
  a.y8 = static_cast<uint8_t*>(y8);
  a.y8_scale = y8_scale;
  a.h8 = static_cast<uint8_t*>(h8);
  a.h8_scale = static_cast<uint8_t*>(h8_scale);
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.rows = rows;
  a.d = d;
  a.y_stride = y_stride;
  a.h_stride = h_stride;
  a.y8_stride = y8_stride;
  a.h8_stride = h8_stride;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.eps = eps;
  a.weight_type = weight_type;
  a.y8_kind = y8_kind;
  e = forward_of(type, a, dev, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}

extern "C" size_t mp_rmsnorm_workspace_bytes(int64_t rows, int64_t d) {
  using namespace mpk;
  if (!unit_shape_ok(rows, d)) return 0;
  return static_cast<size_t>(backward_parts(rows, d)) * d * sizeof(float);
}

extern "C" int mp_rmsnorm_backward(void* dx, void* dweight, const void* dy, const void* dh, const void* h,
                                   const void* h_scale, const void* weight, const float* rstd, int64_t rows,
                                   int64_t d, int64_t dx_stride, int64_t dy_stride, int64_t dh_stride,
                                   int64_t h_stride, int32_t type, int32_t weight_type, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !type_ok(weight_type) || !unit_shape_ok(rows, d) || (dx && !stride_ok(dx_stride, d)) ||
      !stride_ok(dy_stride, d) || (dh && !stride_ok(dh_stride, d)) || !stride_ok(h_stride, d))
    return MP_ERR_RANGE;
  if (rows == 0 && !dweight) return MP_OK;
  if (!dx && !dweight) return MP_ERR_NULL;
  if (rows > 0 && (!dy || !h || !rstd)) return MP_ERR_NULL;
  if (!alias_ok(dx, dx_stride, dy, dy_stride) || !alias_ok(dx, dx_stride, dh, dh_stride) ||
      (dx && dx == h && (h_scale || dx_stride != h_stride)))
    return MP_ERR_RANGE;
  if (!type_aligned(dx, type) || !type_aligned(dy, type) || !type_aligned(dh, type) ||
      (!h_scale && !type_aligned(h, type)) || !type_aligned(weight, weight_type) ||
      !type_aligned(dweight, weight_type) || !aligned4(rstd) || !aligned_to(workspace, 16))
    return MP_ERR_ALIGN;
  if (dweight && (!workspace || workspace_bytes < mp_rmsnorm_workspace_bytes(rows, d))) return MP_ERR_WORKSPACE;
  DeviceInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return record_cuda_error(e);
  RmsArgs a = {};
  a.y = dx;
  a.x = h;
  a.x_scale = static_cast<const uint8_t*>(h_scale);
  a.residual = dh;
  a.dy = dy;
  a.weight = weight;
  a.rstd_in = rstd;
  a.rows = rows;
  a.d = d;
  a.y_stride = dx_stride;
  a.x_stride = h_stride;
  a.residual_stride = dh_stride;
  a.dy_stride = dy_stride;
  a.weight_type = weight_type;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  e = type == MP_BF16 ? backward_h<MP_BF16>(a, dweight, part, dev, s)
                      : type == MP_FP16 ? backward_h<MP_FP16>(a, dweight, part, dev, s)
                                        : backward_h<MP_FP32>(a, dweight, part, dev, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}
