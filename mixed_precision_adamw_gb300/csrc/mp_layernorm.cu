// mp_layernorm.cu — layer norm, forward and backward, with the reduction of
// the weight's and bias's gradients over the rows.
//
// The mean and the variance are taken in two passes over the row (the sum,
// then the squared distances from the mean), so a row with a large common
// offset loses nothing to cancellation; all sums are fp32.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_rows.cuh"

namespace mpk {
namespace {

constexpr int kLnThreads = 256;
constexpr int64_t kMaxD = int64_t{1} << 24;

// Sum over the block, to every thread; `red` holds one float per warp.
__device__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < blockDim.x / 32; ++w) s = __fadd_rn(s, red[w]);
  return s;
}

struct LnArgs {
  void* y;  // dx in the backward pass
  float* mean_out;
  float* rstd_out;
  const void* x;
  const void* dy;
  const void* weight;
  const void* bias;
  const float* mean;
  const float* rstd;
  int64_t rows, d, y_stride, x_stride, dy_stride;
  float eps;
  int weight_type;
};

template <int T>
__global__ void __launch_bounds__(kLnThreads) ln_forward_kernel(LnArgs a) {
  pdl_enter();
  using E = Elem<T>;
  __shared__ float red[kLnThreads / 32];
  const float n = static_cast<float>(a.d);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const typename E::type* x = static_cast<const typename E::type*>(a.x) + r * a.x_stride;
    typename E::type* y = static_cast<typename E::type*>(a.y) + r * a.y_stride;
    float s = 0.0f;
    for (int64_t j = threadIdx.x; j < a.d; j += kLnThreads) s = __fadd_rn(s, E::get(x[j]));
    const float mean = __fdiv_rn(block_sum(s, red), n);
    float q = 0.0f;
    for (int64_t j = threadIdx.x; j < a.d; j += kLnThreads) {
      const float c = __fsub_rn(E::get(x[j]), mean);
      q = __fmaf_rn(c, c, q);
    }
    const float var = __fdiv_rn(block_sum(q, red), n);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
    for (int64_t j = threadIdx.x; j < a.d; j += kLnThreads) {
      const float w = a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f;
      const float b = a.bias ? load_as(a.bias, j, a.weight_type) : 0.0f;
      const float xh = __fmul_rn(__fsub_rn(E::get(x[j]), mean), rstd);
      y[j] = E::put(__fmaf_rn(xh, w, b));
    }
    if (threadIdx.x == 0) {
      if (a.mean_out) a.mean_out[r] = mean;
      if (a.rstd_out) a.rstd_out[r] = rstd;
    }
  }
}

template <int T>
__global__ void __launch_bounds__(kLnThreads) ln_dx_kernel(LnArgs a) {
  pdl_enter();
  using E = Elem<T>;
  __shared__ float red[kLnThreads / 32];
  const float n = static_cast<float>(a.d);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const typename E::type* x = static_cast<const typename E::type*>(a.x) + r * a.x_stride;
    const typename E::type* dy = static_cast<const typename E::type*>(a.dy) + r * a.dy_stride;
    typename E::type* dx = static_cast<typename E::type*>(a.y) + r * a.y_stride;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t j = threadIdx.x; j < a.d; j += kLnThreads) {
      const float w = a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f;
      const float g = __fmul_rn(E::get(dy[j]), w);
      s1 = __fadd_rn(s1, g);
      s2 = __fmaf_rn(g, __fmul_rn(__fsub_rn(E::get(x[j]), mean), rstd), s2);
    }
    const float c1 = __fdiv_rn(block_sum(s1, red), n);
    const float c2 = __fdiv_rn(block_sum(s2, red), n);
    for (int64_t j = threadIdx.x; j < a.d; j += kLnThreads) {
      const float w = a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f;
      const float xh = __fmul_rn(__fsub_rn(E::get(x[j]), mean), rstd);
      const float g = __fmul_rn(E::get(dy[j]), w);
      dx[j] = E::put(__fmul_rn(rstd, __fmaf_rn(-xh, c2, __fsub_rn(g, c1))));
    }
  }
}

// Partial sums over a chunk of rows: part[0][chunk][j] for the weight,
// part[1][chunk][j] for the bias. One column per thread.
constexpr int kChunks = 64;

template <int T>
__global__ void __launch_bounds__(kLnThreads) ln_dw_kernel(LnArgs a, float* part, int chunks) {
  pdl_enter();
  using E = Elem<T>;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kLnThreads + threadIdx.x;
  if (j >= a.d) return;
  for (int c = 0; c < chunks; ++c) {
    const int64_t r0 = a.rows * c / chunks, r1 = a.rows * (c + 1) / chunks;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
      const float xv = E::get(static_cast<const typename E::type*>(a.x)[r * a.x_stride + j]);
      const float g = E::get(static_cast<const typename E::type*>(a.dy)[r * a.dy_stride + j]);
      sw = __fmaf_rn(g, __fmul_rn(__fsub_rn(xv, a.mean[r]), a.rstd[r]), sw);
      sb = __fadd_rn(sb, g);
    }
    part[static_cast<int64_t>(c) * a.d + j] = sw;
    part[(static_cast<int64_t>(chunks) + c) * a.d + j] = sb;
  }
}

__global__ void __launch_bounds__(kLnThreads) ln_dw_finish_kernel(void* dweight, void* dbias, const float* part,
                                                                  int64_t d, int chunks, int weight_type) {
  pdl_enter();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kLnThreads + threadIdx.x;
  if (j >= d) return;
  float sw = 0.0f, sb = 0.0f;
  for (int c = 0; c < chunks; ++c) {
    sw = __fadd_rn(sw, part[static_cast<int64_t>(c) * d + j]);
    sb = __fadd_rn(sb, part[(static_cast<int64_t>(chunks) + c) * d + j]);
  }
  if (dweight) store_as(dweight, j, weight_type, sw);
  if (dbias) store_as(dbias, j, weight_type, sb);
}

template <int T>
cudaError_t forward(const LnArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, 8 * dev.sms));
  return launch_pdl(ln_forward_kernel<T>, grid, kLnThreads, s, a);
}

template <int T>
cudaError_t backward(const LnArgs& a, void* dweight, void* dbias, float* part, const DeviceInfo& dev,
                     cudaStream_t s) {
  const unsigned cols = static_cast<unsigned>((a.d + kLnThreads - 1) / kLnThreads);
  cudaError_t e = cudaSuccess;
  if (dweight || dbias) {  // before dx, which may be written over dy
    e = launch_pdl(ln_dw_kernel<T>, cols, kLnThreads, s, a, part, kChunks);
    if (e != cudaSuccess) return e;
    e = launch_pdl(ln_dw_finish_kernel, cols, kLnThreads, s, dweight, dbias, static_cast<const float*>(part), a.d,
                   kChunks, a.weight_type);
  }
  if (e == cudaSuccess && a.y && a.rows)
    e = launch_pdl(ln_dx_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 8 * dev.sms)), kLnThreads, s, a);
  return e;
}

bool shape_ok(int64_t rows, int64_t d) { return rows_ok(rows) && d >= 1 && d <= kMaxD; }

}  // namespace
}  // namespace mpk

extern "C" int mp_layernorm_forward(void* y, float* mean, float* rstd, const void* x, const void* weight,
                                    const void* bias, int64_t rows, int64_t d, int64_t y_stride, int64_t x_stride,
                                    float eps, int32_t type, int32_t weight_type, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !type_ok(weight_type) || !shape_ok(rows, d) || !stride_ok(y_stride, d) ||
      !stride_ok(x_stride, d) || !(eps >= 0.0f) || !std::isfinite(eps))
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!y || !x) return MP_ERR_NULL;
  if (y == x && y_stride != x_stride) return MP_ERR_RANGE;
  if (!type_aligned(y, type) || !type_aligned(x, type) || !type_aligned(weight, weight_type) || !type_aligned(bias, weight_type) ||
      !aligned4(mean) || !aligned4(rstd))
    return MP_ERR_ALIGN;
  DeviceInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return record_cuda_error(e);
  LnArgs a = {};
  a.y = y;
  a.mean_out = mean;
  a.rstd_out = rstd;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.rows = rows;
  a.d = d;
  a.y_stride = y_stride;
  a.x_stride = x_stride;
  a.eps = eps;
  a.weight_type = weight_type;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = type == MP_BF16 ? forward<MP_BF16>(a, dev, s)
                      : type == MP_FP16 ? forward<MP_FP16>(a, dev, s) : forward<MP_FP32>(a, dev, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}

extern "C" size_t mp_layernorm_workspace_bytes(int64_t rows, int64_t d) {
  using namespace mpk;
  if (!shape_ok(rows, d)) return 0;
  return static_cast<size_t>(2) * kChunks * d * sizeof(float);
}

extern "C" int mp_layernorm_backward(void* dx, void* dweight, void* dbias, const void* dy, const void* x,
                                     const void* weight, const float* mean, const float* rstd, int64_t rows,
                                     int64_t d, int64_t dx_stride, int64_t dy_stride, int64_t x_stride, int32_t type,
                                     int32_t weight_type, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !type_ok(weight_type) || !shape_ok(rows, d) || (dx && !stride_ok(dx_stride, d)) ||
      !stride_ok(dy_stride, d) || !stride_ok(x_stride, d))
    return MP_ERR_RANGE;
  if (!dx && !dweight && !dbias) return MP_ERR_NULL;
  if (rows > 0 && (!dy || !x || !mean || !rstd)) return MP_ERR_NULL;
  if (dx && ((dx == dy && dx_stride != dy_stride) || (dx == x && dx_stride != x_stride))) return MP_ERR_RANGE;
  if (!type_aligned(dx, type) || !type_aligned(dy, type) || !type_aligned(x, type) || !type_aligned(weight, weight_type) ||
      !type_aligned(dweight, weight_type) || !type_aligned(dbias, weight_type) || !aligned4(mean) || !aligned4(rstd) ||
      !aligned_to(workspace, 16))
    return MP_ERR_ALIGN;
  if ((dweight || dbias) && (!workspace || workspace_bytes < mp_layernorm_workspace_bytes(rows, d)))
    return MP_ERR_WORKSPACE;
  DeviceInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return record_cuda_error(e);
  LnArgs a = {};
  a.y = dx;
  a.x = x;
  a.dy = dy;
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.d = d;
  a.y_stride = dx_stride;
  a.x_stride = x_stride;
  a.dy_stride = dy_stride;
  a.weight_type = weight_type;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  e = type == MP_BF16 ? backward<MP_BF16>(a, dweight, dbias, part, dev, s)
                      : type == MP_FP16 ? backward<MP_FP16>(a, dweight, dbias, part, dev, s)
                                        : backward<MP_FP32>(a, dweight, dbias, part, dev, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}
