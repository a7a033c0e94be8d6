// mp_logprob.cu — log probabilities of given tokens with entropy and top
// alternatives, and their backward pass.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_rows.cuh"

namespace mpk {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 32;

struct LpArgs {
  float* logp;
  float* lse;
  float* entropy;
  float* top_logp;
  int32_t* top_index;
  const void* logits;
  const void* targets;
  int64_t rows, vocab, stride;
  float scale;
  int top_k, index_type;
  int32_t* d_status;
  // backward
  void* dlogits;
  int64_t dlogits_stride;
  const float* lse_in;
  const float* entropy_in;
  const float* dlogp;
  const float* dentropy;
};

__device__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < kLpWarps; ++w) s = max_nan(s, red[w]);
  return s;
}

__device__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < kLpWarps; ++w) s = __fadd_rn(s, red[w]);
  return s;
}

// (order of the value, complement of the index): its maximum is the largest
// value, the lowest index among equal ones.
__device__ __forceinline__ uint64_t top_key(float x, int64_t j) {
  return (static_cast<uint64_t>(order_of(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}

template <int T>
__global__ void __launch_bounds__(kLpThreads) lp_forward_kernel(LpArgs a) {
  pdl_enter();
  using E = Elem<T>;
  __shared__ float red[kLpWarps];
  __shared__ uint64_t redk[kLpWarps];
  const float c = __fmul_rn(a.scale, kLog2E);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const typename E::type* x = static_cast<const typename E::type*>(a.logits) + r * a.stride;
    float m = -kInf;
    for (int64_t j = threadIdx.x; j < a.vocab; j += kLpThreads) m = max_nan(m, E::get(x[j]));
    m = block_max(m, red);
    const bool empty = m == -kInf;
    float s = 0.0f, u = 0.0f;
    if (!empty)
      for (int64_t j = threadIdx.x; j < a.vocab; j += kLpThreads) {
        const float t = __fmul_rn(__fsub_rn(E::get(x[j]), m), c);
        const float e = exp2_fast(t);
        s = __fadd_rn(s, e);
        if (e != 0.0f) u = __fmaf_rn(e, t, u);
      }
    s = block_sum(s, red);
    u = block_sum(u, red);
    const float log_s = logf(s);
    const float lse = empty ? -kInf : __fadd_rn(__fmul_rn(m, a.scale), log_s);
    if (threadIdx.x == 0) {
      if (a.lse) a.lse[r] = lse;
      if (a.entropy) a.entropy[r] = empty ? 0.0f : __fsub_rn(log_s, __fmul_rn(__fdiv_rn(u, s), kLn2));
      if (a.logp) {
        const int64_t t = load_index(a.targets, r, a.index_type);
        float v = 0.0f;
        if (t >= a.vocab) {
          v = __int_as_float(0x7FC00000);
          if (a.d_status) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
        } else if (t >= 0) {
          v = empty ? -kInf : __fmaf_rn(__fsub_rn(E::get(x[t]), m), a.scale, -log_s);
        }
        a.logp[r] = v;
      }
    }
    uint64_t last = ~uint64_t{0};
    for (int k = 0; k < a.top_k; ++k) {
      uint64_t best = 0;
      for (int64_t j = threadIdx.x; j < a.vocab; j += kLpThreads) {
        const uint64_t key = top_key(E::get(x[j]), j);
        if (key < last && key > best) best = key;
      }
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(kAll, best, o);
        best = other > best ? other : best;
      }
      __syncthreads();
      if (threadIdx.x % 32 == 0) redk[threadIdx.x / 32] = best;
      __syncthreads();
      for (int w = 0; w < kLpWarps; ++w) best = redk[w] > best ? redk[w] : best;
      last = best;
      if (threadIdx.x == 0) {
        const uint32_t j = 0xFFFFFFFFu - static_cast<uint32_t>(best);
        a.top_index[r * a.top_k + k] = static_cast<int32_t>(j);
        a.top_logp[r * a.top_k + k] = empty ? -kInf : __fmaf_rn(__fsub_rn(E::get(x[j]), m), a.scale, -log_s);
      }
    }
  }
}

template <int T>
__global__ void __launch_bounds__(kLpThreads) lp_backward_kernel(LpArgs a) {
  pdl_enter();
  using E = Elem<T>;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const typename E::type* x = static_cast<const typename E::type*>(a.logits) + r * a.stride;
    typename E::type* dx = static_cast<typename E::type*>(a.dlogits) + r * a.dlogits_stride;
    const float lse = a.lse_in[r];
    int64_t t = a.targets ? load_index(a.targets, r, a.index_type) : -1;
    if (t >= a.vocab) {
      if (a.d_status && threadIdx.x == 0) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
      t = -1;
    }
    const float g = t >= 0 ? a.dlogp[r] : 0.0f;
    const float h = a.dentropy ? a.dentropy[r] : 0.0f;
    const float ent = a.dentropy ? a.entropy_in[r] : 0.0f;
    const bool zero = (g == 0.0f && h == 0.0f) || lse == -kInf;
    // dx / scale = p (-g - h (ent + log p)) + g [j = t]; log p = scale x - lse is
    // rounded once, so its error is relative to log p, small where p is large
    const float a0 = __fsub_rn(-g, __fmul_rn(h, ent));
    for (int64_t j = threadIdx.x; j < a.vocab; j += kLpThreads) {
      float v = 0.0f;
      if (!zero) {
        const float y = __fmaf_rn(E::get(x[j]), a.scale, -lse);
        const float p = exp2_fast(__fmul_rn(y, kLog2E));
        v = p == 0.0f ? 0.0f : __fmul_rn(p, __fmaf_rn(-h, y, a0));
        if (j == t) v = __fadd_rn(v, g);
        v = __fmul_rn(v, a.scale);
      }
      dx[j] = E::put(v);
    }
  }
}

template <int T>
cudaError_t forward(const LpArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  return launch_pdl(lp_forward_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 8 * dev.sms)), kLpThreads,
                    s, a);
}

template <int T>
cudaError_t backward(const LpArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  return launch_pdl(lp_backward_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 8 * dev.sms)), kLpThreads,
                    s, a);
}

}  // namespace
}  // namespace mpk

extern "C" int mp_token_logprob_forward(float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_index,
                                        const void* logits, const void* targets, int64_t rows, int64_t vocab,
                                        int64_t stride, float scale, int32_t top_k, int32_t type,
                                        int32_t index_type, int32_t* d_status, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !index_type_ok(index_type) || !rows_ok(rows) || !vocab_ok(vocab) ||
      !stride_ok(stride, vocab) || !scale_ok(scale) || top_k < 0 || top_k > kMaxTop || top_k > vocab)
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!logits || (logp == nullptr) != (targets == nullptr) || (top_k > 0 && (!top_logp || !top_index)) ||
      (!logp && !lse && !entropy && top_k == 0))
    return MP_ERR_NULL;
  if (!type_aligned(logits, type) || !index_aligned(targets, index_type) || !aligned4(logp) || !aligned4(lse) ||
      !aligned4(entropy) || !aligned4(top_logp) || !aligned4(top_index) || !aligned4(d_status))
    return MP_ERR_ALIGN;
  DeviceInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return record_cuda_error(e);
  LpArgs a = {};
  a.logp = logp;
  a.lse = lse;
  a.entropy = entropy;
  a.top_logp = top_logp;
  a.top_index = top_index;
  a.logits = logits;
  a.targets = targets;
  a.rows = rows;
  a.vocab = vocab;
  a.stride = stride;
  a.scale = scale;
  a.top_k = top_k;
  a.index_type = index_type;
  a.d_status = d_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = type == MP_BF16 ? forward<MP_BF16>(a, dev, s)
                      : type == MP_FP16 ? forward<MP_FP16>(a, dev, s) : forward<MP_FP32>(a, dev, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}

extern "C" int mp_token_logprob_backward(void* dlogits, const void* logits, const void* targets, const float* lse,
                                         const float* entropy, const float* dlogp, const float* dentropy,
                                         int64_t rows, int64_t vocab, int64_t dlogits_stride, int64_t stride,
                                         float scale, int32_t type, int32_t index_type, int32_t* d_status,
                                         void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !index_type_ok(index_type) || !rows_ok(rows) || !vocab_ok(vocab) ||
      !stride_ok(stride, vocab) || !stride_ok(dlogits_stride, vocab) || !scale_ok(scale))
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!dlogits || !logits || !lse || (dlogp == nullptr) != (targets == nullptr) ||
      (entropy == nullptr) != (dentropy == nullptr) || (!dlogp && !dentropy))
    return MP_ERR_NULL;
  if (dlogits == logits && dlogits_stride != stride) return MP_ERR_RANGE;
  if (!type_aligned(dlogits, type) || !type_aligned(logits, type) || !index_aligned(targets, index_type) ||
      !aligned4(lse) || !aligned4(entropy) || !aligned4(dlogp) || !aligned4(dentropy) || !aligned4(d_status))
    return MP_ERR_ALIGN;
  DeviceInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return record_cuda_error(e);
  LpArgs a = {};
  a.dlogits = dlogits;
  a.logits = logits;
  a.targets = targets;
  a.lse_in = lse;
  a.entropy_in = entropy;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.rows = rows;
  a.vocab = vocab;
  a.dlogits_stride = dlogits_stride;
  a.stride = stride;
  a.scale = scale;
  a.index_type = index_type;
  a.d_status = d_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = type == MP_BF16 ? backward<MP_BF16>(a, dev, s)
                      : type == MP_FP16 ? backward<MP_FP16>(a, dev, s) : backward<MP_FP32>(a, dev, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}
