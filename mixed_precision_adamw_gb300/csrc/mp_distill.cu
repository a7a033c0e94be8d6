// mp_distill.cu — distillation from a teacher's top logits: the loss and the
// gradient of the student's logits in one launch.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_rows.cuh"

namespace mpk {
namespace {

constexpr int kDsThreads = 256;
constexpr int kDsWarps = kDsThreads / 32;
constexpr int kMaxTeacher = 1024;

struct DsArgs {
  float* loss;
  void* dlogits;  // nullptr: the loss alone
  const void* logits;
  const void* teacher;
  const void* index;
  const float* row_weight;
  int64_t rows, vocab, dlogits_stride, stride, teacher_stride, index_stride;
  float scale;
  int k, index_type;
  int32_t* d_status;
};

__device__ float block_reduce(float v, float* red, bool maximum) {
  v = maximum ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < kDsWarps; ++w) s = maximum ? max_nan(s, red[w]) : __fadd_rn(s, red[w]);
  return s;
}

template <int T>
__global__ void __launch_bounds__(kDsThreads) distill_kernel(DsArgs a) {
  pdl_enter();
  using E = Elem<T>;
  __shared__ float red[kDsWarps];
  __shared__ int32_t at[kMaxTeacher];
  __shared__ float q[kMaxTeacher], z[kMaxTeacher];
  const float c = __fmul_rn(a.scale, kLog2E);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const typename E::type* x = static_cast<const typename E::type*>(a.logits) + r * a.stride;
    const typename E::type* tl = static_cast<const typename E::type*>(a.teacher) + r * a.teacher_stride;
    typename E::type* dx = a.dlogits ? static_cast<typename E::type*>(a.dlogits) + r * a.dlogits_stride : nullptr;
    const float w = a.row_weight ? a.row_weight[r] : 1.0f;
    if (w == 0.0f) {
      if (dx)
        for (int64_t j = threadIdx.x; j < a.vocab; j += kDsThreads) dx[j] = E::put(0.0f);
      if (threadIdx.x == 0) a.loss[r] = 0.0f;
      continue;
    }
    // the teacher's list: q in (0, 1], 0 for unused entries
    __syncthreads();
    float tm = -kInf;
    bool bad = false;
    for (int i = threadIdx.x; i < a.k; i += kDsThreads) {
      const int64_t j = load_index(a.index, r * a.index_stride + i, a.index_type);
      const bool use = j >= 0 && j < a.vocab;
      bad = bad || j >= a.vocab;
      at[i] = use ? static_cast<int32_t>(j) : -1;
      q[i] = use ? E::get(tl[i]) : -kInf;
      z[i] = use ? E::get(x[j]) : 0.0f;
      tm = max_nan(tm, q[i]);
    }
    tm = block_reduce(tm, red, true);
    bad = __syncthreads_or(bad);
    const bool none = tm == -kInf;
    float ts = 0.0f;
    if (!none)
      for (int i = threadIdx.x; i < a.k; i += kDsThreads)
        ts = __fadd_rn(ts, exp2_fast(__fmul_rn(__fsub_rn(q[i], tm), c)));
    ts = block_reduce(ts, red, false);
    // the student's maximum and sum
    float m = -kInf;
    for (int64_t j = threadIdx.x; j < a.vocab; j += kDsThreads) m = max_nan(m, E::get(x[j]));
    m = block_reduce(m, red, true);
    const bool empty = m == -kInf;
    float s = 0.0f;
    if (!empty)
      for (int64_t j = threadIdx.x; j < a.vocab; j += kDsThreads)
        s = __fadd_rn(s, exp2_fast(__fmul_rn(__fsub_rn(E::get(x[j]), m), c)));
    s = block_reduce(s, red, false);
    // loss = sum q (log q - z + lse), z and lse taken from m, in log2 units
    const float log2_s = log2f(s), log2_ts = log2f(ts);
    float kl = 0.0f;
    if (!none)
      for (int i = threadIdx.x; i < a.k; i += kDsThreads) {
        const float lt = __fsub_rn(__fmul_rn(__fsub_rn(q[i], tm), c), log2_ts);
        const float p = exp2_fast(lt);
        if (p != 0.0f) {
          const float lz = empty ? -kInf : __fsub_rn(__fmul_rn(__fsub_rn(z[i], m), c), log2_s);
          kl = __fmaf_rn(p, __fsub_rn(lt, lz), kl);
        }
        q[i] = p;
      }
    kl = block_reduce(kl, red, false);
    if (threadIdx.x == 0) {
      a.loss[r] = bad ? __int_as_float(0x7FC00000) : none ? 0.0f : __fmul_rn(w, __fmul_rn(kl, kLn2));
      if (bad && a.d_status) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
    }
    if (!dx) continue;
    const float ws = __fmul_rn(w, a.scale);
    const float inv = __fdiv_rn(1.0f, s);
    const bool zero = none || empty;
    for (int64_t j = threadIdx.x; j < a.vocab; j += kDsThreads) {
      float v = 0.0f;
      if (!zero) {
        v = __fmul_rn(exp2_fast(__fmul_rn(__fsub_rn(E::get(x[j]), m), c)), inv);
        for (int i = 0; i < a.k; ++i)
          if (at[i] == j) v = __fsub_rn(v, q[i]);
        v = __fmul_rn(v, ws);
      }
      dx[j] = E::put(v);
    }
  }
}

template <int T>
cudaError_t launch(const DsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  return launch_pdl(distill_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 8 * dev.sms)), kDsThreads, s,
                    a);
}

}  // namespace
}  // namespace mpk

extern "C" int mp_distill_topk(float* loss, void* dlogits, const void* logits, const void* teacher, const void* index,
                               const float* row_weight, int64_t rows, int64_t vocab, int32_t k,
                               int64_t dlogits_stride, int64_t stride, int64_t teacher_stride, int64_t index_stride,
                               float scale, int32_t type, int32_t index_type, int32_t* d_status, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !index_type_ok(index_type) || !rows_ok(rows) || !vocab_ok(vocab) ||
      !stride_ok(stride, vocab) || (dlogits && !stride_ok(dlogits_stride, vocab)) || !scale_ok(scale) || k < 1 ||
      k > kMaxTeacher || !stride_ok(teacher_stride, k) || !stride_ok(index_stride, k))
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!loss || !logits || !teacher || !index) return MP_ERR_NULL;
  if (dlogits == logits && dlogits_stride != stride) return MP_ERR_RANGE;
  if (!type_aligned(dlogits, type) || !type_aligned(logits, type) || !type_aligned(teacher, type) ||
      !index_aligned(index, index_type) || !aligned4(loss) || !aligned4(row_weight) || !aligned4(d_status))
    return MP_ERR_ALIGN;
  DeviceInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return record_cuda_error(e);
  const DsArgs a = {loss, dlogits, logits, teacher, index, row_weight, rows, vocab, dlogits_stride, stride,
                    teacher_stride, index_stride, scale, k, index_type, d_status};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = type == MP_BF16 ? launch<MP_BF16>(a, dev, s)
                      : type == MP_FP16 ? launch<MP_FP16>(a, dev, s) : launch<MP_FP32>(a, dev, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}
