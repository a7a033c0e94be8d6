// mp_distill.cu — distillation from a teacher's top logits: the loss and the
// gradient of the student's logits in one launch.
//
// A block takes a row: one pass over it for the sum of exponentials
// (mp_softmax.cuh), a second that writes the gradient w scale (p - q). The
// second reads the row out of L2, where the rows in flight fit (152 SMs x 4
// blocks x 256 KB at the largest), so HBM sees each logit read once and each
// gradient written once: 4 B an element for 16-bit types. The listed tokens
// (few) are corrected afterwards by one thread each. Few rows are split over
// the blocks of a cluster.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_softmax.cuh"

namespace mpk {
namespace {

namespace cg = cooperative_groups;

constexpr int kDsThreads = 256;  // at most
constexpr int kDsWarps = kDsThreads / 32;
constexpr int kMaxTeacher = 1024;
constexpr int kDsCluster = 8;

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

// The teacher's list of one row in shared memory: token (-1: unused), the
// teacher's logit and later q, and the student's logit; and a hash table of
// the tokens that finds those listed twice.
struct List {
  int32_t* token;
  float* q;
  float* z;
  int32_t* table;
  int slots;  // a power of two, at least 2 k
};

__device__ __forceinline__ float block_reduce(float v, float* red, bool maximum) {
  v = maximum ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < blockDim.x / 32; ++w) s = maximum ? max_nan(s, red[w]) : __fadd_rn(s, red[w]);
  return s;
}

// Enters token into the table; true if it was there.
__device__ __forceinline__ bool enter(const List& l, int32_t token) {
  const uint32_t mask = l.slots - 1;
  uint32_t at = (static_cast<uint32_t>(token) * 0x9E3779B1u) >> 16;
  for (int i = 0; i < l.slots; ++i, ++at) {
    const int32_t was = atomicCAS(&l.table[at & mask], -1, token);
    if (was == token) return true;
    if (was == -1) return false;
  }
  return false;
}

template <int T>
__global__ void __launch_bounds__(kDsThreads, 4) distill_kernel(DsArgs a, int slots) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank(), threads = blockDim.x;
  __shared__ RowStats red[kDsWarps];
  __shared__ RowStats mine;
  __shared__ float redf[kDsWarps];
  extern __shared__ int32_t list_memory[];
  List l;
  l.token = list_memory;
  l.q = reinterpret_cast<float*>(list_memory + a.k);
  l.z = reinterpret_cast<float*>(list_memory + 2 * a.k);
  l.table = list_memory + 3 * a.k;
  l.slots = slots;
  const float c = __fmul_rn(a.scale, kLog2E), slack = __fdiv_rn(kSlack, c);
  const int64_t teams = gridDim.x / parts;
  for (int64_t r = blockIdx.x / parts; r < a.rows; r += teams) {
    const E* x = static_cast<const E*>(a.logits) + r * a.stride;
    const E* tl = static_cast<const E*>(a.teacher) + r * a.teacher_stride;
    E* dx = a.dlogits ? static_cast<E*>(a.dlogits) + r * a.dlogits_stride : nullptr;
    const float w = a.row_weight ? a.row_weight[r] : 1.0f;
    if (w == 0.0f) {
      if (dx) zero_row<T>(RowPart<T>(dx, a.vocab, part, parts), dx);
      if (part == 0 && threadIdx.x == 0) a.loss[r] = 0.0f;
      continue;
    }
    __syncthreads();  // the last row's list is read no more
    float tm = -kInf;
    bool bad = false;
    for (int i = threadIdx.x; i < slots; i += threads) l.table[i] = -1;
    for (int i = threadIdx.x; i < a.k; i += threads) {
      const int64_t j = load_index(a.index, r * a.index_stride + i, a.index_type);
      const bool use = j >= 0 && j < a.vocab;
      bad = bad || j >= a.vocab;
      l.token[i] = use ? static_cast<int32_t>(j) : -1;
      l.q[i] = use ? Elem<T>::get(tl[i]) : -kInf;
      l.z[i] = use ? Elem<T>::get(x[j]) : 0.0f;
      tm = max_nan(tm, l.q[i]);
    }
    RowStats st;
    scan_row<T, false>(st, RowPart<T>(x, a.vocab, part, parts), c, slack, [](float) {});
    st = join_block(st, red, c);
    if (parts > 1) {
      if (threadIdx.x == 0) mine = st;
      cluster.sync();
      st = join_all(parts, c, [&](int q) { return cluster.map_shared_rank(&mine, q); });
      cluster.sync();  // before `mine`, or a logit another block still reads, is overwritten
    }
    const RowLog log(st, c, a.scale);
    // the teacher's distribution and the loss
    tm = block_reduce(tm, redf, true);
    const bool none = tm == -kInf;
    bool twice = false;
    float ts = 0.0f;
    for (int i = threadIdx.x; i < a.k; i += threads) {
      if (!none) ts = __fadd_rn(ts, exp2_fast(__fmul_rn(__fsub_rn(l.q[i], tm), c)));
      if (dx && l.token[i] >= 0) twice = enter(l, l.token[i]) || twice;
    }
    ts = block_reduce(ts, redf, false);
    const float inv_ts = __fdiv_rn(1.0f, ts), log_ts = logf(ts);
    float kl = 0.0f;
    for (int i = threadIdx.x; i < a.k; i += threads) {
      float q = 0.0f;
      if (!none) {
        const float d = __fsub_rn(l.q[i], tm);
        q = __fmul_rn(exp2_fast(__fmul_rn(d, c)), inv_ts);
        if (q != 0.0f) {
          const float log_q = __fmaf_rn(d, a.scale, -log_ts);
          kl = __fmaf_rn(q, __fsub_rn(log_q, log.log_p(l.z[i])), kl);
        }
      }
      l.q[i] = q;
    }
    kl = block_reduce(kl, redf, false);
    bad = __syncthreads_or(bad);
    twice = __syncthreads_or(twice);
    if (part == 0 && threadIdx.x == 0) {
      a.loss[r] = bad ? __int_as_float(0x7FC00000) : none ? 0.0f : __fmul_rn(w, kl);
      if (bad && a.d_status) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
    }
    if (!dx) continue;
    const RowPart<T> out(dx, a.vocab, part, parts);
    if (none || log.empty) {
      zero_row<T>(out, dx);
      continue;
    }
    const float ws = __fmul_rn(w, a.scale), A = __fdiv_rn(ws, st.s);
    map_row<T>(out, dx, x, [&](float v) { return __fmul_rn(exp2_fast(__fmul_rn(__fsub_rn(v, st.ref), c)), A); });
    __syncthreads();
    for (int i = threadIdx.x; i < a.k; i += threads) {
      const int32_t token = l.token[i];
      if (token < 0 || !out.holds(token)) continue;
      float q = l.q[i];
      if (twice) {  // the first entry of a token carries its sum, in the list's order
        bool first = true;
        for (int j = 0; j < i; ++j) first = first && l.token[j] != token;
        if (!first) continue;
        for (int j = i + 1; j < a.k; ++j)
          if (l.token[j] == token) q = __fadd_rn(q, l.q[j]);
      }
      const float t = __fmul_rn(__fsub_rn(l.z[i], st.ref), c);
      dx[token] = Elem<T>::put(__fmul_rn(ws, __fsub_rn(__fdiv_rn(exp2_fast(t), st.s), q)));
    }
  }
}

template <int T>
cudaError_t launch(const DsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t units = a.vocab / 8, step = static_cast<int64_t>(kUnits<T>) * 32;
  const int threads = static_cast<int>(std::min<int64_t>(kDsThreads, std::max<int64_t>(1, units / step) * 32));
  int parts = 1;
  while (parts < kDsCluster && a.rows * parts * 2 <= 2 * dev.sms && units / (2 * parts) >= kUnits<T> * threads / 2)
    parts *= 2;
  int slots = 2;
  while (slots < 2 * a.k) slots *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, 1 << 24) * parts));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (3 * a.k + slots) * sizeof(int32_t);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, distill_kernel<T>, a, slots);
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
