// mp_logprob.cu — log probabilities of given tokens with entropy and top
// alternatives, and their backward pass.
//
// Forward: one pass over the logits (mp_softmax.cuh), so 2 B an element from
// HBM for 16-bit logits is the floor. Few rows are split over the blocks of a
// cluster, which join their statistics and candidates in the first block's
// shared memory.
//
// Alternatives: the pass keeps the maximum of each chunk (32 or 16 elements)
// a thread reads. The k-th largest of 32 maxima, each over one lane position
// of the block's warps, bounds the k-th largest element from below, and only
// chunks whose maximum reaches it are read again (about k of them): so the
// pass itself pays one comparison per 32 elements for them.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_softmax.cuh"

namespace mpk {
namespace {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 128;  // at most; see row_plan
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kSlots = 16;        // chunk maxima a thread keeps
constexpr int kCandidates = 512;  // elements a block ranks without the slow form
constexpr int kVisits = 64;       // chunks a warp reads again without it
constexpr int kLpCluster = 8;     // blocks a row is split over at most

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

// (order of the value, complement of the index): its maximum is the largest
// value, the lowest index among equal ones. 0 is below every element's key.
__device__ __forceinline__ uint64_t top_key(uint32_t order, int64_t j) {
  return (static_cast<uint64_t>(order) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}

struct TopShared {
  uint32_t lane_max[kLpWarps][32];
  uint64_t keys[kCandidates + kMaxTop];
  uint64_t warp_key[kLpWarps];
  int warp_count[kLpWarps];
  uint16_t visits[kLpWarps][kVisits];  // slot * 128 + thread
  int count;
};

// The k-th largest of the 32 lane positions' maxima, to every thread: at least
// k elements reach it.
__device__ __forceinline__ uint32_t lower_bound(const TopShared& sh, int k) {
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
  uint32_t mine = 0;
  for (int w = 0; w < warps; ++w) mine = max(mine, sh.lane_max[w][lane]);
  int rank = 0;
#pragma unroll
  for (int l = 0; l < 32; ++l) {
    const uint32_t other = __shfl_sync(kAll, mine, l);
    rank += other > mine || (other == mine && l < lane);
  }
  return __shfl_sync(kAll, mine, __ffs(__ballot_sync(kAll, rank == k - 1)) - 1);
}

// Appends the keys of elements whose order is at least `bound` to sh.keys
// (sh.count of them): one warp, for the chunks that threads t0 .. t0 + nt - 1
// read. A count above kCandidates says that there are more, or too many chunks
// to look through. A lane reads a unit of a chunk again, so a warp has eight
// chunks (16 for fp32) in flight with one load.
template <int T>
__device__ __forceinline__ void collect(const RowPart<T>& p, const float* slots, int per_slot, uint32_t bound, int t0,
                                        int nt, int threads, uint16_t* visits, TopShared& sh) {
  constexpr int U = kUnits<T>, kAtOnce = 32 / U;
  const int lane = threadIdx.x % 32;
  const int64_t step = static_cast<int64_t>(U) * threads * per_slot;
  const int used = static_cast<int>((p.last - p.first + step - 1) / step);
  const float least = bound ? value_of_order(bound) : -kInf;  // NaN: only NaN reaches it
  int n = 0;
  for (int slot = 0; slot < used; ++slot)
    for (int t = t0 + lane; t < t0 + nt; t += 32) {
      const float m = slots[slot * threads + t];
      const bool pass = m >= least || m != m;
      const uint32_t votes = __ballot_sync(kAll, pass);
      const int at = n + __popc(votes & ((1u << lane) - 1));
      if (pass && at < kVisits) visits[at] = static_cast<uint16_t>(slot * kLpThreads + t);
      n += __popc(votes);
    }
  __syncwarp();
  if (n > kVisits) {
    if (lane == 0) atomicAdd(&sh.count, kCandidates + 1);
    return;
  }
  auto append = [&](uint32_t order, int64_t j) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCandidates) sh.keys[at] = top_key(order, j);
  };
  if (t0 == 0 && lane < p.extra) {
    const int64_t j = p.extra_index(lane);
    const uint32_t order = order_of(Elem<T>::get(p.row[j]));
    if (order >= bound) append(order, j);
  }
  for (int v0 = 0; v0 < n; v0 += kAtOnce)
    for (int in = 0; in < per_slot; ++in) {
      const int v = v0 + lane / U, visit = visits[min(v, n - 1)];
      const int64_t it = static_cast<int64_t>(visit / kLpThreads) * per_slot + in;
      const int64_t unit = p.first + (it * U + lane % U) * threads + visit % kLpThreads;
      Pack8<T> x[1];
      if (v >= n || unit >= p.last) continue;
      x[0].load(p.body + 8 * unit);
      const float top = max_of<T, 1>(x);
      if (!(top >= least || top != top)) continue;
      float f[8];
      x[0].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t order = order_of(f[e]);
        if (order >= bound) append(order, p.head + 8 * unit + e);
      }
    }
}

// Where too many elements reach the bound (masked rows, equal logits): leaves
// the keys of the part's k largest elements (and perhaps more) in sh.keys and
// returns their number, to every thread.
template <int T>
__device__ __noinline__ int find_among_many(const RowPart<T>& p, int k, const float* slots, int per_slot,
                                            uint32_t bound, TopShared& sh) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  // those above the bound, then the first of the equal ones in index order
  int n = kCandidates + 1;
  if (bound != 0xFFFFFFFFu) {
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    collect<T>(p, slots, per_slot, bound + 1, 32 * warp, 32, blockDim.x, sh.visits[warp], sh);
    __syncthreads();
    n = sh.count;
  }
  const int above = n;
  // The part's elements in index order, one per thread and round; the extra
  // elements before the units belong to it, those after them come last.
  const int64_t from = p.extra ? 0 : p.head + 8 * p.first;
  const int64_t body_end = p.head + 8 * p.last;
  const int64_t tail = p.extra ? p.extra - p.head : 0;
  const int64_t total = body_end - from + tail;
  auto element = [&](int64_t i) { return i < body_end - from ? from + i : p.head + 8 * p.units + (i - (body_end - from)); };
  if (bound != 0xFFFFFFFFu && n <= kCandidates) {
    for (int64_t base = 0; base < total && n < kCandidates + kMaxTop; base += blockDim.x) {
      const int64_t i = base + threadIdx.x;
      const bool equal = i < total && order_of(Elem<T>::get(p.row[element(i)])) == bound;
      const uint32_t votes = __ballot_sync(kAll, equal);
      if (lane == 0) sh.warp_count[warp] = __popc(votes);
      __syncthreads();
      int at = n + __popc(votes & ((1u << lane) - 1));
      int sum = 0;
      for (int w = 0; w < warps; ++w) {
        if (w < warp) at += sh.warp_count[w];
        sum += sh.warp_count[w];
      }
      if (equal && at < kCandidates + kMaxTop) sh.keys[at] = top_key(bound, element(i));
      n = min(n + sum, kCandidates + kMaxTop);
      __syncthreads();
      if (above + k <= n) break;
    }
    return n;
  }
  // Very many above the bound (or NaN): the largest key below the last one, k times.
  uint64_t last = ~uint64_t{0};
  for (int q = 0; q < k; ++q) {
    uint64_t best = 0;
    for (int64_t i = threadIdx.x; i < total; i += blockDim.x) {
      const uint64_t key = top_key(order_of(Elem<T>::get(p.row[element(i)])), element(i));
      if (key < last && key > best) best = key;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(kAll, best, o);
      best = other > best ? other : best;
    }
    __syncthreads();
    if (lane == 0) sh.warp_key[warp] = best;
    __syncthreads();
    for (int w = 0; w < warps; ++w) best = sh.warp_key[w] > best ? sh.warp_key[w] : best;
    if (threadIdx.x == 0) sh.keys[q] = best;
    last = best;
  }
  __syncthreads();
  return k;
}

// The keys of the part's k largest elements (and perhaps more), in sh.keys;
// their number, to every thread. sh.lane_max is filled and sh.count 0. Out of
// line, so that the pass over the row keeps its registers.
template <int T>
__device__ __noinline__ int find_top(const typename Elem<T>::type* row, int64_t vocab, int part, int parts, int k,
                                     const float* slots, int per_slot, TopShared& sh) {
  const RowPart<T> p(row, vocab, part, parts);
  const uint32_t bound = lower_bound(sh, k);
  const int warp = threadIdx.x / 32;
  collect<T>(p, slots, per_slot, bound, 32 * warp, 32, blockDim.x, sh.visits[warp], sh);
  __syncthreads();
  const int n = sh.count;
  return n <= kCandidates ? n : find_among_many<T>(p, k, slots, per_slot, bound, sh);
}

// Calls f(rank, key) for the k largest of n keys (all different, or 0).
template <typename F>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int k, F&& f) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const uint64_t key = keys[i];
    if (key == 0) continue;
    int rank = 0;
    for (int q = 0; q < n; ++q) rank += keys[q] > key;
    if (rank < k) f(rank, key);
  }
}

template <int T, bool Entropy, bool Top>
__global__ void __launch_bounds__(kLpThreads, 8) lp_forward_kernel(LpArgs a, int per_slot) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  __shared__ RowStats red[kLpWarps];
  __shared__ RowStats part_stats[kLpCluster];                       // of the first block: every block's
  __shared__ uint64_t part_keys[Top ? kLpCluster * kMaxTop : 1];    // likewise
  __shared__ TopShared top;
  extern __shared__ float slots[];
  const float c = __fmul_rn(a.scale, kLog2E), slack = __fdiv_rn(kSlack, c);
  const int threads = blockDim.x;
  const int64_t teams = gridDim.x / parts;
  for (int64_t r = blockIdx.x / parts; r < a.rows; r += teams) {
    const E* x = static_cast<const E*>(a.logits) + r * a.stride;
    const RowPart<T> p(x, a.vocab, part, parts);
    RowStats st;
    if (Top && threadIdx.x == 0) top.count = 0;
    float* slot = slots + threadIdx.x;
    float slot_max = -kInf;
    int left = per_slot;
    scan_row<T, Entropy>(st, p, c, slack, [&](float m) {
      if (!Top) return;
      slot_max = max_nan(slot_max, m);
      *slot = slot_max;
      if (--left == 0) {
        slot += threads;
        slot_max = -kInf;
        left = per_slot;
      }
    });
    const bool some = p.first + threadIdx.x < p.last || threadIdx.x < p.extra;
    const uint32_t thread_max = some ? order_of(st.m) : 0;
    const int warp = threadIdx.x / 32;
    st = join_warp(st);
    if (threadIdx.x % 32 == 0) red[warp] = st;
    if (Top) top.lane_max[warp][threadIdx.x % 32] = thread_max;
    __syncthreads();
    st = join_all(threads / 32, [&](int i) { return red + i; });
    int n = 0;
    if (Top) {
      n = find_top<T>(x, a.vocab, part, parts, a.top_k, slots, per_slot, top);
    }
    const uint64_t* keys = top.keys;
    if (parts > 1) {
      if (threadIdx.x == 0) *cluster.map_shared_rank(&part_stats[part], 0) = st;
      if (Top) {
        uint64_t* to = cluster.map_shared_rank(&part_keys[part * kMaxTop], 0);
        if (threadIdx.x >= min(n, a.top_k) && threadIdx.x < kMaxTop) to[threadIdx.x] = 0;
        rank_keys(top.keys, n, a.top_k, [&](int rank, uint64_t key) { to[rank] = key; });
      }
      cluster.sync();
      if (part == 0) {
        st = join_all(parts, [&](int q) { return part_stats + q; });
        keys = part_keys;
        n = parts * kMaxTop;
      }
    }
    if (part == 0) {
      const bool plain = out_of_range(st);
      if (plain) st = plain_stats<T, Entropy>(x, a.vocab, st.m, c, red);
      const RowLog log(st, plain, c, a.scale);
      if (threadIdx.x == 0) {
        if (a.lse) a.lse[r] = log.lse;
        if (Entropy) a.entropy[r] = log.entropy;
        if (a.logp) {
          const int64_t t = load_index(a.targets, r, a.index_type);
          float v = 0.0f;
          if (t >= a.vocab) {
            v = __int_as_float(0x7FC00000);
            if (a.d_status) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
          } else if (t >= 0) {
            v = log.log_p(Elem<T>::get(x[t]));
          }
          a.logp[r] = v;
        }
      }
      if (Top)
        rank_keys(keys, n, a.top_k, [&](int rank, uint64_t key) {
          a.top_index[r * a.top_k + rank] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
          a.top_logp[r * a.top_k + rank] = log.log_p(value_of_order(static_cast<uint32_t>(key >> 32)));
        });
    }
    if (r + teams < a.rows) {  // before the next row's sums go where this row's were read
      if (parts > 1) cluster.sync();
      __syncthreads();
    }
  }
}

// ---- backward ---------------------------------------------------------------
// dx / scale = p (-g - h (entropy + log p)) + g [j = target], for dlogp = g and
// dentropy = h: elementwise, 4 B an element for 16-bit types. log p =
// scale x - lse is rounded once, so its error is relative to log p, small
// where p is large. A row is divided over `parts` blocks.
template <int T>
__global__ void __launch_bounds__(kLpThreads) lp_backward_kernel(LpArgs a, int parts) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const int part = blockIdx.x % parts;
  const int64_t teams = gridDim.x / parts;
  for (int64_t r = blockIdx.x / parts; r < a.rows; r += teams) {
    const E* x = static_cast<const E*>(a.logits) + r * a.stride;
    E* dx = static_cast<E*>(a.dlogits) + r * a.dlogits_stride;
    const RowPart<T> out(dx, a.vocab, part, parts);
    const float lse = a.lse_in[r], scale = a.scale;
    int64_t t = a.targets ? load_index(a.targets, r, a.index_type) : -1;
    if (t >= a.vocab) {
      if (a.d_status && threadIdx.x == 0) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
      t = -1;
    }
    const float g = t >= 0 ? a.dlogp[r] : 0.0f;
    const float h = a.dentropy ? a.dentropy[r] : 0.0f;
    if ((g == 0.0f && h == 0.0f) || lse == -kInf) {
      zero_row<T>(out, dx);
      continue;
    }
    const float a0 = __fmul_rn(-scale, __fmaf_rn(h, a.dentropy ? a.entropy_in[r] : 0.0f, g));
    const float a1 = __fmul_rn(-scale, h);
    // the target's element is written by one thread, from the value read before the row is overwritten
    const float xt = t >= 0 ? Elem<T>::get(x[t]) : 0.0f;
    __syncthreads();
    auto of = [&](float v) {
      const float y = __fmaf_rn(v, scale, -lse);
      const float p = exp2_fast(__fmul_rn(y, kLog2E));
      // y is finite where p is not 0 (or NaN)
      return __fmul_rn(p, __fmaf_rn(a1, max_nan(y, kLowest), a0));
    };
    if (h == 0.0f)
      map_row<T>(out, dx, x, [&](float v) {
        return __fmul_rn(a0, exp2_fast(__fmul_rn(__fmaf_rn(v, scale, -lse), kLog2E)));
      });
    else
      map_row<T>(out, dx, x, of);
    __syncthreads();
    if (t >= 0 && threadIdx.x == 0 && out.holds(t)) dx[t] = Elem<T>::put(__fmaf_rn(g, scale, of(xt)));
  }
}

// Threads of a block and blocks of a row. A thread should have at least one
// chunk. Blocks of 128 threads, eight an SM, hide the end of a row (joining
// and ranking, all latency) behind other rows better than fewer larger ones,
// and pay it less often than more smaller ones: 8192 x 50304 bf16 with entropy
// and 20 alternatives took 222 us with 128 threads, 252 with 256, 339 with 64.
// Rows are split over a cluster while that leaves the grid short of four
// blocks an SM and each block with half a chunk a thread.
struct RowPlan {
  int threads, parts;
};

RowPlan row_plan(int64_t rows, int64_t vocab, int type, const DeviceInfo& dev) {
  const int64_t chunk = type == MP_FP32 ? 16 : 32;
  RowPlan p;
  p.threads = static_cast<int>(std::min<int64_t>(kLpThreads, std::max<int64_t>(1, (vocab / chunk + 31) / 32) * 32));
  p.parts = 1;
  while (p.parts < kLpCluster && rows * p.parts * 2 <= 4 * dev.sms && vocab / (2 * p.parts) >= chunk * p.threads / 2)
    p.parts *= 2;
  return p;
}

template <int T, bool Entropy, bool Top>
cudaError_t launch_forward(const LpArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const RowPlan p = row_plan(a.rows, a.vocab, T, dev);
  const int64_t per_part = (a.vocab / 8 + p.parts - 1) / p.parts + 1;
  const int64_t step = static_cast<int64_t>(kUnits<T>) * p.threads;
  const int64_t its = (per_part + step - 1) / step;
  const int per_slot = static_cast<int>((its + kSlots - 1) / kSlots);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, 1 << 24) * p.parts));
  cfg.blockDim = dim3(p.threads);
  cfg.dynamicSmemBytes = Top ? kSlots * p.threads * sizeof(float) : 0;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, lp_forward_kernel<T, Entropy, Top>, a, per_slot);
}

template <int T>
cudaError_t forward(const LpArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.entropy) return a.top_k ? launch_forward<T, true, true>(a, dev, s) : launch_forward<T, true, false>(a, dev, s);
  return a.top_k ? launch_forward<T, false, true>(a, dev, s) : launch_forward<T, false, false>(a, dev, s);
}

template <int T>
cudaError_t backward(const LpArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t units = a.vocab / 8, step = static_cast<int64_t>(kUnits<T>) * 32;
  const int threads = static_cast<int>(std::min<int64_t>(kLpThreads, std::max<int64_t>(1, units / step) * 32));
  int parts = 1;
  while (parts < 64 && a.rows * parts < 4 * dev.sms && units / (2 * parts) >= kUnits<T> * threads / 2) parts *= 2;
  return launch_pdl(lp_backward_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 1 << 24) * parts),
                    static_cast<unsigned>(threads), s, a, parts);
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
