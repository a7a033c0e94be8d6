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

constexpr int kLpThreads = 128;  // that read a row, at most; see row_plan
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kSlots = 16;        // chunk maxima a thread keeps
constexpr int kCandidates = 512;  // elements a block ranks at most
constexpr int kVisits = 256;      // chunks read again at most
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

// What the threads that read a part leave of it, besides the slots.
struct PartShared {
  RowStats stats[kLpWarps];
  uint32_t lane_max[kLpWarps][32];
};

struct TopShared {
  uint64_t keys[kCandidates + kMaxTop];
  uint4 staged[32][5];       // 32 chunks read again, 64 B each
  uint16_t visits[kVisits];  // slot * 128 + thread
  uint8_t threads[kLpThreads];
};

// The chunks of a part: what `threads` threads read and keep maxima of.
struct Chunks {
  const float* slots;
  int per_slot, threads;
};

// One warp looks for the alternatives, once a row: what it runs is paid for in
// instruction fetches (none of it is in the instruction cache after a row's
// worth of the reading loop), so its loops stay rolled.

// The k-th largest of the 32 lane positions' maxima: at least k elements reach it.
__device__ __forceinline__ uint32_t lower_bound(const PartShared& sh, int warps, int k) {
  const int lane = threadIdx.x % 32;
  uint32_t mine = 0;
#pragma unroll 1
  for (int w = 0; w < warps; ++w) mine = max(mine, sh.lane_max[w][lane]);
  int rank = 0;
#pragma unroll 4
  for (int l = 0; l < 32; ++l) {
    const uint32_t other = __shfl_sync(kAll, mine, l);
    rank += other > mine || (other == mine && l < lane);
  }
  return __shfl_sync(kAll, mine, __ffs(__ballot_sync(kAll, rank == k - 1)) - 1);
}

__device__ __forceinline__ void copy16_async(void* shared, const void* global) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(shared))),
               "l"(global)
               : "memory");
}

__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Leaves the keys of the part's elements whose order is at least `bound` in
// sh.keys and returns their number. A result above kCandidates says that there
// are more, or too many chunks to look through; sh.keys then holds as many as
// fit, or those of the chunks looked through. Each lane looks through a thread's
// chunk maxima, then through a chunk that passes, 32 of them read again at a
// time by asynchronous copies.
template <int T>
__device__ __forceinline__ int collect(const RowPart<T>& p, const PartShared& ps, const Chunks& ch, uint32_t bound,
                                       TopShared& sh, int& found) {
  constexpr int U = kUnits<T>;
  const int lane = threadIdx.x % 32;
  const uint32_t below = (1u << lane) - 1;
  const int64_t step = static_cast<int64_t>(U) * ch.threads * ch.per_slot;
  const int used = static_cast<int>((p.last - p.first + step - 1) / step);
  const float least = bound ? value_of_order(bound) : -kInf;  // NaN: only NaN reaches it
  auto reaches = [&](float m) { return m >= least || m != m; };
  int readers = 0;
#pragma unroll 1
  for (int t = lane; t < ch.threads; t += 32) {
    const bool pass = ps.lane_max[t / 32][lane] >= bound;
    const uint32_t votes = __ballot_sync(kAll, pass);
    if (pass) sh.threads[readers + __popc(votes & below)] = static_cast<uint8_t>(t);
    readers += __popc(votes);
  }
  __syncwarp();
  int n = 0;
#pragma unroll 1
  for (int i = lane; i - lane < readers; i += 32) {
    const int t = i < readers ? sh.threads[i] : -1;
#pragma unroll 1
    for (int slot = 0; slot < used; ++slot) {
      const bool pass = t >= 0 && reaches(ch.slots[slot * ch.threads + t]);
      const uint32_t votes = __ballot_sync(kAll, pass);
      const int at = n + __popc(votes & below);
      if (pass && at < kVisits) sh.visits[at] = static_cast<uint16_t>(slot * kLpThreads + t);
      n += __popc(votes);
    }
  }
  __syncwarp();
  const bool over = n > kVisits;
  n = min(n, kVisits);
  auto unit_of = [&](int v, int in, int q) {
    const int visit = sh.visits[v];
    const int64_t it = static_cast<int64_t>(visit / kLpThreads) * ch.per_slot + in;
    return p.first + (it * U + q) * ch.threads + visit % kLpThreads;
  };
  int keys = 0;
  auto append = [&](bool pass, float x, int64_t j) {
    const uint32_t votes = __ballot_sync(kAll, pass);
    const int at = keys + __popc(votes & below);
    if (pass && at < kCandidates) sh.keys[at] = top_key(order_of(x), j);
    keys += __popc(votes);
  };
  constexpr int kPieces = 4 / U, kWords = 16 / U;  // 16-B pieces and 4-B words of a unit
#pragma unroll 1
  for (int v0 = 0; v0 < n; v0 += 32)
#pragma unroll 1
    for (int in = 0; in < ch.per_slot; ++in) {
      __syncwarp();
#pragma unroll 1
      for (int v = lane / 4; v < min(n - v0, 32); v += 8) {
        const int64_t unit = unit_of(v0 + v, in, lane % 4 / kPieces);
        if (unit < p.last)
          copy16_async(&sh.staged[v][lane % 4], reinterpret_cast<const uint4*>(p.body + 8 * unit) + lane % kPieces);
      }
      copy_async_wait();
      __syncwarp();
      int64_t unit = v0 + lane < n ? unit_of(v0 + lane, in, 0) : p.last;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(sh.staged[lane]);
#pragma unroll 1
      for (int q = 0; q < U; ++q, unit += ch.threads)
#pragma unroll 1
        for (int i = 0; i < kWords; ++i) {
          const bool live = unit < p.last;
          const uint32_t w = words[q * kWords + i];
          const int64_t j = p.head + 8 * unit + i * (8 / kWords);
          if (T == MP_FP32) {
            append(live && reaches(__uint_as_float(w)), __uint_as_float(w), j);
          } else {
            using H = Elem<T == MP_FP32 ? MP_BF16 : T>;
            const float lo = H::get(static_cast<uint16_t>(w)), hi = H::get(static_cast<uint16_t>(w >> 16));
            if (!__any_sync(kAll, live && (reaches(lo) || reaches(hi)))) continue;
            append(live && reaches(lo), lo, j);
            append(live && reaches(hi), hi, j + 1);
          }
        }
    }
  if (p.extra) {
    const int64_t j = p.extra_index(lane);
    const float x = lane < p.extra ? Elem<T>::get(p.row[j]) : 0.0f;
    append(lane < p.extra && reaches(x), x, j);
  }
  __syncwarp();
  found = min(keys, kCandidates);
  return over ? kCandidates + 1 : keys;
}

// The keys of the part's k largest elements (and perhaps more) in sh.keys, by
// one warp; returns their number. Out of line, so that the pass over the row
// keeps its registers.
//
// Where more elements reach the bound than there is room for, the k-th largest
// of those found is a higher bound and the chunks are looked through again; if
// it is no higher, very many elements are equal to it (masked rows, equal
// logits), and those above it are joined by the first equal ones in index order.
template <int T>
__device__ __noinline__ int find_top(const typename Elem<T>::type* row, int64_t vocab, int part, int parts, int k,
                                     const PartShared& ps, const Chunks& ch, TopShared& sh) {
  const RowPart<T> p(row, vocab, part, parts);
  const int lane = threadIdx.x % 32;
  uint32_t bound = lower_bound(ps, ch.threads / 32, k);
  int n = 0;
  for (bool strict = false;;) {
    int found;
    n = collect<T>(p, ps, ch, bound + strict, sh, found);
    if (n <= kCandidates) {
      if (!strict) return n;
      break;
    }
    // the k-th largest order of some of the keys found
    found = min(found, 128);
    uint32_t higher = bound;
    if (found >= k)
      for (int i0 = 0; i0 < found; i0 += 32) {
        const uint64_t key = i0 + lane < found ? sh.keys[i0 + lane] : 0;
        int rank = 0;
        for (int q = 0; q < found; ++q) rank += sh.keys[q] > key;
        const uint32_t votes = __ballot_sync(kAll, key != 0 && rank == k - 1);
        if (votes) higher = __shfl_sync(kAll, static_cast<uint32_t>(key >> 32), __ffs(votes) - 1);
      }
    __syncwarp();
    if (higher > bound) {
      bound = higher;
      strict = false;
    } else if (bound == 0xFFFFFFFFu) {
      n = 0;  // NaN: nothing is above it
      break;
    } else {
      strict = true;
    }
  }
  // The part's elements in index order, one per lane and round; the extra
  // elements before the units belong to it, those after them come last.
  const int above = n;
  const int64_t from = p.extra ? 0 : p.head + 8 * p.first;
  const int64_t body_end = p.head + 8 * p.last;
  const int64_t tail = p.extra ? p.extra - p.head : 0;
  const int64_t total = body_end - from + tail;
  auto element = [&](int64_t i) { return i < body_end - from ? from + i : p.head + 8 * p.units + (i - (body_end - from)); };
#pragma unroll 4
  for (int64_t i = lane; i - lane < total && n < above + k; i += 32) {
    const bool equal = i < total && order_of(Elem<T>::get(p.row[element(i)])) == bound;
    const uint32_t votes = __ballot_sync(kAll, equal);
    const int at = n + __popc(votes & ((1u << lane) - 1));
    if (equal && at < above + k) sh.keys[at] = top_key(bound, element(i));
    n += __popc(votes);
  }
  __syncwarp();
  return min(n, above + k);
}

// Calls f(rank, key) for the k largest of n keys (all different, or 0).
template <typename Team, typename F>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int k, F&& f) {
#pragma unroll 1
  for (int i = Team::thread(); i < n; i += Team::threads()) {
    const uint64_t key = keys[i];
    if (key == 0) continue;
    int rank = 0;
#pragma unroll 4
    for (int q = 0; q < n; ++q) rank += keys[q] > key;
    if (rank < k) f(rank, key);
  }
}

// One pass over the part by `threads` threads, which leave
// the statistics in ps and the chunk maxima in slots.
template <int T, bool Entropy, bool Top, typename Ahead>
__device__ __forceinline__ void read_part(const LpArgs& a, Pack8<T> (&x)[kUnits<T>], const RowPart<T>& p, int t, int threads,
                                          float c, float slack, float* slots, int per_slot, PartShared& ps,
                                          Ahead&& ahead) {
  RowStats st;
  float* slot = slots + t;
  float slot_max = -kInf;
  int left = per_slot;
  scan_row<T, Entropy>(
      st, x, p, t, threads, c, slack,
      [&](float m) {
        if (!Top) return;
        slot_max = max_nan(slot_max, m);
        *slot = slot_max;
        if (--left == 0) {
          slot += threads;
          slot_max = -kInf;
          left = per_slot;
        }
      },
      ahead);
  const bool some = p.first + t < p.last || t < p.extra;
  if (Top) ps.lane_max[t / 32][t % 32] = some ? order_of(st.m) : 0;
  st = join_warp(st);
  if (t % 32 == 0) ps.stats[t / 32] = st;
}

// A row's outputs from its statistics and its n candidates, by a team.
template <int T, bool Entropy, bool Top, typename Team>
__device__ __forceinline__ void write_row(const LpArgs& a, int64_t r, RowStats st, float c, const uint64_t* keys,
                                          int n, RowStats* red) {
  const typename Elem<T>::type* x = static_cast<const typename Elem<T>::type*>(a.logits) + r * a.stride;
  const bool difference = out_of_range(st);
  if (difference) st = difference_stats<T, Entropy, Team>(x, a.vocab, st.m, c, red);
  const RowLog log(st, difference, c, a.scale);
  if (Team::thread() == 0) {
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
    rank_keys<Team>(keys, n, a.top_k, [&](int rank, uint64_t key) {
      a.top_index[r * a.top_k + rank] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
      a.top_logp[r * a.top_k + rank] = log.log_p(value_of_order(static_cast<uint32_t>(key >> 32)));
    });
}

// The two halves of a cluster barrier, for every thread of the cluster.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Short or few rows: a block, or the blocks of a cluster, read a row and
// finish it.
template <int T, bool Entropy, bool Top>
__global__ void __launch_bounds__(kLpThreads, 8) lp_forward_kernel(LpArgs a, int per_slot) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  // The first block's shared memory may be written once that block runs and, in
  // later rows, has finished the row before: the blocks arrive here and at each
  // row's end, and wait only where they write to it.
  if (parts > 1) cluster_arrive();
  __shared__ PartShared ps;
  __shared__ RowStats part_stats[kLpCluster];                     // of the first block: every block's
  __shared__ uint64_t part_keys[Top ? kLpCluster * kMaxTop : 1];  // likewise
  __shared__ TopShared top;
  __shared__ int found;
  extern __shared__ float slots[];
  const float c = __fmul_rn(a.scale, kLog2E), slack = __fdiv_rn(kSlack, c);
  const int threads = blockDim.x;
  const int64_t teams = gridDim.x / parts;
  for (int64_t r = blockIdx.x / parts; r < a.rows; r += teams) {
    const E* x = static_cast<const E*>(a.logits) + r * a.stride;
    const RowPart<T> p(x, a.vocab, part, parts);
    Pack8<T> units[kUnits<T>];
    first_chunk(units, p, threadIdx.x, threads);
    read_part<T, Entropy, Top>(a, units, p, threadIdx.x, threads, c, slack, slots, per_slot, ps, [](auto&) {});
    __syncthreads();
    RowStats st = join_all(threads / 32, [&](int i) { return ps.stats + i; });
    int n = 0;
    if (Top) {
      if (threadIdx.x < 32) {
        n = find_top<T>(x, a.vocab, part, parts, a.top_k, ps, Chunks{slots, per_slot, threads}, top);
        if (threadIdx.x == 0) found = n;
      }
      __syncthreads();
      n = found;
    }
    const uint64_t* keys = top.keys;
    if (parts > 1) {
      cluster_wait();
      if (threadIdx.x == 0) *cluster.map_shared_rank(&part_stats[part], 0) = st;
      if (Top) {
        uint64_t* to = cluster.map_shared_rank(&part_keys[part * kMaxTop], 0);
        if (threadIdx.x >= min(n, a.top_k) && threadIdx.x < kMaxTop) to[threadIdx.x] = 0;
        rank_keys<BlockTeam>(top.keys, n, a.top_k, [&](int rank, uint64_t key) { to[rank] = key; });
      }
      cluster.sync();
      if (part == 0) {
        st = join_all(parts, [&](int q) { return part_stats + q; });
        keys = part_keys;
        n = parts * kMaxTop;
      }
    }
    if (part == 0) write_row<T, Entropy, Top, BlockTeam>(a, r, st, c, keys, n, ps.stats);
    if (r + teams < a.rows) {  // before the next row's sums go where this row's were read
      if (parts > 1) cluster_arrive();
      __syncthreads();
    }
  }
}

// Many long rows: four warps read one row after the other without a pause, the
// first warp finishes each row (all latency: joining, looking for the
// alternatives, ranking them) while they read the next. Two sets of shared
// memory change hands through named barriers: `full` when the readers have left
// a row there, `empty` when the first warp is done with it. On 8192 x 50304
// bf16 this takes 132 us with entropy (6.2 TB/s) against 146 us for blocks that
// read and finish a row each, and 197 against 204 us with 20 alternatives. Six
// blocks an SM, what its registers hold: 8192 x 32003 fp32 with 5 alternatives
// 168 us, five 179, four 204; with 2047 rows, whose last round is a quarter
// full, 56, 54 and 62.
constexpr int kLpRowThreads = kLpThreads + 32;

// Barrier `first` of set 0, `first` + 1 of set 1. The numbers are constants of
// the instructions: with one in a register a block holds all sixteen, and
// fewer blocks fit an SM.
template <int first>
__device__ __forceinline__ void barrier_sync(int set) {
  if (set)
    asm volatile("bar.sync %0, %1;" ::"n"(first + 1), "n"(kLpRowThreads) : "memory");
  else
    asm volatile("bar.sync %0, %1;" ::"n"(first), "n"(kLpRowThreads) : "memory");
}

template <int first>
__device__ __forceinline__ void barrier_arrive(int set) {
  if (set)
    asm volatile("bar.arrive %0, %1;" ::"n"(first + 1), "n"(kLpRowThreads) : "memory");
  else
    asm volatile("bar.arrive %0, %1;" ::"n"(first), "n"(kLpRowThreads) : "memory");
}

template <int T, bool Entropy, bool Top>
__global__ void __launch_bounds__(kLpRowThreads, 6) lp_rows_kernel(LpArgs a, int per_slot) {
  pdl_enter();
  using E = typename Elem<T>::type;
  constexpr int kFull = 1, kEmpty = 3;  // barriers 1, 2 and 3, 4
  __shared__ PartShared ps[2];
  __shared__ TopShared top;
  extern __shared__ float slots[];  // two sets
  const float c = __fmul_rn(a.scale, kLog2E);
  const int64_t teams = gridDim.x;
  int round = 0;
  if (threadIdx.x >= 32) {
    const int t = threadIdx.x - 32;
    const float slack = __fdiv_rn(kSlack, c);
    auto part = [&](int64_t r) {
      return RowPart<T>(static_cast<const E*>(a.logits) + r * a.stride, a.vocab, 0, 1);
    };
    Pack8<T> units[kUnits<T>];
    if (blockIdx.x < a.rows) first_chunk(units, part(blockIdx.x), t, kLpThreads);
    for (int64_t r = blockIdx.x; r < a.rows; r += teams, ++round) {
      const int set = round & 1;
      if (round >= 2) barrier_sync<kEmpty>(set);
      read_part<T, Entropy, Top>(a, units, part(r), t, kLpThreads, c, slack, slots + set * kSlots * kLpThreads, per_slot,
                                 ps[set], [&](auto& next) {
                                   if (r + teams < a.rows) first_chunk(next, part(r + teams), t, kLpThreads);
                                 });
      barrier_arrive<kFull>(set);
    }
  } else {
    for (int64_t r = blockIdx.x; r < a.rows; r += teams, ++round) {
      const int set = round & 1;
      barrier_sync<kFull>(set);
      const RowStats st = join_all(kLpWarps, [&](int i) { return ps[set].stats + i; });
      int n = 0;
      if (Top) {
        n = find_top<T>(static_cast<const E*>(a.logits) + r * a.stride, a.vocab, 0, 1, a.top_k, ps[set],
                                  Chunks{slots + set * kSlots * kLpThreads, per_slot, kLpThreads}, top);
        __syncwarp();
      }
      write_row<T, Entropy, Top, WarpTeam>(a, r, st, c, top.keys, n, nullptr);
      barrier_arrive<kEmpty>(set);
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
    // the target's element is written by one thread of the block whose part it is
    // in, from the value read before that part is overwritten
    const float xt = t >= 0 && (parts == 1 || out.holds(t)) ? Elem<T>::get(x[t]) : 0.0f;
    __syncthreads();
    auto of = [&](float v) {
      const float y = __fmaf_rn(v, scale, -lse);
      const float p = exp2_fast(__fmul_rn(y, kLog2E));
      // y is finite where p is not 0 (or NaN)
      return __fmul_rn(p, __fmaf_rn(a1, max_nan(y, kLowest), a0));
    };
    if (h == 0.0f)
      map_row<T, false>(out, dx, x, [&](float v) {
        return __fmul_rn(a0, exp2_fast(__fmul_rn(__fmaf_rn(v, scale, -lse), kLog2E)));
      });
    else
      map_row<T, false>(out, dx, x, of);
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
  bool rows_kernel;
};

RowPlan row_plan(int64_t rows, int64_t vocab, int type, const DeviceInfo& dev) {
  const int64_t chunk = type == MP_FP32 ? 16 : 32;
  RowPlan p;
  p.threads = static_cast<int>(std::min<int64_t>(kLpThreads, std::max<int64_t>(1, (vocab / chunk + 31) / 32) * 32));
  p.parts = 1;
  while (p.parts < kLpCluster && rows * p.parts * 2 <= 4 * dev.sms && vocab / (2 * p.parts) >= chunk * p.threads / 2)
    p.parts *= 2;
  p.rows_kernel = p.parts == 1 && p.threads == kLpThreads && rows >= 12 * dev.sms && vocab >= 16384;
  return p;
}

template <int T, bool Entropy, bool Top>
cudaError_t launch_forward(const LpArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const RowPlan p = row_plan(a.rows, a.vocab, T, dev);
  const int64_t per_part = (a.vocab / 8 + p.parts - 1) / p.parts + 1;
  const int64_t step = static_cast<int64_t>(kUnits<T>) * p.threads;
  const int64_t its = (per_part + step - 1) / step;
  const int per_slot = static_cast<int>((its + kSlots - 1) / kSlots);
  const size_t smem = Top ? kSlots * p.threads * sizeof(float) : 0;
  if (p.rows_kernel) {
    const int64_t grid = std::min<int64_t>(a.rows, 6 * dev.sms);
    return launch_pdl_smem(lp_rows_kernel<T, Entropy, Top>, static_cast<unsigned>(grid), kLpRowThreads, 2 * smem, s,
                           a, per_slot);
  }
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
  cfg.dynamicSmemBytes = smem;
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
