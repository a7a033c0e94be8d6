// mp_distill.cu — distillation from a teacher's top logits: the loss and the
// gradient of the student's logits in one launch.
//
// A block takes a row: one pass over it for the sum of exponentials
// (mp_softmax.cuh), a second that writes the gradient w scale (p - q). The
// second reads the row out of L2 where the rows in flight fit (6 blocks an SM,
// 91 MB at 50304 logits of 16 bits), so that HBM sees each logit read once and
// each gradient written once: 4 B an element for 16-bit types. The listed
// tokens (few) are corrected afterwards by one thread each. Six blocks an SM
// leave a thread 80 registers, and 36 to 64 bytes of it spill. Few rows are split
// over the blocks of a cluster. Many long rows take the ring below, which holds
// most of a row in shared memory instead (8192 x 50304 bf16: 339 us).
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_softmax.cuh"
#include "mp_tma.cuh"

namespace mpk {
namespace {

namespace cg = cooperative_groups;

constexpr int kDsThreads = 128;  // at most
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
__device__ __forceinline__ bool enter(const List& l, int32_t token) {  // the table is at most half full
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
__global__ void __launch_bounds__(kDsThreads, 6) distill_kernel(DsArgs a, int slots) {
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
    const RowPart<T> in(x, a.vocab, part, parts);
    Pack8<T> units[kUnits<T>];
    first_chunk(units, in, threadIdx.x, threads);  // on its way while the list is read
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
    scan_row<T, false>(st, units, in, threadIdx.x, threads, c, slack, [](float) {}, [](auto&) {});
    st = join_block(st, red);
    if (parts > 1) {
      if (threadIdx.x == 0) mine = st;
      cluster.sync();
      st = join_all(parts, [&](int q) { return cluster.map_shared_rank(&mine, q); });
      cluster.sync();  // before `mine`, or a logit another block still reads, is overwritten
    }
    const bool difference = out_of_range(st);
    if (difference) {
      st = difference_stats<T, false, BlockTeam>(x, a.vocab, st.m, c, red);
      if (parts > 1) cluster.sync();  // every block has read the row
    }
    const RowLog log(st, difference, c, a.scale);
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
          // times w first: at the lowest fp32 logit the sum alone would be beyond fp32
          kl = __fmaf_rn(__fmul_rn(w, q), __fsub_rn(log_q, log.log_p(l.z[i])), kl);
        }
      }
      l.q[i] = q;
    }
    kl = block_reduce(kl, redf, false);
    bad = __syncthreads_or(bad);
    twice = __syncthreads_or(twice);
    if (part == 0 && threadIdx.x == 0) {
      a.loss[r] = bad ? __int_as_float(0x7FC00000) : none ? 0.0f : kl;
      if (bad && a.d_status) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
    }
    if (!dx) continue;
    const RowPart<T> out(dx, a.vocab, part, parts);
    if (none || log.empty) {
      zero_row<T>(out, dx);
      continue;
    }
    const float ws = __fmul_rn(w, a.scale), A = __fdiv_rn(ws, st.s);
    if (difference)
      map_row<T, true>(out, dx, x, [&](float v) { return __fmul_rn(exp2_fast(__fmul_rn(__fsub_rn(v, st.m), c)), A); });
    else
      map_row<T, true>(out, dx, x, [&](float v) { return __fmul_rn(exp2_fast(__fmaf_rn(v, c, -st.R)), A); });
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
      const float t = difference ? __fmul_rn(__fsub_rn(l.z[i], st.m), c) : __fmaf_rn(l.z[i], c, -st.R);
      dx[token] = Elem<T>::put(__fmul_rn(ws, __fsub_rn(__fdiv_rn(exp2_fast(t), st.s), q)));
    }
  }
}

// ---- many long rows -----------------------------------------------------------
// One block an SM streams rows through a ring of shared-memory tiles, so that
// HBM never waits for a row to be finished. A row's tiles are loaded by the TMA
// engine (1D bulk copies) and read once for the sum; the last `resident` of
// them stay, are turned into the gradient in place and stored from there by
// bulk copies, the others are freed at once and loaded a second time, out of
// L2. Meanwhile the loads of the following rows fill what is free.
//
// Warps: 0 loads tiles, 1 and 2 patch the listed tokens and store tiles, 3 and 4
// read the teacher's lists a row or two ahead (every second row each: what they
// do is all latency), the others compute. mbarriers:
// full (tile has landed), freed (its slot may be loaded again: by each computing
// warp, or as often by the storing thread), done (its gradient is written;
// one set for each storing warp, because a wait tells phases apart by their
// parity alone and may not begin before the one before last is over), listed
// and taken (the two list buffers), joined (the row's sums). Every wait
// gives up after a second; the block's rows from there on get a loss of NaN
// and NaN in the gradient's first element, and MP_ERR_CUDA is recorded. Nothing
// waits without that limit, and the loads and stores in flight are waited for
// before a block ends. (With a barrier of the block at its end, for one mark of
// all its rows, 8192 x 128256 bf16 took 690 us instead of 681.)
// Measured on 8192 rows of 50304 and of 128256 bf16 (us), computing warps x
// vectors a thread x slots: 12 x 3 x 12 338 and 688, 16 x 2 x 13 356 and 738,
// 8 x 4 x 13 373 and 775, 14 x 3 x 10 334 and 691, 16 x 3 x 9 340 and 687,
// 10 x 4 x 10 331 and 735, 20 x 2 x 10 339 and 723.
constexpr int kRingWarps = 12;
constexpr int kRingVectors = 3;                       // 16-B vectors of a tile a thread takes
constexpr int kRingThreads = 32 * kRingWarps;         // that compute
constexpr int kRingHelpers = 5;                       // warps that do not compute
constexpr int kRingBlock = kRingThreads + 32 * kRingHelpers;
constexpr uint32_t kTileBytes = 16 * kRingVectors * kRingThreads;
constexpr int kTileVectors = kTileBytes / 16;
constexpr uint32_t kRingSlots = 12;
constexpr int kRingResident = 10;                     // tiles of a row kept between its passes, at most
constexpr int kRingTeacher = 128;                     // list length, at most
constexpr int kRingOwn = kRingTeacher / 32;           // list entries a lane holds

struct RingList {
  int32_t token[kRingTeacher];  // -1: unused; below: -2 - token of a later entry of a token listed twice
  float q[kRingTeacher];
  float q_sum[kRingTeacher];    // over a token's entries
  float z[kRingTeacher];
  float w, kl0;                 // row weight; sum q log q
  int none, bad;
};

// A row's sum: s = sum 2^((x - ref) c); ref is -inf where nothing is above it.
struct RingSum {
  float ref, s;

  // of a warp's lanes, to each of them
  __device__ __forceinline__ RingSum join(float c) const {
    RingSum a;
    a.ref = warp_max(ref);
    const float f = exp2_fast(__fmul_rn(__fsub_rn(ref, a.ref), c));
    a.s = warp_sum(ref == -kInf ? 0.0f : __fmul_rn(s, f));
    return a;
  }
};

struct RingShared {
  RingList list[2];
  RingSum sums[2][kRingWarps];
  int32_t table[2][2 * kRingTeacher];
  unsigned long long full[kRingSlots], freed[kRingSlots], done[2][kRingSlots], listed[2], taken[2], joined;
};

constexpr size_t kRingBytes = kRingSlots * kTileBytes + sizeof(RingShared);
static_assert(kRingBytes <= 227 * 1024, "one block's shared memory");

// A row in the ring: its body's tiles and their places in the stream of loads.
template <int T>
struct RingRow {
  RowPart<T> part;
  int tiles, resident;
  int64_t vectors;

  __device__ __forceinline__ RingRow(const DsArgs& a, int64_t r)
      : part(static_cast<const typename Elem<T>::type*>(a.logits) + r * a.stride, a.vocab, 0, 1) {
    vectors = part.units * (T == MP_FP32 ? 2 : 1);
    tiles = static_cast<int>((vectors + kTileVectors - 1) / kTileVectors);
    resident = min(tiles, kRingResident);
  }
  __device__ __forceinline__ int loads() const { return 2 * tiles - resident; }
  // the j-th load's tile; tiles are in pass-two order from load tiles - resident on
  __device__ __forceinline__ int tile_of(int load) const { return load < tiles ? load : load - tiles; }
  __device__ __forceinline__ uint32_t bytes(int tile) const {
    return static_cast<uint32_t>(min(static_cast<int64_t>(kTileVectors), vectors - static_cast<int64_t>(tile) * kTileVectors)) * 16;
  }
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(kAll, mbar_wait(bar, parity));
}

__device__ __forceinline__ float row_weight(const DsArgs& a, int64_t r) { return a.row_weight ? a.row_weight[r] : 1.0f; }

// The slot and phase of the stream's next load or tile.
struct RingPlace {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n = 1) {
    slot += n;
    while (slot >= kRingSlots) {
      slot -= kRingSlots;
      phase ^= 1;
    }
  }
};

// A wait gave up in row r (only a fault can cause that): this warp's rows from
// there on do not pass for whole. A row's loss is written only once all of the
// row is, and nothing that waits gets past the row that another warp left, so
// each row that is not whole is marked, by a computing or a storing warp.
template <int T>
__device__ __noinline__ void ring_gave_up(const DsArgs& a, int64_t r, int64_t step) {
  using E = typename Elem<T>::type;
  bulk_wait_all();  // what this thread has stored is not stored over the mark
  __syncwarp();
  for (r += step * (threadIdx.x % 32); r < a.rows; r += 32 * step) {
    a.loss[r] = __int_as_float(0x7FC00000);
    (static_cast<E*>(a.dlogits) + r * a.dlogits_stride)[0] = Elem<T>::put(__int_as_float(0x7FC00000));
  }
}

template <int T>
__device__ __noinline__ bool ring_load(const DsArgs& a, uint32_t tiles, const RingShared& sh) {
  RingPlace at;
  const uint64_t once = l2_evict_first();
  float w = blockIdx.x < a.rows ? row_weight(a, blockIdx.x) : 0.0f;
  int64_t loads = 0;
  bool ok = true;
  for (int64_t r = blockIdx.x; ok && r < a.rows; r += gridDim.x) {
    const float w_next = r + gridDim.x < a.rows ? row_weight(a, r + gridDim.x) : 0.0f;
    if (w != 0.0f) {
      const RingRow<T> row(a, r);
      for (int i = 0; i < row.loads(); ++i, ++loads, at.next()) {
        if (loads >= kRingSlots && !mbar_wait(smem_u32(&sh.freed[at.slot]), at.phase ^ 1)) {
          ok = false;
          break;
        }
        const int tile = row.tile_of(i);
        const uint32_t bar = smem_u32(&sh.full[at.slot]), bytes = row.bytes(tile);
        const void* src = reinterpret_cast<const char*>(row.part.body) + static_cast<int64_t>(tile) * kTileBytes;
        mbar_expect_tx(bar, bytes);
        if (i < row.tiles - row.resident)  // to be loaded again
          bulk_load(tiles + at.slot * kTileBytes, src, bytes, bar);
        else
          bulk_load(tiles + at.slot * kTileBytes, src, bytes, bar, once);
      }
    }
    w = w_next;
  }
  // the last loads land before the block ends
  if (loads < kRingSlots) at = RingPlace{0, 1};
  for (int64_t q = min(loads, static_cast<int64_t>(kRingSlots)); q > 0; --q, at.next())
    ok = mbar_drain(smem_u32(&sh.full[at.slot]), at.phase ^ 1) && ok;
  return ok;
}

// The teacher's list of each row: q, the loss's share that the student has no
// part in, the student's logits, entries of one token joined. The index, the
// teacher's logits and the weight of the next row are on their way while a row
// is worked on.
template <int T>
__device__ __noinline__ bool ring_list(const DsArgs& a, RingShared& sh, int set) {
  using E = typename Elem<T>::type;
  const int lane = threadIdx.x % 32;
  const float c = __fmul_rn(a.scale, kLog2E);
  uint32_t slots = 2;
  while (slots < 2u * a.k) slots *= 2;
  int64_t index[kRingOwn];
  typename Elem<T>::type teacher[kRingOwn];
  float w = 0.0f;
  auto fetch = [&](int64_t r) {
    if (r >= a.rows) return;
    w = row_weight(a, r);
#pragma unroll
    for (int u = 0; u < kRingOwn; ++u) {
      const int i = 32 * u + lane;
      index[u] = -1;
      if (i < a.k) {
        index[u] = load_index(a.index, r * a.index_stride + i, a.index_type);
        teacher[u] = (static_cast<const E*>(a.teacher) + r * a.teacher_stride)[i];
      }
    }
  };
  const int64_t step = 2 * static_cast<int64_t>(gridDim.x);
  RingList& l = sh.list[set];
  fetch(blockIdx.x + set * gridDim.x);
  uint32_t round = 0;  // of this set
  for (int64_t r = blockIdx.x + set * gridDim.x; r < a.rows; r += step, ++round) {
    const E* x = static_cast<const E*>(a.logits) + r * a.stride;
    const float weight = w;
    int32_t token[kRingOwn];
    float q[kRingOwn], z[kRingOwn];
    float tm = -kInf;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kRingOwn; ++u) {
      const bool use = index[u] >= 0 && index[u] < a.vocab;
      bad = bad || index[u] >= a.vocab;
      token[u] = use ? static_cast<int32_t>(index[u]) : -1;
      q[u] = use ? Elem<T>::get(teacher[u]) : -kInf;
      z[u] = use && weight != 0.0f ? Elem<T>::get(x[index[u]]) : 0.0f;
      tm = max_nan(tm, q[u]);
    }
    fetch(r + step);
    if (round >= 1 && !warp_wait(smem_u32(&sh.taken[set]), (round - 1) & 1)) return false;
    if (weight != 0.0f) {
      tm = warp_max(tm);
      bad = __any_sync(kAll, bad);
      const bool none = tm == -kInf;
      float ts = 0.0f;
#pragma unroll
      for (int u = 0; u < kRingOwn; ++u)
        if (!none) ts = __fadd_rn(ts, exp2_fast(__fmul_rn(__fsub_rn(q[u], tm), c)));
      ts = warp_sum(ts);
      const float inv_ts = __fdiv_rn(1.0f, ts), log_ts = logf(ts);
      float kl0 = 0.0f;
#pragma unroll 1
      for (int i = lane; i < static_cast<int>(slots); i += 32) sh.table[set][i] = -1;
      __syncwarp();
      uint32_t twice = 0;  // bit u: entry u's token was in the table
#pragma unroll
      for (int u = 0; u < kRingOwn; ++u) {
        float p = 0.0f;
        if (!none) {
          const float d = __fsub_rn(q[u], tm);
          p = __fmul_rn(exp2_fast(__fmul_rn(d, c)), inv_ts);
          if (p != 0.0f) kl0 = __fmaf_rn(p, __fmaf_rn(d, a.scale, -log_ts), kl0);
        }
        q[u] = p;
        if (token[u] >= 0) {
          uint32_t at = (static_cast<uint32_t>(token[u]) * 0x9E3779B1u) >> 16;
          for (uint32_t n = 0; n < slots; ++n, ++at) {
            const int32_t was = atomicCAS(&sh.table[set][at & (slots - 1)], -1, token[u]);
            if (was == token[u]) twice |= 1u << u;
            if (was == -1 || was == token[u]) break;
          }
        }
      }
      kl0 = warp_sum(kl0);
#pragma unroll
      for (int u = 0; u < kRingOwn; ++u)
        if (32 * u + lane < a.k) {
          l.q[32 * u + lane] = l.q_sum[32 * u + lane] = q[u];
          l.z[32 * u + lane] = z[u];
        }
      // tokens listed twice: the first entry carries the sum, in the list's order
      if (__any_sync(kAll, twice)) {
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kRingOwn; ++u)
          for (uint32_t left = __ballot_sync(kAll, twice >> u & 1); left; left &= left - 1) {
            const int32_t again = __shfl_sync(kAll, token[u], __ffs(left) - 1);
            if (again < 0) continue;  // joined before
            int owner = -1;
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < kRingOwn; ++v)
              for (uint32_t with = __ballot_sync(kAll, token[v] == again); with; with &= with - 1) {
                const int from = __ffs(with) - 1;
                sum = __fadd_rn(sum, __shfl_sync(kAll, q[v], from));
                if (owner >= 0 && lane == from) token[v] = -2 - again;
                owner = owner < 0 ? 32 * v + from : owner;
              }
            if (lane == 0) l.q_sum[owner] = sum;
          }
      }
#pragma unroll
      for (int u = 0; u < kRingOwn; ++u)
        if (32 * u + lane < a.k) l.token[32 * u + lane] = token[u];
      if (lane == 0) {
        l.kl0 = kl0;
        l.none = none;
        l.bad = bad;
      }
    }
    if (lane == 0) l.w = weight;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.listed[set]));
  }
  return true;
}

// Loss, listed tokens and stores.
template <int T>
__device__ __noinline__ bool ring_store(const DsArgs& a, uint8_t* tiles, RingShared& sh, int mine) {
  using E = typename Elem<T>::type;
  const int lane = threadIdx.x % 32;
  const float c = __fmul_rn(a.scale, kLog2E);
  RingPlace at;
  uint32_t done_phase = 0;  // bit s: the parity of slot s's next use of `done`
  int round = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, ++round) {
    const int set = round & 1;
    if (!warp_wait(smem_u32(&sh.listed[set]), (round / 2) & 1)) {
      ring_gave_up<T>(a, set == mine ? r : r + gridDim.x, 2 * static_cast<int64_t>(gridDim.x));
      return false;
    }
    RingList& l = sh.list[set];
    const float w = l.w;
    if (w == 0.0f) {  // the computing warps write the row
    } else if (set != mine) {  // the other warp's row
      at.next(RingRow<T>(a, r).loads());
    } else {
      const RingRow<T> row(a, r);
      const E* x = row.part.row;
      E* dx = static_cast<E*>(a.dlogits) + r * a.dlogits_stride;
      at.next(row.tiles - row.resident);
      RingSum st;
      bool zero = true;
      int32_t token[kRingOwn];
      E grad[kRingOwn];
#pragma unroll 1
      for (int i = 0; i < row.tiles; ++i, at.next()) {
        const int tile = row.tile_of(row.tiles - row.resident + i);
        const uint32_t done = smem_u32(&sh.done[set][at.slot]);
        if (!warp_wait(done, done_phase >> at.slot & 1)) {
          ring_gave_up<T>(a, r, 2 * static_cast<int64_t>(gridDim.x));
          return false;
        }
        done_phase ^= 1u << at.slot;
        if (i == 0) {  // every computing warp has left its sums
          st = sh.sums[set][lane < kRingWarps ? lane : 0];
          if (lane >= kRingWarps) st.ref = -kInf;
          st = st.join(c);
          zero = l.none || st.ref == -kInf;
          const float ws = __fmul_rn(w, a.scale);
#pragma unroll
          for (int u = 0; u < kRingOwn; ++u) {  // the listed tokens' gradients
            const int j = 32 * u + lane;
            token[u] = -1;
            if (j >= a.k) continue;
            const float p = __fdiv_rn(exp2_fast(__fmul_rn(__fsub_rn(l.z[j], st.ref), c)), st.s);
            token[u] = l.token[j];
            grad[u] = Elem<T>::put(zero ? 0.0f : __fmul_rn(ws, __fsub_rn(p, l.q_sum[j])));
          }
          if (row.part.extra) {  // the elements before and after the tiles
            if (lane < row.part.extra) {
              const int64_t j = row.part.extra_index(lane);
              const float p = exp2_fast(__fmul_rn(__fsub_rn(Elem<T>::get(x[j]), st.ref), c));
              dx[j] = Elem<T>::put(zero ? 0.0f : __fmul_rn(p, __fdiv_rn(ws, st.s)));
            }
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kRingOwn; ++u)
              if (token[u] >= 0 && (token[u] < row.part.head || token[u] >= row.part.head + 8 * row.part.units))
                dx[token[u]] = grad[u];
          }
        }
        constexpr int kTileElems = kTileBytes / sizeof(E);
        const int64_t first = row.part.head + static_cast<int64_t>(tile) * kTileElems;
        const int64_t end = min(first + kTileElems, row.part.head + 8 * row.part.units);
        E* data = reinterpret_cast<E*>(tiles + at.slot * kTileBytes);
#pragma unroll
        for (int u = 0; u < kRingOwn; ++u)
          if (token[u] >= first && token[u] < end) data[token[u] - first] = grad[u];
        fence_to_bulk();
        __syncwarp();
        if (lane == 0) {
          bulk_store(dx + first, smem_u32(data), row.bytes(tile));
          bulk_commit();
          if (i > 0) {  // the tile before has been read
            bulk_wait_read<1>();
            mbar_arrive_n(smem_u32(&sh.freed[at.slot == 0 ? kRingSlots - 1 : at.slot - 1]), kRingWarps);
          }
        }
      }
      if (lane == 0) {
        bulk_wait_read<0>();
        mbar_arrive_n(smem_u32(&sh.freed[at.slot == 0 ? kRingSlots - 1 : at.slot - 1]), kRingWarps);
      }
      const float log_s = logf(st.s);
      float kl = 0.0f;
#pragma unroll 1
      for (int j = lane; j < a.k; j += 32)
        if (l.q[j] != 0.0f) {
          const float log_p = st.ref == -kInf ? -kInf : __fmaf_rn(__fsub_rn(l.z[j], st.ref), a.scale, -log_s);
          kl = __fmaf_rn(-__fmul_rn(w, l.q[j]), log_p, kl);  // times w first, as above
        }
      kl = __fmaf_rn(w, l.kl0, warp_sum(kl));
      if (lane == 0) {
        a.loss[r] = l.bad ? __int_as_float(0x7FC00000) : l.none ? 0.0f : kl;
        if (l.bad && a.d_status) atomicCAS(a.d_status, 0, MP_ERR_RANGE);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.taken[set]));
  }
  return true;
}

template <int T>
__global__ void __launch_bounds__(kRingBlock, 1) distill_ring_kernel(DsArgs a) {
  pdl_enter();
  using E = typename Elem<T>::type;
  using V = Vec16<T>;
  extern __shared__ __align__(128) uint8_t tiles[];
  RingShared& sh = *reinterpret_cast<RingShared*>(tiles + kRingSlots * kTileBytes);
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kRingSlots; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.freed[i]), kRingWarps);
      mbar_init(smem_u32(&sh.done[0][i]), kRingWarps);
      mbar_init(smem_u32(&sh.done[1][i]), kRingWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.listed[i]), 1);
      mbar_init(smem_u32(&sh.taken[i]), 2 + kRingWarps);
    }
    mbar_init(smem_u32(&sh.joined), kRingWarps);
    mbar_init_fence();
  }
  __syncthreads();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) ok = ring_load<T>(a, smem_u32(tiles), sh);
  } else if (warp <= 2) {
    ok = ring_store<T>(a, tiles, sh, warp - 1);
    if (lane == 0) bulk_wait_all();
  } else if (warp <= 4) {
    ok = ring_list<T>(a, sh, warp - 3);
  } else {
    const int t = threadIdx.x - 32 * kRingHelpers;
    const float c = __fmul_rn(a.scale, kLog2E), slack = __fdiv_rn(kSlack, c);
    RingPlace at;
    uint32_t joined = 0;
    int round = 0;
    int64_t r = blockIdx.x;
    for (; r < a.rows; r += gridDim.x, ++round) {
      const int set = round & 1;
      ok = warp_wait(smem_u32(&sh.listed[set]), (round / 2) & 1);
      if (!ok) break;
      E* dx = static_cast<E*>(a.dlogits) + r * a.dlogits_stride;
      const RingRow<T> row(a, r);
      if (sh.list[set].w == 0.0f) {
        const RowPart<T>& p = row.part;  // dx divides alike
        const V zero = {make_uint4(0u, 0u, 0u, 0u)};
        for (int64_t i = t; i < row.vectors; i += kRingThreads)
          reinterpret_cast<uint4*>(dx + p.head)[i] = zero.v;
        if (t < p.extra) dx[p.extra_index(t)] = Elem<T>::put(0.0f);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.taken[set]));
          mbar_arrive(smem_u32(&sh.joined));
        }
        ok = warp_wait(smem_u32(&sh.joined), joined);
        if (!ok) break;
        joined ^= 1;
        if (t == 0) a.loss[r] = 0.0f;  // all of the row is written
        continue;
      }
      RingSum st = {-kInf, 0.0f};
      float lim = -kInf;
      auto note = [&](float top) {
        if (top <= lim) return;
        st.s = st.ref == -kInf ? 0.0f : __fmul_rn(st.s, exp2_fast(__fmul_rn(__fsub_rn(st.ref, top), c)));
        st.ref = max_nan(st.ref, top);  // NaN stays, whatever follows it
        lim = __fadd_rn(top, slack);
      };
      for (int i = 0; i < row.tiles; ++i, at.next()) {
        ok = warp_wait(smem_u32(&sh.full[at.slot]), at.phase);
        if (!ok) break;
        const uint4* data = reinterpret_cast<const uint4*>(tiles + at.slot * kTileBytes) + t;
        V v[kRingVectors];
        if (i + 1 < row.tiles || row.vectors % kTileVectors == 0) {
#pragma unroll
          for (int q = 0; q < kRingVectors; ++q) v[q].v = data[q * kRingThreads];
        } else {
          const int n = static_cast<int>(row.vectors % kTileVectors);
#pragma unroll
          for (int q = 0; q < kRingVectors; ++q) {
            v[q].fill_minus_inf();
            if (t + q * kRingThreads < n) v[q].v = data[q * kRingThreads];
          }
        }
        if (i < row.tiles - row.resident) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.freed[at.slot]));
        }
        note(V::max_of(v));
        float sum[kRingVectors];
#pragma unroll
        for (int q = 0; q < kRingVectors; ++q) {
          float f[V::N];
          v[q].get(f);
          sum[q] = 0.0f;
#pragma unroll
          for (int e = 0; e < V::N; ++e)
            sum[q] = __fadd_rn(sum[q], exp2_fast(__fmul_rn(__fsub_rn(f[e], st.ref), c)));
        }
#pragma unroll
        for (int q = 0; q < kRingVectors; ++q) st.s = __fadd_rn(st.s, sum[q]);
      }
      if (!ok) break;
      if (t < row.part.extra) {
        const float x = Elem<T>::get(row.part.row[row.part.extra_index(t)]);
        note(x);
        st.s = __fadd_rn(st.s, exp2_fast(__fmul_rn(__fsub_rn(x, st.ref), c)));
      }
      st = st.join(c);
      if (lane == 0) {
        sh.sums[set][warp - kRingHelpers] = st;
        mbar_arrive(smem_u32(&sh.joined));
      }
      ok = warp_wait(smem_u32(&sh.joined), joined);
      if (!ok) break;
      joined ^= 1;
      st = sh.sums[set][lane < kRingWarps ? lane : 0];
      if (lane >= kRingWarps) st.ref = -kInf;
      st = st.join(c);
      const float A = __fdiv_rn(__fmul_rn(sh.list[set].w, a.scale), st.s), ref = st.ref;
      const bool zero = sh.list[set].none || ref == -kInf;
      // A 2^((x - ref) c) as 2^(c x + B): two operations fewer an element. B, where
      // |B| and |ref c| are below 64, is off by half a step of 2^-18 for its own
      // rounding and for that of ref c, and by a step of log2(A), 2^-17 below 128:
      // below 2^-16, a relative error below 2^-16.5 of the gradient, which is then
      // rounded by up to 2^-11 (fp16) or 2^-8 (bf16) of it. Other rows, and fp32,
      // take the difference first.
      const float B = __fsub_rn(log2f(A), __fmul_rn(ref, c));
      const bool folded = T != MP_FP32 && fabsf(B) < 64.0f && fabsf(__fmul_rn(ref, c)) < 64.0f;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.taken[set]));
      // pass two: from the first resident tile on
      RingPlace two = at;
      two.slot += kRingSlots - row.resident;
      two.phase ^= 1;
      if (two.slot >= kRingSlots) {
        two.slot -= kRingSlots;
        two.phase ^= 1;
      }
      for (int i = 0; i < row.tiles; ++i, two.next()) {
        if (i >= row.resident) {
          ok = warp_wait(smem_u32(&sh.full[two.slot]), two.phase);
          if (!ok) break;
        }
        uint4* data = reinterpret_cast<uint4*>(tiles + two.slot * kTileBytes) + t;
        const int tile = row.tile_of(row.tiles - row.resident + i);
        const int n = tile + 1 < row.tiles ? kTileVectors : static_cast<int>(row.vectors - static_cast<int64_t>(tile) * kTileVectors);
        V v[kRingVectors];
#pragma unroll
        for (int q = 0; q < kRingVectors; ++q) v[q].v = data[q * kRingThreads];  // past the row: not stored
#pragma unroll
        for (int q = 0; q < kRingVectors; ++q) {
          float f[V::N];
          v[q].get(f);
          if (folded) {
#pragma unroll
            for (int e = 0; e < V::N; ++e) f[e] = exp2_fast(__fmaf_rn(f[e], c, B));
          } else {
#pragma unroll
            for (int e = 0; e < V::N; ++e) f[e] = __fmul_rn(exp2_fast(__fmul_rn(__fsub_rn(f[e], ref), c)), A);
          }
          v[q].put(f);
          if (zero) v[q].v = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int q = 0; q < kRingVectors; ++q)
          if (t + q * kRingThreads < n) data[q * kRingThreads] = v[q].v;
        fence_to_bulk();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.done[set][two.slot]));
      }
      if (!ok) break;
      at = two;
    }
    if (!ok) ring_gave_up<T>(a, r, gridDim.x);
  }
  if (!ok && lane == 0 && a.d_status) atomicCAS(a.d_status, 0, MP_ERR_CUDA);
}

// Whether the ring takes these rows: logits and gradient divide into 16-B
// vectors alike, and the rows are long and many enough.
bool ring_takes(const DsArgs& a, int type, const DeviceInfo& dev) {
  const int64_t size = type == MP_FP32 ? 4 : 2;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.logits), dx = reinterpret_cast<uintptr_t>(a.dlogits);
  return a.dlogits && a.k <= kRingTeacher && (x - dx) % 16 == 0 && (a.stride - a.dlogits_stride) * size % 16 == 0 &&
         a.rows >= 2 * dev.sms && a.vocab * size >= 4 * kTileBytes;
}

template <int T>
cudaError_t launch(const DsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (ring_takes(a, T, dev)) {
    static std::atomic<bool> ready[64];
    const cudaError_t e = allow_shared(distill_ring_kernel<T>, static_cast<int>(kRingBytes), ready);
    if (e != cudaSuccess) return e;
    return launch_pdl_smem(distill_ring_kernel<T>, static_cast<unsigned>(dev.sms), kRingBlock, kRingBytes, s, a);
  }
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
