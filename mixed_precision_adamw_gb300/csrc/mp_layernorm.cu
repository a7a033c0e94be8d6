// mp_layernorm.cu — layer norm, forward and backward, with the reduction of
// the weight's and bias's gradients over the rows.
//
// The mean and the variance are taken in two passes over the row (the sum,
// then the squared distances from the mean), so a row with a large common
// offset loses nothing to cancellation; all sums are fp32. A row stays in
// registers between the passes, so each element is read from memory once.
// Everything is bound by HBM: 4 B an element forward and 6 B backward for
// 16-bit types.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_rows.cuh"
#include "mp_tma.cuh"

namespace mpk {
namespace {

constexpr int kLnThreads = 256;
constexpr int64_t kMaxD = int64_t{1} << 24;

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

// The columns of thread t of the L that share a row of d, NV units of eight
// elements: element e of unit v. Wide rows: a unit is eight neighbours, so one
// 16-B access (two for fp32). Other rows: S lanes (a warp, or all of a shorter
// group) have a span of the row, in which neighbouring lanes take neighbouring
// elements; whatever the lane and the warp add to a column is in `first`, the
// rest is a constant of the access (bf16, forward and backward: 32768 x 1357
// 62 and 92 us; 136 and 139 with neighbours over the whole group, whose
// addresses and tests are computed for each element).
template <bool Wide, int NV, int S = 32>
struct Columns {
  int first, left, step;  // left: columns from the first one on, to the row's or the span's end

  __device__ __forceinline__ Columns(int t, int L, int64_t d) {
    if (Wide) {
      first = 8 * t;
      left = static_cast<int>(d) - first;
      step = 8 * L;
    } else {
      const int n = static_cast<int>(d), spans = L / S, span = ((n + spans - 1) / spans + S - 1) / S * S;
      first = t / S * span + t % S;
      left = min(n, (t / S + 1) * span) - first;
      step = 8 * S;
    }
  }
  __device__ __forceinline__ int offset(int v, int e) const { return Wide ? v * step + e : (8 * v + e) * S; }
  __device__ __forceinline__ int at(int v, int e) const { return first + offset(v, e); }
  // whether the element lies in the row (Wide units are in or out whole)
  __device__ __forceinline__ bool has(int v, int e) const { return offset(v, Wide ? 0 : e) < left; }

  template <int T>
  __device__ __forceinline__ void load(Pack8<T>& u, const typename Elem<T>::type* row, int v) const {
    if (!Wide)
      u.load_stepped(row + first, offset(v, 0), S, left);
    else if (has(v, 0))
      u.load(row + at(v, 0));
    else
      u.zero();
  }
  template <int T>
  __device__ __forceinline__ void store(const Pack8<T>& u, typename Elem<T>::type* row, int v) const {
    if (!Wide)
      u.store_stepped(row + first, offset(v, 0), S, left);
    else if (has(v, 0))
      u.store(row + at(v, 0));
  }
};

// Sum over groups of L <= 32 neighbouring lanes, to each of them.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Sum over the block, to every thread; `red` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < blockDim.x / 32; ++w) s = __fadd_rn(s, red[w]);
  return s;
}

// ---- rows staged through shared memory ------------------------------------------
// The TMA engine copies rows into shared memory ahead of their use (1D bulk
// copies, two stages), so that loads stay in flight without registers or
// resident warps to hold them. A copy moves the whole 16-B pieces of a row; the
// fewer than 8 elements before and after them (rows that do not start or end on
// a 16-B boundary) are loaded by threads and put beside them. A row lies in its
// buffer at the offset that its address has from a 16-B boundary, so the next
// row's copy may cover what was put there: the threads that did order it before
// later copies (fence_to_bulk).
template <int T, bool Wide>
struct StagedRow {
  using E = typename Elem<T>::type;
  const E* row;
  uint32_t offset;  // bytes of the row's first element in the buffer
  int head, tail;   // elements before and after the whole pieces
  uint32_t bytes;   // of the whole pieces

  __device__ __forceinline__ StagedRow(const E* p, int64_t d) : row(p) {
    constexpr int kAlign = 16 / sizeof(E);
    if (Wide) {
      offset = 0;
      head = tail = 0;
      bytes = static_cast<uint32_t>(d) * sizeof(E);
      return;
    }
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) / sizeof(E) % kAlign);
    offset = off * sizeof(E);
    head = off ? kAlign - off : 0;
    if (head > d) head = static_cast<int>(d);
    tail = static_cast<int>((d - head) % kAlign);
    bytes = static_cast<uint32_t>(d - head - tail) * sizeof(E);
  }
  __device__ __forceinline__ void copy(uint32_t buffer, uint32_t bar) const {
    if (bytes) bulk_load(buffer + offset + head * sizeof(E), row + head, bytes, bar);
  }
  // the i-th of the elements that the copy leaves out
  __device__ __forceinline__ int edge(int i, int64_t d) const {
    return i < head ? i : static_cast<int>(d) - tail + (i - head);
  }
};

constexpr int kStages = 2;      // of the forward pass
constexpr int kMaxStages = 4;   // of the backward pass

// Bytes of a row's buffer.
inline uint32_t staged_pitch(int64_t d, int type) {
  return static_cast<uint32_t>((d * (type == MP_FP32 ? 4 : 2) + 15) / 16 * 16 + 16);
}

// ---- forward ----------------------------------------------------------------
// Weight and bias are widened into shared memory once a block: at most 8 B a
// column are read there for 4 B or more of memory traffic, and neither their
// type nor their alignment (they may sit anywhere in a flat buffer) matters
// afterwards.
//
// Eight weights of a unit lie in two planes of four, so that the lanes of a
// warp read 16 consecutive bytes each.
__device__ __forceinline__ int plane_index(int64_t unit, int e, int64_t units) {
  return static_cast<int>((e / 4 * units + unit) * 4 + e % 4);
}

template <bool Wide>
__device__ __forceinline__ void stage_weights(float* sw, const LnArgs& a, int64_t units, int threads) {
  for (int64_t j = threadIdx.x; j < a.d; j += threads) {
    const int at = Wide ? plane_index(j / 8, j % 8, units) : static_cast<int>(j);
    sw[at] = a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f;
    sw[8 * units + at] = a.bias ? load_as(a.bias, j, a.weight_type) : 0.0f;
  }
}

// y of a unit of a row from its x.
template <int T, bool Wide, int NV, int S>
__device__ __forceinline__ void normalise_unit(Pack8<T>& u, const float* sw, const float* sb, float mean, float rstd,
                                               int v, const Columns<Wide, NV, S>& c, int64_t units) {
  float f[8], w[8], b[8];
  u.get(f);
  if (Wide) {
    const int64_t unit = min(static_cast<int64_t>(c.at(v, 0) / 8), units - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 p = *reinterpret_cast<const float4*>(sw + (h * units + unit) * 4);
      const float4 q = *reinterpret_cast<const float4*>(sb + (h * units + unit) * 4);
      w[4 * h] = p.x, w[4 * h + 1] = p.y, w[4 * h + 2] = p.z, w[4 * h + 3] = p.w;
      b[4 * h] = q.x, b[4 * h + 1] = q.y, b[4 * h + 2] = q.z, b[4 * h + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool has = c.has(v, e);
      w[e] = has ? sw[c.at(v, e)] : 0.0f;
      b[e] = has ? sb[c.at(v, e)] : 0.0f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = __fmaf_rn(__fmul_rn(__fsub_rn(f[e], mean), rstd), w[e], b[e]);
  u.put(f);
}

// Short rows, up to 8 * L elements: L lanes of a warp take a row each, four
// rows a round so that enough loads are in flight, no barrier.
template <int T, bool Wide, int L>
__global__ void __launch_bounds__(kLnThreads, 4) ln_forward_short_kernel(LnArgs a) {
  pdl_enter();
  using E = typename Elem<T>::type;
  constexpr int R = T == MP_FP32 ? 2 : 4;
  extern __shared__ __align__(128) uint8_t smem[];
  float* sw = reinterpret_cast<float*>(smem);
  const int t = threadIdx.x % L;
  const int64_t units = (a.d + 7) / 8;
  const Columns<Wide, 1, L> cols(t, L, a.d);
  const float n = static_cast<float>(a.d);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kLnThreads / L);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kLnThreads / L) + threadIdx.x / L;
  stage_weights<Wide>(sw, a, units, kLnThreads);
  __syncthreads();
  // every lane of a warp runs the same number of rounds (the shuffles are whole-warp)
  for (int64_t r0 = 0; r0 < a.rows; r0 += R * groups) {
    Pack8<T> u[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + i * groups + first;
      const bool live = r < a.rows;
      if (live)
        cols.load(u[i], static_cast<const E*>(a.x) + r * a.x_stride, 0);
      else
        u[i].zero();
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + i * groups + first;
      float f[8], s = 0.0f, q = 0.0f;
      u[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __fadd_rn(s, f[e]);  // elements past the row are 0
      const float mean = __fdiv_rn(lanes_sum<L>(s), n);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (cols.has(0, e)) {
          const float c = __fsub_rn(f[e], mean);
          q = __fmaf_rn(c, c, q);
        }
      const float var = __fdiv_rn(lanes_sum<L>(q), n);
      const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
      if (r >= a.rows) continue;
      normalise_unit(u[i], sw, sw + 8 * units, mean, rstd, 0, cols, units);
      cols.store(u[i], static_cast<E*>(a.y) + r * a.y_stride, 0);
      if (t == 0) {
        if (a.mean_out) a.mean_out[r] = mean;
        if (a.rstd_out) a.rstd_out[r] = rstd;
      }
    }
  }
}

// Longer rows: groups of G warps (1, 2, 4 or 8 of a block's 8) take a row each
// from two staged buffers of their own, NV units a thread in registers. A
// group's warps meet at a named barrier of their own for each of the two sums.
template <int T, bool Wide, int NV>
__global__ void __launch_bounds__(kLnThreads, NV >= 8 ? 2 : NV >= 4 ? 3 : 4) ln_forward_kernel(LnArgs a, int G, uint32_t pitch) {
  pdl_enter();
  using E = typename Elem<T>::type;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][kLnThreads / 32];
  __shared__ unsigned long long full[kStages * kLnThreads / 32];
  __shared__ uint32_t gave_up[kLnThreads / 32];  // stage + 2 phase of the wait that a group's first thread gave up
  const int64_t units = (a.d + 7) / 8;
  float* sw = reinterpret_cast<float*>(smem);
  const int L = 32 * G, t = threadIdx.x % L, group = threadIdx.x / L, count = kLnThreads / L;
  const Columns<Wide, NV> cols(t, L, a.d);
  uint8_t* buffers = smem + 64 * units + static_cast<size_t>(group) * kStages * pitch;
  const int64_t step = static_cast<int64_t>(gridDim.x) * count;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * count + group;
  if (threadIdx.x < kStages * count) {
    mbar_init(smem_u32(&full[threadIdx.x]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  E edge0 = {}, edge1 = {};  // of the two stages
  auto fetch = [&](int64_t r, int stage) {  // by the group's first warp
    if (r >= a.rows || t >= 32) return;
    const StagedRow<T, Wide> row(static_cast<const E*>(a.x) + r * a.x_stride, a.d);
    if (t == 0) {
      const uint32_t bar = smem_u32(&full[group * kStages + stage]);
      mbar_expect_tx(bar, row.bytes);
      row.copy(smem_u32(buffers + stage * pitch), bar);
    }
    if (!Wide && t < row.head + row.tail) (stage ? edge1 : edge0) = row.row[row.edge(t, a.d)];
  };
  fetch(first, 0);
  fetch(first + step, 1);
  stage_weights<Wide>(sw, a, units, kLnThreads);
  __syncthreads();
  const float n = static_cast<float>(a.d);
  auto meet = [&]() {
    if (G == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(L) : "memory");
  };
  auto group_sum = [&](float v, int which) {
    v = warp_sum(v);
    if (G == 1) return v;
    if (t % 32 == 0) red[which][threadIdx.x / 32] = v;
    meet();
    float s = 0.0f;
    for (int w = 0; w < G; ++w) s = __fadd_rn(s, red[which][group * G + w]);
    return s;
  };
  bool ok = true;
  uint32_t stage = 0, phase = 0;
  // One copy of the body: with the stages unrolled the loop outgrows the
  // instruction caches (32768 x 1600 bf16: 43 us twice over, 82 us four times).
#pragma unroll 1
  for (int64_t r = first; r < a.rows; r += step, phase ^= stage, stage ^= 1) {
    {
      // a wait that gives up (only a fault can cause that) makes what follows NaN,
      // and nothing more is fetched
      if (ok && !mbar_wait(smem_u32(&full[group * kStages + stage]), phase)) {
        ok = false;
        if (t == 0) gave_up[group] = stage + 2 * phase;
      }
      const StagedRow<T, Wide> row(static_cast<const E*>(a.x) + r * a.x_stride, a.d);
      E* data = reinterpret_cast<E*>(buffers + stage * pitch + (Wide ? 0 : row.offset));
      if (!Wide) {
        if (t < row.head + row.tail) data[row.edge(t, a.d)] = stage ? edge1 : edge0;
        if (t < 32) fence_to_bulk();
        meet();
      }
      Pack8<T> u[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) cols.load(u[v], data, v);
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
        u[v].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __fadd_rn(s, f[e]);  // elements past the row are 0
      }
      if (!ok) s = __int_as_float(0x7FC00000);
      const float mean = __fdiv_rn(group_sum(s, 0), n);
      if (G == 1) __syncwarp();
      if (ok) fetch(r + kStages * step, stage);  // every thread of the group has read the buffer
      float q = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
        u[v].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (cols.has(v, e)) {
            const float c = __fsub_rn(f[e], mean);
            q = __fmaf_rn(c, c, q);
          }
      }
      const float var = __fdiv_rn(group_sum(q, 1), n);
      const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
      E* y = static_cast<E*>(a.y) + r * a.y_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!cols.has(v, 0)) continue;
        normalise_unit(u[v], sw, sw + 8 * units, mean, rstd, v, cols, units);
        cols.store(u[v], y, v);
      }
      if (t == 0) {
        if (a.mean_out) a.mean_out[r] = mean;
        if (a.rstd_out) a.rstd_out[r] = rstd;
      }
    }
  }
  // The copy that was waited for and the one after it (if there was one) land
  // before the block ends.
  if (!ok && t == 0) {
    stage = gave_up[group] % 2;
    phase = gave_up[group] / 2;
    mbar_drain(smem_u32(&full[group * kStages + stage]), phase);
    mbar_drain(smem_u32(&full[group * kStages + (stage ^ 1)]), phase ^ stage);
  }
}

// Rows longer than the registers hold: three passes over the row, the later
// ones out of the caches.
template <int T>
__global__ void __launch_bounds__(kLnThreads) ln_forward_long_kernel(LnArgs a) {
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

// ---- backward ---------------------------------------------------------------
// One pass gives dx and the block's share of dweight and dbias: a thread owns
// the same columns in every row it sees, so it adds their dy xh and dy in
// registers, and a block writes its sums once, part[block][0 or 1][d]; a
// second, small launch adds the blocks' sums in block order.

// Adds N per-lane values over the 32 lanes: N / 2 + N / 4 + ... + 1 shuffles
// halve the values each lane carries, the rest finish the one left. Lane l
// ends with the total of value many_index<N>(l).
template <int N>
__device__ __forceinline__ float many_sum(float (&v)[N]) {
  const int lane = threadIdx.x % 32;
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = up ? v[i] : v[i + n / 2];
      const float keep = up ? v[i + n / 2] : v[i];
      v[i] = __fadd_rn(keep, __shfl_xor_sync(kAll, send, o));
    }
    o >>= 1;
  }
  float s = v[0];
#pragma unroll
  for (int q = 16 / N; q > 0; q >>= 1) s = __fadd_rn(s, __shfl_xor_sync(kAll, s, q));
  return s;
}

// The value whose total lane l holds: the top log2(N) bits of l.
template <int N>
__device__ __forceinline__ int many_index(int lane) {
  return lane / (32 / N);
}

// Rows of up to 8 * NV * L elements for the block's L computing threads, R rows
// a round. The last warp stages the rounds' rows of x and dy, their mean and
// rstd and the elements that the copies leave out, as stages become free; what
// it takes to prepare a copy (hundreds of cycles) is off the others' path. One
// barrier a round joins the computing warps' sums (which alternate between two
// buffers) and says that the stage has been read. xh and dy stay in registers,
// widened, from the sums to dx. xh is taken from the difference x - mean: one
// FMA, x rstd - mean rstd, saves an operation (57.8 us against 58.3 at 32768 x
// 1600 bf16, 42.6 against 43.1 at 8192 x 4096), but leaves the rounding of mean
// rstd in every xh of a row whose offset is large beside its spread. Rows past
// the block's last are staged as zeros instead of being tested for.
template <int T, bool Wide, int NV, int R, int MaxThreads, int MinBlocks>
__global__ void __launch_bounds__(MaxThreads + 32, MinBlocks)
ln_backward_kernel(LnArgs a, float* part, uint32_t pitch, int stages) {
  pdl_enter();
  using E = typename Elem<T>::type;
  constexpr int N = 2 * R;
  __shared__ float red[2][16][N];
  __shared__ float stats[kMaxStages][N];  // mean and rstd of a stage's rows
  __shared__ unsigned long long full[kMaxStages], freed[kMaxStages];
  extern __shared__ __align__(128) uint8_t smem[];
  const int t = threadIdx.x, L = blockDim.x - 32, lane = t % 32, warp = t / 32, warps = L / 32;
  const int64_t begin = a.rows * blockIdx.x / gridDim.x, end = a.rows * (blockIdx.x + 1) / gridDim.x;
  const int rounds = static_cast<int>((end - begin + R - 1) / R);
  if (t < stages) {
    mbar_init(smem_u32(&full[t]), 1);
    mbar_init(smem_u32(&freed[t]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  // buffer of row i of x (which = 0) or dy (1) in a stage
  auto buffer = [&](int stage, int i, int which) { return smem + ((stage * R + i) * 2 + which) * pitch; };
  auto source = [&](int64_t r, int which) {
    return which ? static_cast<const E*>(a.dy) + r * a.dy_stride : static_cast<const E*>(a.x) + r * a.x_stride;
  };
  if (warp == warps) {  // the staging warp
    // Lane l < N holds row l / 2's mean or rstd of the next round; each lane
    // the element (l % 16) of x (l < 16) or dy that the copies of each row leave out.
    float stat = 0.0f;
    E edge[R] = {};
    auto ahead = [&](int round) {
      const int64_t r0 = begin + static_cast<int64_t>(round) * R;
      if (lane < N) stat = r0 + lane / 2 < end ? (lane % 2 ? a.rstd : a.mean)[r0 + lane / 2] : 0.0f;
      if (!Wide)
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (r0 + i < end) {
            const StagedRow<T, Wide> row(source(r0 + i, lane / 16), a.d);
            if (lane % 16 < row.head + row.tail) edge[i] = row.row[row.edge(lane % 16, a.d)];
          }
    };
    if (rounds) ahead(0);
    int stage = 0;
    uint32_t phase = 1;
    bool ok = true;
    int round = 0;
    for (; round < rounds; ++round) {
      const int64_t r0 = begin + static_cast<int64_t>(round) * R;
      ok = round < stages || __all_sync(kAll, mbar_wait(smem_u32(&freed[stage]), phase));
      if (!ok) break;
      const uint32_t bar = smem_u32(&full[stage]);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (r0 + i < end) {
          const StagedRow<T, Wide> x(source(r0 + i, 0), a.d), dy(source(r0 + i, 1), a.d);
          if (lane == 0) {
            mbar_more_tx(bar, x.bytes + dy.bytes);
            x.copy(smem_u32(buffer(stage, i, 0)), bar);
            dy.copy(smem_u32(buffer(stage, i, 1)), bar);
          }
          if (!Wide) {
            const StagedRow<T, Wide>& row = lane < 16 ? x : dy;
            if (lane % 16 < row.head + row.tail)
              reinterpret_cast<E*>(buffer(stage, i, lane / 16) + row.offset)[row.edge(lane % 16, a.d)] = edge[i];
          }
        } else {
          for (uint32_t k = lane; k < 2 * pitch / 16; k += 32)
            reinterpret_cast<uint4*>(buffer(stage, i, 0))[k] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (lane < N) stats[stage][lane] = stat;
      if (!Wide) fence_to_bulk();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      if (round + 1 < rounds) ahead(round + 1);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // copies in flight land before the block ends
    if (lane == 0)
      for (int i = max(0, round - stages); i < round; ++i) mbar_drain(smem_u32(&full[i % stages]), (i / stages) & 1);
    return;
  }
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(a.d));
  const Columns<Wide, NV> cols(t, L, a.d);
  float w[NV][8], dw[NV][8], db[NV][8], xh[R][NV][8], g[R][NV][8];
  bool mine[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    mine[v] = cols.has(v, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = cols.at(v, e);
      w[v][e] = cols.has(v, e) ? (a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f) : 0.0f;
      dw[v][e] = db[v][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) xh[i][v][e] = g[i][v][e] = 0.0f;  // stays so past the row
    }
  }
  E* out = a.y ? static_cast<E*>(a.y) + begin * a.y_stride + (Wide ? 8 * t : 0) : nullptr;
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  // one copy of the body, as in the forward pass
#pragma unroll 1
  for (int round = 0; round < rounds; ++round) {
    const int64_t r0 = begin + static_cast<int64_t>(round) * R;
    // A wait that gives up (only a fault can cause that) makes the sums NaN, and
    // the stage, whose copies may still be in flight, is not given back.
    ok = ok && mbar_wait(smem_u32(&full[stage]), phase);
    float rstd[R], sums[N];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const E* x = reinterpret_cast<const E*>(buffer(stage, i, 0));
      const E* dy = reinterpret_cast<const E*>(buffer(stage, i, 1));
      if (!Wide && r0 + i < end) {
        x += StagedRow<T, Wide>(source(r0 + i, 0), a.d).offset / sizeof(E);
        dy += StagedRow<T, Wide>(source(r0 + i, 1), a.d).offset / sizeof(E);
      }
      const float mean = stats[stage][2 * i];
      rstd[i] = stats[stage][2 * i + 1];
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (mine[v]) {
          Pack8<T> u;
          float f[8];
          cols.load(u, dy, v);
          u.get(g[i][v]);
          cols.load(u, x, v);
          u.get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) xh[i][v][e] = __fmul_rn(__fsub_rn(f[e], mean), rstd[i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gw = __fmul_rn(g[i][v][e], w[v][e]);  // 0 past the row
          s1 = __fadd_rn(s1, gw);
          s2 = __fmaf_rn(gw, xh[i][v][e], s2);
        }
      }
      sums[2 * i] = ok ? s1 : __int_as_float(0x7FC00000);
      sums[2 * i + 1] = s2;
    }
    const float part_sum = many_sum<N>(sums);
    if (lane % (32 / N) == 0) red[round & 1][warp][many_index<N>(lane)] = part_sum;
    asm volatile("bar.sync 1, %0;" ::"r"(L) : "memory");
    if (t == 0 && ok) mbar_arrive(smem_u32(&freed[stage]));
    float total = 0.0f;
    for (int q = lane % (32 / N); q < warps; q += 32 / N)
      total = __fadd_rn(total, red[round & 1][q][many_index<N>(lane)]);
#pragma unroll
    for (int o = 16 / N; o > 0; o >>= 1) total = __fadd_rn(total, __shfl_xor_sync(kAll, total, o));
    total = __fmul_rn(total, inv_d);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // dx = g rstd + (xh (-c2 rstd) - c1 rstd)
      const float c1 = -__fmul_rn(__shfl_sync(kAll, total, (2 * i) * (32 / N)), rstd[i]);
      const float c2 = -__fmul_rn(__shfl_sync(kAll, total, (2 * i + 1) * (32 / N)), rstd[i]);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = __fmaf_rn(__fmul_rn(g[i][v][e], w[v][e]), rstd[i], __fmaf_rn(xh[i][v][e], c2, c1));
          dw[v][e] = __fmaf_rn(g[i][v][e], xh[i][v][e], dw[v][e]);
          db[v][e] = __fadd_rn(db[v][e], g[i][v][e]);
        }
        if (mine[v] && out && r0 + i < end) {
          Pack8<T> u;
          u.put(o);
          if (Wide)
            u.store(out + v * 8 * L);
          else
            cols.store(u, out, v);
        }
      }
      if (out) out += a.y_stride;
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!part) return;
  float* pw = part + static_cast<int64_t>(blockIdx.x) * 2 * a.d;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (cols.has(v, e)) {
        const int j = cols.at(v, e);
        pw[j] = ok ? dw[v][e] : __int_as_float(0x7FC00000);
        pw[a.d + j] = ok ? db[v][e] : __int_as_float(0x7FC00000);
      }
}

// Rows of up to 8 * L elements, one per L <= 32 lanes, no barrier; the groups
// of a block join their sums through shared memory at the end.
template <int T, bool Wide, int L>
__global__ void __launch_bounds__(kLnThreads) ln_backward_short_kernel(LnArgs a, float* part) {
  pdl_enter();
  using E = typename Elem<T>::type;
  constexpr int G = kLnThreads / L;
  __shared__ float joined[G][8 * L];
  const int t = threadIdx.x % L, group = threadIdx.x / L;
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(a.d));
  const Columns<Wide, 1, L> cols(t, L, a.d);
  float w[8], dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int j = cols.at(0, e);
    w[e] = cols.has(0, e) ? (a.weight ? load_as(a.weight, j, a.weight_type) : 1.0f) : 0.0f;
    dw[e] = db[e] = 0.0f;
  }
  const int64_t groups = static_cast<int64_t>(gridDim.x) * G;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * G; r0 < a.rows; r0 += groups) {
    const int64_t r = r0 + group;
    const bool live = r < a.rows;
    Pack8<T> x, g;
    x.zero();
    g.zero();
    if (live) {
      cols.load(x, static_cast<const E*>(a.x) + r * a.x_stride, 0);
      cols.load(g, static_cast<const E*>(a.dy) + r * a.dy_stride, 0);
    }
    const float mean = live ? a.mean[r] : 0.0f, rstd = live ? a.rstd[r] : 0.0f;
    float fx[8], fg[8], s1 = 0.0f, s2 = 0.0f;
    x.get(fx);
    g.get(fg);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      fx[e] = __fmul_rn(__fsub_rn(fx[e], mean), rstd);
      const float gw = __fmul_rn(fg[e], w[e]);
      s1 = __fadd_rn(s1, gw);
      s2 = __fmaf_rn(gw, fx[e], s2);
      dw[e] = __fmaf_rn(fg[e], fx[e], dw[e]);
      db[e] = __fadd_rn(db[e], fg[e]);
    }
    const float c1 = __fmul_rn(lanes_sum<L>(s1), inv_d), c2 = __fmul_rn(lanes_sum<L>(s2), inv_d);
    if (a.y && live) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        fx[e] = __fmul_rn(rstd, __fmaf_rn(-fx[e], c2, __fsub_rn(__fmul_rn(fg[e], w[e]), c1)));
      x.put(fx);
      cols.store(x, static_cast<E*>(a.y) + r * a.y_stride, 0);
    }
  }
  if (!part) return;
  float* pw = part + static_cast<int64_t>(blockIdx.x) * 2 * a.d;
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) joined[group][e * L + t] = k ? db[e] : dw[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * L; i += kLnThreads) {
      const int j = Columns<Wide, 1, L>(i % L, L, a.d).at(0, i / L);
      if (j >= a.d) continue;
      float s = 0.0f;
      for (int q = 0; q < G; ++q) s = __fadd_rn(s, joined[q][i]);
      pw[k * a.d + j] = s;
    }
  }
}

// Rows longer than the registers hold: dx row by row, in two passes.
template <int T>
__global__ void __launch_bounds__(kLnThreads) ln_dx_long_kernel(LnArgs a) {
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

// ... and the weight gradients column by column: block (i, c) adds 256 columns
// over the c-th chunk of rows.
template <int T>
__global__ void __launch_bounds__(kLnThreads) ln_dw_long_kernel(LnArgs a, float* part) {
  pdl_enter();
  using E = Elem<T>;
  const int64_t strips = (a.d + kLnThreads - 1) / kLnThreads;
  const int64_t c = blockIdx.x / strips, chunks = gridDim.x / strips;
  const int64_t j = (blockIdx.x % strips) * kLnThreads + threadIdx.x;
  if (j >= a.d) return;
  const int64_t r1 = a.rows * (c + 1) / chunks;
  float sw = 0.0f, sb = 0.0f;
#pragma unroll 4
  for (int64_t r = a.rows * c / chunks; r < r1; ++r) {
    const float xv = E::get(static_cast<const typename E::type*>(a.x)[r * a.x_stride + j]);
    const float g = E::get(static_cast<const typename E::type*>(a.dy)[r * a.dy_stride + j]);
    sw = __fmaf_rn(g, __fmul_rn(__fsub_rn(xv, a.mean[r]), a.rstd[r]), sw);
    sb = __fadd_rn(sb, g);
  }
  part[c * 2 * a.d + j] = sw;
  part[(c * 2 + 1) * a.d + j] = sb;
}

// dweight and dbias from `parts` blocks' sums: 32 columns a block, 32 threads
// a column, each adding every 32nd block's sum.
constexpr int kFinishSlices = 32;

__global__ void __launch_bounds__(32 * kFinishSlices) ln_finish_kernel(void* dweight, void* dbias, const float* part,
                                                                       int64_t d, int parts, int weight_type) {
  pdl_enter();
  __shared__ float red[2][kFinishSlices][33];
  const int c = threadIdx.x % 32, slice = threadIdx.x / 32;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float sw = 0.0f, sb = 0.0f;
  if (j < d) {
#pragma unroll 8
    for (int p = slice; p < parts; p += kFinishSlices) {
      sw = __fadd_rn(sw, part[static_cast<int64_t>(p) * 2 * d + j]);
      sb = __fadd_rn(sb, part[(static_cast<int64_t>(p) * 2 + 1) * d + j]);
    }
  }
  red[0][slice][c] = sw;
  red[1][slice][c] = sb;
  __syncthreads();
  if (slice >= 2 || j >= d) return;
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < kFinishSlices; ++q) s = __fadd_rn(s, red[slice][q][c]);
  if (slice == 0 && dweight) store_as(dweight, j, weight_type, s);
  if (slice == 1 && dbias) store_as(dbias, j, weight_type, s);
}

// ---- launches ---------------------------------------------------------------

// Blocks of the backward pass and their threads for rows of d elements. Fewer
// blocks mean fewer partial sums to write and add; two to four blocks a SM
// keep enough loads in flight. The sums' order, and so their bits, and the
// workspace's size follow from rows and d alone.
constexpr int64_t kSms = 152;

constexpr int kLnShared = 227 * 1024;  // an SM's shared memory for blocks
constexpr int64_t kStagedD = 8192;     // longer rows take the long kernels

struct LnPlan {
  int threads, parts, units, per_sm;  // threads that compute, units a thread
};

LnPlan backward_plan(int64_t rows, int64_t d) {
  LnPlan p = {kLnThreads, 0, 1, 1};
  int64_t per_block = 32, cap = 64;  // rows that make a further block worth its partial sum; blocks
  if (d <= 256) {
    per_block = kLnThreads / (d <= 64 ? 8 : d <= 128 ? 16 : 32);
    cap = 4 * kSms;
  } else if (d <= kStagedD) {
    const int64_t units = (d + 7) / 8;
    p.units = d > 7680 ? 3 : d > 4096 ? 2 : 1;
    p.threads = static_cast<int>((units + 32 * p.units - 1) / (32 * p.units) * 32);
    p.per_sm = p.units > 1 ? 1 : std::max(1, std::min(5, 16 / (p.threads / 32 + 1)));
    per_block = 2;
    cap = p.per_sm * kSms;
  }
  p.parts = static_cast<int>(std::max<int64_t>(1, std::min(cap, (rows + per_block - 1) / per_block)));
  return p;
}

template <int T, bool Wide, int L>
cudaError_t forward_short(const LnArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t per_block = kLnThreads / L * (T == MP_FP32 ? 2 : 4);
  const int64_t blocks = std::min<int64_t>((a.rows + per_block - 1) / per_block, 4 * dev.sms);
  return launch_pdl_smem(ln_forward_short_kernel<T, Wide, L>, static_cast<unsigned>(blocks), kLnThreads,
                         (a.d + 7) / 8 * 64, s, a);
}

template <int T, bool Wide, int NV>
cudaError_t forward_staged(const LnArgs& a, int G, const DeviceInfo& dev, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  const int64_t groups = 8 / G;
  const uint32_t pitch = staged_pitch(a.d, T);
  const size_t smem = (a.d + 7) / 8 * 64 + groups * kStages * pitch;
  const cudaError_t e = allow_shared(ln_forward_kernel<T, Wide, NV>, kLnShared - 4096, ready);
  if (e != cudaSuccess) return e;
  const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(NV >= 8 ? 2 : NV >= 4 ? 3 : 4, kLnShared / (smem + 2048)));
  const int64_t blocks = std::min((a.rows + groups - 1) / groups, per_sm * dev.sms);
  return launch_pdl_smem(ln_forward_kernel<T, Wide, NV>, static_cast<unsigned>(blocks), kLnThreads, smem, s, a, G,
                         pitch);
}

template <int T, bool Wide>
cudaError_t forward_wide(const LnArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.d > kStagedD)
    return launch_pdl(ln_forward_long_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 8 * dev.sms)),
                      kLnThreads, s, a);
  if (a.d <= 64) return forward_short<T, Wide, 8>(a, dev, s);
  if (a.d <= 128) return forward_short<T, Wide, 16>(a, dev, s);
  if (a.d <= 256) return forward_short<T, Wide, 32>(a, dev, s);
  // Warps of a row: few enough that the units fit the registers (8 a thread
  // of aligned 16-bit rows, 4 of others), more where there are too few rows to fill
  // the GPU with as many warps.
  constexpr int kMost = T == MP_FP32 || !Wide ? 4 : 8;
  const int64_t units = (a.d + 7) / 8;
  int G = 1;
  while (G < 8 && (units > 32 * G * kMost || (a.rows * G < 8 * dev.sms && units > 32 * G))) G *= 2;
  const int64_t nv = (units + 32 * G - 1) / (32 * G);
  if (nv == 1) return forward_staged<T, Wide, 1>(a, G, dev, s);
  if (nv == 2) return forward_staged<T, Wide, 2>(a, G, dev, s);
  if (nv <= 4) return forward_staged<T, Wide, 4>(a, G, dev, s);
  if constexpr (kMost == 8) return forward_staged<T, Wide, 8>(a, G, dev, s);
  return cudaErrorInvalidValue;  // not reached: 8 warps of 4 units hold kStagedD
}

template <int T>
cudaError_t forward(const LnArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const bool wide = wide_rows(a.x, a.d, a.x_stride, a.rows, T) && wide_rows(a.y, a.d, a.y_stride, a.rows, T);
  return wide ? forward_wide<T, true>(a, dev, s) : forward_wide<T, false>(a, dev, s);
}

template <int T, bool Wide, int NV, int R, int MaxThreads, int MinBlocks>
cudaError_t backward_staged(const LnArgs& a, const LnPlan& p, float* part, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  const auto kernel = ln_backward_kernel<T, Wide, NV, R, MaxThreads, MinBlocks>;
  const cudaError_t e = allow_shared(kernel, kLnShared - 4096, ready);
  if (e != cudaSuccess) return e;
  const uint32_t pitch = staged_pitch(a.d, T), stage = 2 * R * pitch;
  const int stages = static_cast<int>(
      std::max(2u, std::min<uint32_t>(kMaxStages, (kLnShared / static_cast<uint32_t>(p.per_sm) - 4096) / stage)));
  return launch_pdl_smem(kernel, static_cast<unsigned>(p.parts), static_cast<unsigned>(p.threads) + 32,
                         static_cast<size_t>(stages) * stage, s, a, part, pitch, stages);
}

template <int T, bool Wide>
cudaError_t backward_wide(const LnArgs& a, const LnPlan& p, float* part, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.parts), threads = static_cast<unsigned>(p.threads);
  if (a.d <= 64) return launch_pdl(ln_backward_short_kernel<T, Wide, 8>, grid, threads, s, a, part);
  if (a.d <= 128) return launch_pdl(ln_backward_short_kernel<T, Wide, 16>, grid, threads, s, a, part);
  if (a.d <= 256) return launch_pdl(ln_backward_short_kernel<T, Wide, 32>, grid, threads, s, a, part);
  // Units a thread and rows a round are what the registers hold: a unit of a
  // row takes 16, its weights and sums 24. Two rows of one unit fit 128, and 16
  // such warps fill the register file. 32768 x 1600 bf16: 58 us; four rows a
  // round 83 (spilled registers), 24 warps of 80 registers 86. Longer rows take
  // more units in fewer warps; 8192 rows of bf16, us:
  //   d     2 units, 2 rows   2 units, 1 row   3 units, 1 row    2 units, 1 row
  //         168 registers     128              168 (12-28 B      96 (spilled)
  //                                            of it spill)
  //   5632  55                62                                 81
  //   6144                    62               70                85
  //   7680                    71               80                104
  //   8192                                     82                108
  // 4096 with one unit and two rows: 43, although 12 to 32 bytes of the 96
  // registers a thread spill; two units of 168 registers 45.
  if (p.units == 3) return backward_staged<T, Wide, 3, 1, 352, 1>(a, p, part, s);
  if (p.units == 2 && p.threads > 352) return backward_staged<T, Wide, 2, 1, 480, 1>(a, p, part, s);
  if (p.units == 2) return backward_staged<T, Wide, 2, 2, 352, 1>(a, p, part, s);
  if (p.threads > 480) return backward_staged<T, Wide, 1, 2, 512, 1>(a, p, part, s);
  if (p.threads > 224) return backward_staged<T, Wide, 1, 2, 480, 1>(a, p, part, s);
  if (p.threads > 128) return backward_staged<T, Wide, 1, 2, 224, 2>(a, p, part, s);
  if (p.threads > 96) return backward_staged<T, Wide, 1, 2, 128, 3>(a, p, part, s);
  return backward_staged<T, Wide, 1, 2, 96, 4>(a, p, part, s);
}

template <int T>
cudaError_t backward(const LnArgs& a, void* dweight, void* dbias, float* part, const DeviceInfo& dev,
                     cudaStream_t s) {
  const bool sums = dweight || dbias;
  const LnPlan p = backward_plan(a.rows, a.d);
  const int64_t strips = (a.d + kLnThreads - 1) / kLnThreads;
  cudaError_t e = cudaSuccess;
  if (a.d <= kStagedD) {
    if (a.rows || sums) {
      const bool wide = wide_rows(a.x, a.d, a.x_stride, a.rows, T) && wide_rows(a.dy, a.d, a.dy_stride, a.rows, T) &&
                        (!a.y || wide_rows(a.y, a.d, a.y_stride, a.rows, T));
      float* to = sums ? part : nullptr;
      e = wide ? backward_wide<T, true>(a, p, to, s) : backward_wide<T, false>(a, p, to, s);
    }
  } else {
    if (sums)  // before dx, which may be written over dy or x
      e = launch_pdl(ln_dw_long_kernel<T>, static_cast<unsigned>(strips * p.parts), kLnThreads, s, a, part);
    if (e == cudaSuccess && a.y && a.rows)
      e = launch_pdl(ln_dx_long_kernel<T>, static_cast<unsigned>(std::min<int64_t>(a.rows, 8 * dev.sms)), kLnThreads,
                     s, a);
  }
  if (e == cudaSuccess && sums)
    e = launch_pdl(ln_finish_kernel, static_cast<unsigned>((a.d + 31) / 32), 32 * kFinishSlices, s, dweight, dbias,
                   static_cast<const float*>(part), a.d, p.parts, a.weight_type);
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
  return static_cast<size_t>(2) * backward_plan(rows, d).parts * d * sizeof(float);
}

extern "C" int mp_layernorm_backward(void* dx, void* dweight, void* dbias, const void* dy, const void* x,
                                     const void* weight, const float* mean, const float* rstd, int64_t rows,
                                     int64_t d, int64_t dx_stride, int64_t dy_stride, int64_t x_stride, int32_t type,
                                     int32_t weight_type, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !type_ok(weight_type) || !shape_ok(rows, d) || (dx && !stride_ok(dx_stride, d)) ||
      !stride_ok(dy_stride, d) || !stride_ok(x_stride, d))
    return MP_ERR_RANGE;
  if (rows == 0 && !dweight && !dbias) return MP_OK;
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
