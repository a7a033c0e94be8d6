// mp_rmsnorm.cu — RMS norm with the residual's addition, forward and backward,
// with outputs and kept activations in 8 bits.
//
// A row of up to 8192 columns is read once and stays in registers from the sum of
// its squares to its outputs; longer ones are read twice, backward with the weight
// gradient three times. All sums are fp32. HBM is the bound: 8 B an element
// forward with a residual and 16-bit types (7 with the output in 8 bits, 9 with h kept in
// 8 bits as well), 8 B backward (7 with h kept in 8 bits).
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_tma.cuh"
#include "mp_units.cuh"

namespace mpk {
namespace {

constexpr int64_t kShortD = 256;   // a warp or less a row
constexpr int64_t kStagedD = 8192; // longest row that a block's registers hold
constexpr int kMaxThreads = 512;
// Threads of the backward pass's blocks over short rows, one an SM: what the registers
// hold (bf16 65536 x 128: 14.9 us with 768, 17.0 with 512; 20000 x 93, off the grid, 16.9 and 9.5).
template <int T, bool Wide>
constexpr int kShortThreads = Wide && T != MP_FP32 ? 768 : 512;
constexpr int kLongThreads = 512;
constexpr int64_t kSms = 152;
constexpr int kMaxStages = 4;       // of the forward pass's rings
constexpr int kBackwardStages = 3;  // 8192 x 4096 bf16 47 us, with two 47 and with four 49
constexpr uint32_t kSmShared = 227 * 1024;  // an SM's shared memory for blocks

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
  void* dweight;  // written by the one block that there is; nullptr: blocks' sums go to the workspace
  int64_t rows, d, y_stride, h_stride, y8_stride, h8_stride, x_stride, residual_stride, dy_stride;
  float eps;
  int weight_type;
  int y8_kind;
};

// The weights of a lane's slots.
template <int T, bool Wide>
__device__ __forceinline__ F8 load_weights(const RmsArgs& a, int base, int l) {
  float w[8];
  const auto all = [&](auto load) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = slot_column<T, Wide>(base, l, i);
      w[i] = c < a.d ? load(c) : 0.0f;
    }
  };
  const uint16_t* h = static_cast<const uint16_t*>(a.weight);
  if (!a.weight)
    all([](int) { return 1.0f; });
  else if (a.weight_type == MP_FP32)
    all([&](int c) { return static_cast<const float*>(a.weight)[c]; });
  else if (a.weight_type == MP_BF16)
    all([&](int c) { return Elem<MP_BF16>::get(h[c]); });
  else
    all([&](int c) { return Elem<MP_FP16>::get(h[c]); });
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = make_float2(w[2 * i], w[2 * i + 1]);
  return r;
}

// Weights widened into shared memory once a block: neither their type nor their
// place (they may sit anywhere in a flat buffer) matters afterwards. `n` columns,
// a multiple of 256, those past the row 0. For wide rows a unit's eight lie in two
// planes of four, so that a warp's lanes read neighbouring 16 bytes.
template <bool Wide>
__device__ __forceinline__ void stage_weights(float* sw, const RmsArgs& a, int n, int threads) {
  // several loads on their way at a time, with no question of their type between them
  const auto all = [&](auto load) {
#pragma unroll 8
    for (int j = threadIdx.x; j < n; j += threads) {
      const int at = Wide ? (j / 4 % 2 * (n / 8) + j / 8) * 4 + j % 4 : j;
      sw[at] = j < a.d ? load(j) : 0.0f;
    }
  };
  const uint16_t* h = static_cast<const uint16_t*>(a.weight);
  if (!a.weight)
    all([](int) { return 1.0f; });
  else if (a.weight_type == MP_FP32)
    all([&](int j) { return static_cast<const float*>(a.weight)[j]; });
  else if (a.weight_type == MP_BF16)
    all([&](int j) { return Elem<MP_BF16>::get(h[j]); });
  else
    all([&](int j) { return Elem<MP_FP16>::get(h[j]); });
}

template <int T, bool Wide>
__device__ __forceinline__ F8 staged_weights(const float* sw, int base, int l, int n) {
  base = min(base, n - 256);
  F8 r;
  if constexpr (Wide) {
    const float4* p = reinterpret_cast<const float4*>(sw) + base / 8 + l;
    const float4 a = p[0], b = p[n / 8];
    r.p[0] = make_float2(a.x, a.y);
    r.p[1] = make_float2(a.z, a.w);
    r.p[2] = make_float2(b.x, b.y);
    r.p[3] = make_float2(b.z, b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.p[i] = T == MP_FP32 ? make_float2(sw[base + 64 * i + l], sw[base + 64 * i + 32 + l])
                            : reinterpret_cast<const float2*>(sw)[base / 2 + 32 * i + l];
  }
  return r;
}

template <int T>
__device__ __forceinline__ void fill_nan(Pack8<T>& u) {
  if constexpr (T == MP_FP32)
    u.fill(__uint_as_float(0x7FC00000u));
  else
    u.fill(T == MP_BF16 ? 0x7FC0 : 0x7E00);
}

// Which of the optional inputs and outputs a call has. A few sets are template
// arguments (Set, the bits below), so that a thread's units are one straight piece of
// code whose instructions overlap; others ask at run time (Set < 0). Wide rows:
// y or 8 bits alone (8192 x 4096 bf16, y: 23.5 us, asking 31). With a residual asking is
// as fast or faster (8192 x 8192 81 us, 94 without), except off the grid (8192 x 4097: 72, 65 without).
//
// Of wide rows with scales of 32 columns (kSetBlocks) a thread's four units go through
// each output together (put_units): 16384 x 4096 bf16 with y and h in 8 bits (88 to 90 us) 10 us less
// than asking for each unit, 3789 x 1280 with h in 8 bits, when it took four, 15.5 us instead of 16.5. Without
// such scales that measured slower (8192 x 8192 y 86 us, for each unit 82).
constexpr int kSetBlocks = -2;
enum : int { kHasRes = 1, kHasH = 2, kHasY = 4, kHasRow8 = 8, kHasBlock8 = 16, kHasH8 = 32 };

__host__ __device__ inline int set_of(const RmsArgs& a) {
  return (a.residual ? kHasRes : 0) | (a.h ? kHasH : 0) | (a.y ? kHasY : 0) |
         (!a.y8 ? 0 : a.y8_kind == MP_SCALE_ROW ? kHasRow8 : kHasBlock8) | (a.h8 ? kHasH8 : 0);
}

template <int Set>
__device__ __forceinline__ bool has(int bit, int set) {
  return (Set < 0 ? set : Set) & bit;
}

// A lane's outputs. All lanes of a warp call; where `live` is false nothing is
// written. `inverse`: of the row's 8-bit scale.
template <int T, bool Wide, int Set>
__device__ __forceinline__ void put_unit(const RmsArgs& a, int set, const Pack8<T>& u, const F8& w, float rstd,
                                         float inverse, int64_t r, int base, int l, int d, bool live) {
  using E = typename Elem<T>::type;
  const int64_t blocks = (d + 31) / 32;
  const F8 f = get8(u);
  float m[8 / kShare<T, Wide>];
  if (has<Set>(kHasH, set) && live) store_unit<T, Wide>(u, static_cast<E*>(a.h) + r * a.h_stride, base, l, d);
  if (has<Set>(kHasH8, set)) {
    blocks_amax<T, Wide>(m, u);
    put_block8<T, T, Wide>(f, m, a.h8 + r * a.h8_stride, a.h8_scale + r * blocks, base, l, d, live);
  }
  if (!has<Set>(kHasY | kHasRow8 | kHasBlock8, set)) return;
  const F8 y = mul8(mul8(f, rstd), w);
  if (has<Set>(kHasY, set) && live) {
    Pack8<T> o;
    put8(o, y);
    store_unit<T, Wide>(o, static_cast<E*>(a.y) + r * a.y_stride, base, l, d);
  }
  if (has<Set>(kHasRow8, set)) {
    if (live) store_unit8<T, Wide>(e4m3_pack(mul8(y, inverse)), a.y8 + r * a.y8_stride, base, l, d);
  } else if (has<Set>(kHasBlock8, set)) {
    blocks_amax<T, Wide>(m, y);
    put_block8<T, MP_FP32, Wide>(y, m, a.y8 + r * a.y8_stride, static_cast<uint8_t*>(a.y8_scale) + r * blocks, base, l,
                                 d, live);
  }
}

// The same of a thread's NV units u, unit v at column base(v) with weights(v), for
// kSetBlocks: the units' chains of largest magnitude, scale and rounding side by side.
template <int T, bool Wide, int NV, typename Base, typename Weights>
__device__ __forceinline__ void put_units(const RmsArgs& a, int set, const Pack8<T> (&u)[NV], Weights weights,
                                          float rstd, float inverse, int64_t r, Base base, int l, int d) {
  using E = typename Elem<T>::type;
  const int64_t blocks = (d + 31) / 32;
  const auto y_of = [&](int v) { return mul8(mul8(get8(u[v]), rstd), weights(v)); };
  float m[NV][8 / kShare<T, Wide>];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (has<kSetBlocks>(kHasH, set)) store_unit<T, Wide>(u[v], static_cast<E*>(a.h) + r * a.h_stride, base(v), l, d);
    if (!has<kSetBlocks>(kHasY | kHasRow8, set)) continue;
    const F8 y = y_of(v);
    if (has<kSetBlocks>(kHasY, set)) {
      Pack8<T> o;
      put8(o, y);
      store_unit<T, Wide>(o, static_cast<E*>(a.y) + r * a.y_stride, base(v), l, d);
    }
    if (has<kSetBlocks>(kHasRow8, set))
      store_unit8<T, Wide>(e4m3_pack(mul8(y, inverse)), a.y8 + r * a.y8_stride, base(v), l, d);
  }
  if (has<kSetBlocks>(kHasH8, set)) {
#pragma unroll
    for (int v = 0; v < NV; ++v) blocks_amax<T, Wide>(m[v], u[v]);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      put_block8<T, T, Wide>(get8(u[v]), m[v], a.h8 + r * a.h8_stride, a.h8_scale + r * blocks, base(v), l, d, true);
  }
  if (has<kSetBlocks>(kHasBlock8, set)) {
    F8 y[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      y[v] = y_of(v);
      blocks_amax<T, Wide>(m[v], y[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
      put_block8<T, MP_FP32, Wide>(y[v], m[v], a.y8 + r * a.y8_stride, static_cast<uint8_t*>(a.y8_scale) + r * blocks,
                                   base(v), l, d, true);
  }
}

// From a row's sums (to each of its threads): rstd and the inverse of its 8-bit
// scale; the first thread writes what there is one of.
__device__ __forceinline__ float row_results(const RmsArgs& a, float s, float m, float inv_d, bool row8, int64_t r,
                                             bool writes, float& inverse) {
  const float rstd = rsqrtf(__fmaf_rn(s, inv_d, a.eps));
  inverse = 0.0f;
  if (row8) {
    const float scale = row_scale(__fmul_rn(m, rstd));
    asm("rcp.approx.f32 %0, %1;" : "=f"(inverse) : "f"(scale));
    if (writes) static_cast<float*>(a.y8_scale)[r] = scale;
  }
  if (writes && a.rstd) a.rstd[r] = rstd;
  return rstd;
}

// Short rows, up to 8 * L elements: L lanes of a warp take a row, and the next row
// is on its way while one is summed and written.
template <int T, bool Wide, int L>
__global__ void __launch_bounds__(256) rms_forward_short_kernel(RmsArgs a) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const int t = threadIdx.x % L, d = static_cast<int>(a.d);
  const int64_t groups = 256 / L, step = gridDim.x * groups;
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(d));
  const int set = set_of(a);
  const bool row8 = set & kHasRow8;
  const F8 w = load_weights<T, Wide>(a, 0, t);
  Raw<T, Wide> xn, rn;
  auto fetch = [&](int64_t r) {
    const int n = r < a.rows ? d : 0;
    xn.load(static_cast<const E*>(a.x) + r * a.x_stride, 0, t, n);
    if (a.residual) rn.load(static_cast<const E*>(a.residual) + r * a.residual_stride, 0, t, n);
  };
  int64_t r = blockIdx.x * groups + threadIdx.x / L;
  const int64_t ahead = threadIdx.x % 32 / L;
  fetch(r);
  // every lane of a warp runs the same number of rounds (the shuffles are whole-warp)
#pragma unroll 1
  for (; r - ahead < a.rows; r += step) {
    const bool live = r < a.rows;
    Pack8<T> u = xn.unit();
    if (a.residual) u = sum_of(u, rn.unit());
    fetch(r + step);
    const F8 f = get8(u);
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) s2 = fma2(f.p[i], f.p[i], s2);
    float s = __fadd_rn(s2.x, s2.y), m = row8 ? amax8(0.0f, mul8(f, w)) : 0.0f;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(kAll, s, o));
    if (row8)
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, o));
    float inverse;
    const float rstd = row_results(a, s, m, inv_d, row8, r, t == 0 && live, inverse);
    put_unit<T, Wide, -1>(a, set, u, w, rstd, inverse, r, 0, t, d, live);
  }
}

// Longer rows: groups of G warps take a row each, NV units a thread, from a ring
// of staged rows of their own. A group's warps meet at a named barrier of their
// own once a row, for its sum; by then they have read the stage, which is filled
// again.
template <int T, bool Wide, int NV, int Set>
__global__ void __launch_bounds__(kMaxThreads, 1)
rms_forward_kernel(RmsArgs a, int G, uint32_t pitch, int stages) {
  pdl_enter();
  using E = typename Elem<T>::type;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][kMaxThreads / 32];
  __shared__ unsigned long long full[kMaxThreads / 32 * kMaxStages];
  const int L = 32 * G, t = threadIdx.x % L, group = threadIdx.x / L, groups = blockDim.x / L;
  const int lane = t % 32, first_column = 8 * (t - lane), d = static_cast<int>(a.d), padded = (d + 255) / 256 * 256;
  const int set = set_of(a);
  const bool has_res = has<Set>(kHasRes, set), row8 = has<Set>(kHasRow8, set);
  const uint32_t stage_bytes = has_res ? 2 * pitch : pitch;
  float* sw = reinterpret_cast<float*>(smem);
  uint8_t* ring = smem + 4 * padded + static_cast<size_t>(group) * stages * stage_bytes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
  if (threadIdx.x < groups * stages) {
    mbar_init(smem_u32(&full[threadIdx.x]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  const E* x = static_cast<const E*>(a.x);
  const E* res = static_cast<const E*>(a.residual);
  const uint32_t length = static_cast<uint32_t>(d) * sizeof(E);
  auto fetch = [&](int64_t r, int stage) {  // by the group's first thread
    if (r >= a.rows) return;
    const uint32_t bar = smem_u32(&full[group * stages + stage]), to = smem_u32(ring + stage * stage_bytes);
    const Pieces p(x + r * a.x_stride, length);
    if (has_res) {
      const Pieces q(res + r * a.residual_stride, length);
      mbar_expect_tx(bar, p.bytes + q.bytes);
      bulk_load(to + pitch, q.src, q.bytes, bar);
    } else {
      mbar_expect_tx(bar, p.bytes);
    }
    bulk_load(to, p.src, p.bytes, bar);
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i) fetch(first + i * step, i);
  stage_weights<Wide>(sw, a, padded, blockDim.x);
  __syncthreads();
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(d));
  bool ok = true;
  int stage = 0, parity = 0;
  uint32_t phase = 0;
  int64_t gave_up = 0;
#pragma unroll 1
  for (int64_t r = first; r < a.rows; r += step, parity ^= 1) {
    // a wait that gives up (only a fault can cause that) makes what follows NaN,
    // and nothing more is fetched
    if (ok && !mbar_wait(smem_u32(&full[group * stages + stage]), phase)) {
      ok = false;
      gave_up = r;
    }
    const uint8_t* at = ring + stage * stage_bytes;
    const E* xs = reinterpret_cast<const E*>(at + (Wide ? 0 : Pieces(x + r * a.x_stride, length).offset));
    const E* rs = reinterpret_cast<const E*>(
        at + pitch + (Wide || !has_res ? 0 : Pieces(res + r * a.residual_stride, length).offset));
    Pack8<T> u[NV];
    float2 s2 = make_float2(0.0f, 0.0f);
    float m = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int base = first_column + 8 * v * L;
      Raw<T, Wide> p, q;
      p.load(xs, base, lane, d);
      if (has_res) q.load(rs, base, lane, d);
      u[v] = p.unit();
      if (has_res) {
        // the same sums; with four units a thread the widened ones ran faster (16384 x 4096 to
        // 8 bits 75 us against 81), with two the others (8192 x 8192 81 against 85)
        if (NV == 4)
          put8(u[v], add8(get8(u[v]), get8(q.unit())));
        else
          u[v] = sum_of(u[v], q.unit());
      }
      if (!ok) fill_nan(u[v]);
      const F8 f = get8(u[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = fma2(f.p[i], f.p[i], s2);
      if (row8) m = amax8(m, mul8(f, staged_weights<T, Wide>(sw, base, lane, padded)));
    }
    float s = warp_sum(__fadd_rn(s2.x, s2.y));
    if (row8) m = warp_max(m);
    if (G > 1) {
      if (t % 32 == 0) red[parity][threadIdx.x / 32] = make_float2(s, m);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(L) : "memory");
      s = 0.0f;
      for (int i = 0; i < G; ++i) {
        const float2 f = red[parity][group * G + i];
        s = __fadd_rn(s, f.x);
        m = max_nan(m, f.y);
      }
    } else {
      __syncwarp();
    }
    if (t == 0 && ok) fetch(r + stages * step, stage);
    float inverse;
    const float rstd = row_results(a, s, m, inv_d, row8, r, t == 0, inverse);
    const auto base = [&](int v) { return first_column + 8 * v * L; };
    const auto weights = [&](int v) { return staged_weights<T, Wide>(sw, base(v), lane, padded); };
    if constexpr (Set == kSetBlocks) {
      put_units<T, Wide>(a, set, u, weights, rstd, inverse, r, base, lane, d);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        put_unit<T, Wide, Set>(a, set, u[v], weights(v), rstd, inverse, r, base(v), lane, d, true);
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // the copies that were not waited for land before the block ends
  if (!ok && t == 0) {
    const int64_t round = (gave_up - first) / step;
    for (int64_t i = round; i < round + stages && first + i * step < a.rows; ++i)
      mbar_drain(smem_u32(&full[group * stages + i % stages]), (i / stages) & 1);
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

template <int V>
__device__ __forceinline__ void long_block8(float f, uint8_t* row, uint8_t* scales, int64_t j, int64_t d) {
  const uint32_t byte = block_scale(warp_max(fabsf(f)));
  if (j >= d) return;
  const float g = __fmul_rn(f, block_inverse(byte));
  row[j] = static_cast<uint8_t>(e4m3_pair(block_top<V>(byte) ? below_256(g) : g, 0.0f));
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
    const float rstd = rsqrtf(__fmaf_rn(long_sum(s, red), __fdiv_rn(1.0f, static_cast<float>(a.d)), a.eps));
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

// Short rows, L lanes each.
template <int T, bool Wide, bool H8, int L>
__global__ void __launch_bounds__(kShortThreads<T, Wide>) rms_backward_short_kernel(RmsArgs a, float* part) {
  pdl_enter();
  using E = typename Elem<T>::type;
  constexpr int kThreads = kShortThreads<T, Wide>, kGroups = kThreads / L;
  __shared__ float joined[kThreads * 8];  // the groups' sums
  const int t = threadIdx.x % L, group = threadIdx.x / L, d = static_cast<int>(a.d);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups, blocks = (d + 31) / 32;
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(d));
  const F8 w = load_weights<T, Wide>(a, 0, t);
  F8 dw = zero8();
  Raw<T, Wide> yn, gn, hn;
  Raw8<T, Wide> qn;
  RawScales<T, Wide> bn;
  float rstd_n = 0.0f;
  auto fetch = [&](int64_t r) {
    const bool live = r < a.rows;
    const int n = live ? d : 0;
    rstd_n = live ? a.rstd_in[r] : 0.0f;
    yn.load(static_cast<const E*>(a.dy) + r * a.dy_stride, 0, t, n);
    if constexpr (H8) {
      qn.load(static_cast<const uint8_t*>(a.x) + r * a.x_stride, 0, t, n);
      bn.load(a.x_scale + r * blocks, 0, t, n);
    } else {
      hn.load(static_cast<const E*>(a.x) + r * a.x_stride, 0, t, n);
    }
    if (a.residual) gn.load(static_cast<const E*>(a.residual) + r * a.residual_stride, 0, t, n);
  };
  int64_t r = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const int64_t ahead = threadIdx.x % 32 / L;
  fetch(r);
#pragma unroll 1
  for (; r - ahead < a.rows; r += step) {
    const bool live = r < a.rows;
    const float rstd = rstd_n;
    F8 xh;
    if constexpr (H8)
      xh = bn.values(qn.unit(), rstd);
    else
      xh = mul8(get8(hn.unit()), rstd);
    const F8 f = get8(yn.unit()), g = mul8(f, w);
    F8 o = zero8();
    if (a.residual) o = get8(gn.unit());
    fetch(r + step);
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s2 = fma2(g.p[i], xh.p[i], s2);
      dw.p[i] = fma2(f.p[i], xh.p[i], dw.p[i]);
    }
    float s = __fadd_rn(s2.x, s2.y);
#pragma unroll
    for (int q = L / 2; q > 0; q >>= 1) s = __fadd_rn(s, __shfl_xor_sync(kAll, s, q));
    if (!a.y || !live) continue;
    const float k = -__fmul_rn(__fmul_rn(s, inv_d), rstd);
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = fma2(g.p[i], both(rstd), fma2(xh.p[i], both(k), o.p[i]));
    Pack8<T> u;
    put8(u, o);
    store_unit<T, Wide>(u, static_cast<E*>(a.y) + r * a.y_stride, 0, t, d);
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    joined[group * 8 * L + slot_column<T, Wide>(0, t, 2 * i)] = dw.p[i].x;
    joined[group * 8 * L + slot_column<T, Wide>(0, t, 2 * i + 1)] = dw.p[i].y;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < d; j += kThreads) {
    float s = 0.0f;
    for (int q = 0; q < kGroups; ++q) s = __fadd_rn(s, joined[q * 8 * L + j]);
    if (a.dweight)
      store_as(a.dweight, j, a.weight_type, s);
    else
      part[static_cast<int64_t>(blockIdx.x) * d + j] = s;
  }
}

// Longer rows: groups of G warps take a row each, NV units a thread, from a ring of
// staged rows (dy, h and its scales, dh) of their own, as in the forward pass. dy, xh and
// dh stay in registers from the sum to dx, so a row's one barrier also says that its
// stage has been read. At the end a block's groups add their weight gradients
// through shared memory.
struct StageMap {  // a stage in bytes
  uint32_t pitch, h_pitch;  // a row of dy and dh; of h
  uint32_t size;
};

// What a call wants: dx, dx with dh added, or dweight alone. Asked at run time for each
// unit, it cost 2 to 8 % (16384 x 2592 bf16 62 us instead of 57).
enum class Wanted { dx, dx_dh, dweight };

template <int T, bool Wide, bool H8, int NV, Wanted Want>
__global__ void __launch_bounds__(kMaxThreads, 1)
rms_backward_kernel(RmsArgs a, float* part, int G, StageMap map, int stages) {
  pdl_enter();
  using E = typename Elem<T>::type;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][kMaxThreads / 32];
  __shared__ unsigned long long full[kMaxThreads / 32 * kMaxStages];
  const int L = 32 * G, t = threadIdx.x % L, group = threadIdx.x / L, groups = blockDim.x / L;
  const int lane = t % 32, first_column = 8 * (t - lane), d = static_cast<int>(a.d);
  const uint32_t blocks = (d + 31) / 32;
  constexpr bool has_dh = Want == Wanted::dx_dh;
  uint8_t* ring = smem + static_cast<size_t>(group) * stages * map.size;
  const int64_t first = a.rows * blockIdx.x / gridDim.x + group, end = a.rows * (blockIdx.x + 1) / gridDim.x;
  if (threadIdx.x < groups * stages) {
    mbar_init(smem_u32(&full[threadIdx.x]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  const E* dy = static_cast<const E*>(a.dy);
  const E* dh = static_cast<const E*>(a.residual);
  const uint32_t length = static_cast<uint32_t>(d) * sizeof(E);
  auto dy_row = [&](int64_t r) { return Pieces(dy + r * a.dy_stride, length); };
  auto dh_row = [&](int64_t r) { return Pieces(dh + r * a.residual_stride, length); };
  auto h_row = [&](int64_t r) {
    return H8 ? Pieces(static_cast<const uint8_t*>(a.x) + r * a.x_stride, static_cast<uint32_t>(d))
              : Pieces(static_cast<const E*>(a.x) + r * a.x_stride, length);
  };
  auto scale_row = [&](int64_t r) { return Pieces(a.x_scale + r * blocks, blocks); };
  // In a stage: dy, dh (if any), h, h's scales.
  const uint32_t h_at = has_dh ? 2 * map.pitch : map.pitch;
  auto fetch = [&](int64_t r, int stage) {  // by the group's first thread
    if (r >= end) return;
    const uint32_t bar = smem_u32(&full[group * stages + stage]), to = smem_u32(ring + stage * map.size);
    const Pieces p = dy_row(r), q = h_row(r);
    uint32_t bytes = p.bytes + q.bytes;
    if (has_dh) bytes += dh_row(r).bytes;
    if (H8) bytes += scale_row(r).bytes;
    mbar_expect_tx(bar, bytes);
    bulk_load(to, p.src, p.bytes, bar);
    if (has_dh) {
      const Pieces g = dh_row(r);
      bulk_load(to + map.pitch, g.src, g.bytes, bar);
    }
    bulk_load(to + h_at, q.src, q.bytes, bar);
    if (H8) {
      const Pieces s = scale_row(r);
      bulk_load(to + h_at + map.h_pitch, s.src, s.bytes, bar);
    }
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i) fetch(first + static_cast<int64_t>(i) * groups, i);
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(d));
  F8 w[NV], dw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    w[v] = load_weights<T, Wide>(a, first_column + 8 * v * L, lane);
    dw[v] = zero8();
  }
  float rstd_next = first < end ? a.rstd_in[first] : 0.0f;
  bool ok = true;
  int stage = 0, parity = 0;
  uint32_t phase = 0;
  int64_t gave_up = 0;
#pragma unroll 1
  for (int64_t r = first; r < end; r += groups, parity ^= 1) {
    const float rstd = rstd_next;
    if (r + groups < end) rstd_next = a.rstd_in[r + groups];
    // a wait that gives up (only a fault can cause that) makes what follows NaN,
    // and nothing more is fetched
    if (ok && !mbar_wait(smem_u32(&full[group * stages + stage]), phase)) {
      ok = false;
      gave_up = r;
    }
    const uint8_t* at = ring + stage * map.size;
    const E* ys = reinterpret_cast<const E*>(at + (Wide ? 0 : dy_row(r).offset));
    const E* gs = reinterpret_cast<const E*>(at + map.pitch + (Wide || !has_dh ? 0 : dh_row(r).offset));
    // 8-bit rows are on an 8-byte grid at least
    const uint8_t* hs = at + h_at + (Wide && !H8 ? 0 : h_row(r).offset);
    const uint8_t* ss = H8 ? at + h_at + map.h_pitch + scale_row(r).offset : nullptr;
    F8 xh[NV], f[NV];
    Pack8<T> e[NV];
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int base = first_column + 8 * v * L;
      Raw<T, Wide> y, h, g;
      Raw8<T, Wide> q;
      RawScales<T, Wide> b;
      if (Wide && has_dh) g.load(gs, base, lane, d);  // the order that ran fastest, of either kind
      y.load(ys, base, lane, d);
      if constexpr (H8) {
        q.load(hs, base, lane, d);
        b.load(ss, base, lane, d);
      } else {
        h.load(reinterpret_cast<const E*>(hs), base, lane, d);
      }
      if (!Wide && has_dh) g.load(gs, base, lane, d);
      f[v] = get8(y.unit());
      if constexpr (H8)
        xh[v] = b.values(q.unit(), rstd);
      else
        xh[v] = mul8(get8(h.unit()), rstd);
      if (has_dh)
        e[v] = g.unit();
      else
        e[v].zero();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        dw[v].p[q] = fma2(f[v].p[q], xh[v].p[q], dw[v].p[q]);
        f[v].p[q] = mul2(f[v].p[q], w[v].p[q]);
        s2 = fma2(f[v].p[q], xh[v].p[q], s2);
      }
    }
    float s = warp_sum(__fadd_rn(s2.x, s2.y));
    if (!ok) s = __uint_as_float(0x7FC00000u);
    if (G > 1) {
      if (t % 32 == 0) red[parity][threadIdx.x / 32] = s;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(L) : "memory");
      s = 0.0f;
      for (int i = 0; i < G; ++i) s = __fadd_rn(s, red[parity][group * G + i]);
    } else {
      __syncwarp();
    }
    if (t == 0 && ok) fetch(r + static_cast<int64_t>(stages) * groups, stage);
    if constexpr (Want != Wanted::dweight) {
      const float k = -__fmul_rn(__fmul_rn(s, inv_d), rstd);
      E* out = static_cast<E*>(a.y) + r * a.y_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        F8 o = get8(e[v]);
#pragma unroll
        for (int q = 0; q < 4; ++q) o.p[q] = fma2(f[v].p[q], both(rstd), fma2(xh[v].p[q], both(k), o.p[q]));
        put8(e[v], o);
        store_unit<T, Wide>(e[v], out, first_column + 8 * v * L, lane, d);
      }
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // the copies that were not waited for land before the block ends
  if (!ok && t == 0) {
    const int64_t round = (gave_up - first) / groups;
    for (int64_t i = round; i < round + stages && first + i * groups < end; ++i)
      mbar_drain(smem_u32(&full[group * stages + i % stages]), (i / stages) & 1);
  }
  if (!part) return;
  if (!ok)
#pragma unroll
    for (int v = 0; v < NV; ++v) dw[v] = mul8(dw[v], __uint_as_float(0x7FC00000u));
  __syncthreads();  // no stage is read or filled any more
  float* joined = reinterpret_cast<float*>(smem);
  const int width = 8 * NV * L;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* to = joined + group * width;
      to[slot_column<T, Wide>(first_column + 8 * v * L, lane, 2 * i)] = dw[v].p[i].x;
      to[slot_column<T, Wide>(first_column + 8 * v * L, lane, 2 * i + 1)] = dw[v].p[i].y;
    }
  __syncthreads();
  float* to = part + static_cast<int64_t>(blockIdx.x) * d;
  for (int j = threadIdx.x; j < d; j += blockDim.x) {
    float s = 0.0f;
    for (int q = 0; q < groups; ++q) s = __fadd_rn(s, joined[q * width + j]);
    if (a.dweight)
      store_as(a.dweight, j, a.weight_type, s);
    else
      to[j] = s;
  }
}

// Rows longer than the registers hold: dx row by row, in two passes.
template <int T, bool H8>
__device__ __forceinline__ float long_h(const RmsArgs& a, int64_t r, int64_t j) {
  if constexpr (H8) {
    const F8 f = e4m3_unpack(make_uint2(static_cast<const uint8_t*>(a.x)[r * a.x_stride + j], 0u));
    return __fmul_rn(f.p[0].x, block_scale_value(a.x_scale[r * ((a.d + 31) / 32) + j / 32]));
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

// dweight from `parts` blocks' sums: 32 columns a block, 32 threads a column, each
// adding every 32nd block's sum, five of them on their way at a time.
constexpr int kFinishSlices = 32, kFinishAhead = 5;

__global__ void __launch_bounds__(32 * kFinishSlices) rms_finish_kernel(void* dweight, const float* part, int64_t d,
                                                                        int parts, int weight_type) {
  pdl_enter();
  __shared__ float red[kFinishSlices][32];
  const int c = threadIdx.x % 32, slice = threadIdx.x / 32;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float s = 0.0f;
  if (j < d)
    for (int p = slice; p < parts; p += kFinishAhead * kFinishSlices) {
      float v[kFinishAhead];
#pragma unroll
      for (int i = 0; i < kFinishAhead; ++i) {
        const int q = p + i * kFinishSlices;
        v[i] = q < parts ? part[static_cast<int64_t>(q) * d + j] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kFinishAhead; ++i) s = __fadd_rn(s, v[i]);
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

template <int T, bool Wide, int L>
cudaError_t forward_short(const RmsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t groups = 256 / L, blocks = std::min<int64_t>((a.rows + groups - 1) / groups, 4 * dev.sms);
  return launch_pdl(rms_forward_short_kernel<T, Wide, L>, static_cast<unsigned>(blocks), 256, s, a);
}

template <int T, bool Wide, int NV, int Set>
cudaError_t forward_staged_set(const RmsArgs& a, int G, const DeviceInfo& dev, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  const cudaError_t e = allow_shared(rms_forward_kernel<T, Wide, NV, Set>, kSmShared - 4096, ready);
  if (e != cudaSuccess) return e;
  const uint32_t pitch = pieces_pitch(a.d * (T == MP_FP32 ? 4 : 2)), row = (a.residual ? 2 : 1) * pitch;
  const uint32_t weights = static_cast<uint32_t>((a.d + 255) / 256 * 1024), room = kSmShared - 4096 - weights;
  // one block an SM: as many groups as have two stages each
  const int groups = static_cast<int>(std::max<uint32_t>(1, std::min<uint32_t>(kMaxThreads / (32 * G), room / (2 * row))));
  const int stages = static_cast<int>(std::max<uint32_t>(2, std::min<uint32_t>(kMaxStages, room / (groups * row))));
  const int64_t blocks = std::min<int64_t>((a.rows + groups - 1) / groups, dev.sms);
  return launch_pdl_smem(rms_forward_kernel<T, Wide, NV, Set>, static_cast<unsigned>(blocks),
                         static_cast<unsigned>(32 * G * groups), weights + static_cast<size_t>(stages) * groups * row,
                         s, a, G, pitch, stages);
}

template <int T, bool Wide, int NV>
cudaError_t forward_staged(const RmsArgs& a, int G, const DeviceInfo& dev, cudaStream_t s) {
  if constexpr (NV > 1) {
    constexpr int kOther = Wide ? kHasRow8 : kHasRes | kHasH | kHasY;
    const int set = set_of(a);
    if (set == kHasY) return forward_staged_set<T, Wide, NV, kHasY>(a, G, dev, s);
    if (set == kOther) return forward_staged_set<T, Wide, NV, kOther>(a, G, dev, s);
  }
  if constexpr (Wide && NV == 4)
    if (set_of(a) & (kHasBlock8 | kHasH8)) return forward_staged_set<T, Wide, NV, kSetBlocks>(a, G, dev, s);
  return forward_staged_set<T, Wide, NV, -1>(a, G, dev, s);
}

template <int T, bool Wide>
cudaError_t forward_wide(const RmsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if constexpr (Wide) {  // other rows take whole warps
    if (a.d <= 64) return forward_short<T, Wide, 8>(a, dev, s);
    if (a.d <= 128) return forward_short<T, Wide, 16>(a, dev, s);
  }
  if (a.d <= kShortD) return forward_short<T, Wide, 32>(a, dev, s);
  const int units = static_cast<int>((a.d + 7) / 8);
  const auto warps = [&](int nv) { return (units + 32 * nv - 1) / (32 * nv); };      // of a row
  const auto busy = [&](int nv) { return kMaxThreads / 32 / warps(nv) * warps(nv); };  // of a block
  // Few rows: one or two units a thread, so that more warps share them.
  if (warps(1) <= kMaxThreads / 32 && a.rows * warps(2) < 8 * dev.sms) return forward_staged<T, Wide, 1>(a, warps(1), dev, s);
  if (a.rows * warps(4) < 8 * dev.sms || units <= 64) return forward_staged<T, Wide, 2>(a, warps(2), dev, s);
  // Many: four, so that what a row costs each of its threads is shared by many elements. Two
  // for rows that fill the lanes so, with a residual and no second reduction or
  // quantising of y (8192 x 4096 bf16 43 us, with four 48; but 32768 x 1600 76 against 68, without a
  // residual 35 against 31, y in 8 bits 45 against 40). Rows off the grid: two, as four take more
  // code than the instruction caches hold, unless they leave a block with few warps.
  const bool full = units == 64 * warps(2) && busy(2) >= 14 && a.residual && a.y && !a.y8;
  // With a residual also two for three warps a row (1025 to 1536 columns), where two
  // warps with four would leave a quarter of their lanes or more without work (bf16 y, 3789 x 1280
  // 10.9 us instead of 13.5, 16384 rows of 1032 to 1472 columns, every 64th, 31.8 to 33.3 instead of 35.4 to 37.1, of
  // 1536 33.8 both ways; 16384 x 1536 to 8 bits 36.7 instead of 38.4; without a residual 19.8 against 18.0).
  const bool three = warps(2) == 3 && a.residual;
  if (Wide ? full || three : busy(2) >= 12) return forward_staged<T, Wide, 2>(a, warps(2), dev, s);
  return forward_staged<T, Wide, 4>(a, warps(4), dev, s);
}

template <int T>
cudaError_t forward(const RmsArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.d > kStagedD)
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

// Threads and blocks of the backward pass, from rows and d alone: they fix the
// order of the sums over rows and the workspace.
struct BackwardPlan {
  int parts, G, groups;  // blocks; warps of a row; rows that a block has in hand
};

// A thread's. Two fill the registers: with three (held packed until dx) and so fuller
// blocks for rows of 2500 to 6000, 16471 x 2592 bf16 from 8 bits took 66 us instead of
// 69, but 8192 x 4097 78 instead of 58.
constexpr int kBackwardUnits = 2;

BackwardPlan backward_plan(int64_t rows, int64_t d) {
  BackwardPlan p = {0, 1, 1};
  int64_t cap = 64, per_block = 32;  // blocks; rows that make a further block worth its partial sum
  if (d <= kShortD) {
    cap = kSms;  // more blocks cost more in their sums' addition than they gain
    per_block = 2 * 512 / (d <= 64 ? 8 : d <= 128 ? 16 : 32);
  } else if (d <= kStagedD) {
    p.G = static_cast<int>((d + 256 * kBackwardUnits - 1) / (256 * kBackwardUnits));
    p.groups = kMaxThreads / 32 / p.G;
    cap = kSms;
    per_block = p.groups;
  }
  // Few rows: one block, which needs no second launch (1 x 4096 bf16 4.2 us instead of 5.9).
  const bool one = d <= kStagedD && rows <= 2 * per_block;
  p.parts = one ? 1 : static_cast<int>(std::max<int64_t>(1, std::min(cap, (rows + per_block - 1) / per_block)));
  return p;
}

template <int T, bool Wide, bool H8, int L>
cudaError_t backward_short(const RmsArgs& a, const BackwardPlan& p, float* part, cudaStream_t s) {
  return launch_pdl(rms_backward_short_kernel<T, Wide, H8, L>, static_cast<unsigned>(p.parts),
                    kShortThreads<T, Wide>, s, a, part);
}

template <int T, bool Wide, bool H8, int NV, Wanted Want>
cudaError_t backward_staged(const RmsArgs& a, const BackwardPlan& p, float* part, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  const auto kernel = rms_backward_kernel<T, Wide, H8, NV, Want>;
  const cudaError_t e = allow_shared(kernel, kSmShared - 4096, ready);
  if (e != cudaSuccess) return e;
  StageMap map = {};
  map.pitch = pieces_pitch(a.d * (T == MP_FP32 ? 4 : 2));
  map.h_pitch = H8 ? pieces_pitch(a.d) : map.pitch;
  map.size = (Want == Wanted::dx_dh ? 2 : 1) * map.pitch + map.h_pitch + (H8 ? pieces_pitch((a.d + 31) / 32) : 0);
  const uint32_t per_stage = p.groups * map.size;
  const int stages = static_cast<int>(std::max(2u, std::min<uint32_t>(kBackwardStages, (kSmShared - 4096) / per_stage)));
  const uint32_t threads = 32 * p.G * p.groups;
  const size_t smem = std::max<size_t>(static_cast<size_t>(stages) * per_stage, threads * 8 * NV * sizeof(float));
  return launch_pdl_smem(kernel, static_cast<unsigned>(p.parts), threads, smem, s, a, part, p.G, map, stages);
}

template <int T, bool Wide, bool H8>
cudaError_t backward_wide(const RmsArgs& a, const BackwardPlan& p, float* part, cudaStream_t s) {
  if constexpr (Wide) {
    if (a.d <= 64) return backward_short<T, Wide, H8, 8>(a, p, part, s);
    if (a.d <= 128) return backward_short<T, Wide, H8, 16>(a, p, part, s);
  }
  if (a.d <= kShortD) return backward_short<T, Wide, H8, 32>(a, p, part, s);
  constexpr int NV = kBackwardUnits;
  if (!a.y) return backward_staged<T, Wide, H8, NV, Wanted::dweight>(a, p, part, s);
  return a.residual ? backward_staged<T, Wide, H8, NV, Wanted::dx_dh>(a, p, part, s)
                    : backward_staged<T, Wide, H8, NV, Wanted::dx>(a, p, part, s);
}

template <int T, bool H8>
cudaError_t backward(RmsArgs a, void* dweight, float* part, const DeviceInfo& dev, cudaStream_t s) {
  const BackwardPlan p = backward_plan(a.rows, a.d);
  const bool one = p.parts == 1 && a.d <= kStagedD;
  if (one) a.dweight = dweight;
  cudaError_t e = cudaSuccess;
  if (a.d <= kStagedD) {
    const bool wide = wide_rows(a.dy, a.d, a.dy_stride, a.rows, T) &&
                      (!a.residual || wide_rows(a.residual, a.d, a.residual_stride, a.rows, T)) &&
                      (!a.y || wide_rows(a.y, a.d, a.y_stride, a.rows, T)) &&
                      (H8 ? wide_rows8(a.x, a.d, a.x_stride, a.rows) : wide_rows(a.x, a.d, a.x_stride, a.rows, T));
    float* to = dweight ? part : nullptr;
    e = wide ? backward_wide<T, true, H8>(a, p, to, s) : backward_wide<T, false, H8>(a, p, to, s);
  } else {
    const int64_t strips = (a.d + kLongThreads - 1) / kLongThreads;
    if (dweight)  // before dx, which may be written over dy or h
      e = launch_pdl(rms_dw_long_kernel<T, H8>, static_cast<unsigned>(strips * p.parts), kLongThreads, s, a, part);
    if (e == cudaSuccess && a.y && a.rows)
      e = launch_pdl(rms_dx_long_kernel<T, H8>, static_cast<unsigned>(std::min<int64_t>(a.rows, 4 * dev.sms)),
                     kLongThreads, s, a);
  }
  if (e == cudaSuccess && dweight && !one)
    e = launch_pdl(rms_finish_kernel, static_cast<unsigned>((a.d + 31) / 32), 32 * kFinishSlices, s, dweight,
                   static_cast<const float*>(part), a.d, p.parts, a.weight_type);
  return e;
}

template <int T>
cudaError_t backward_h(const RmsArgs& a, void* dweight, float* part, const DeviceInfo& dev, cudaStream_t s) {
  return a.x_scale ? backward<T, true>(a, dweight, part, dev, s) : backward<T, false>(a, dweight, part, dev, s);
}

}  // namespace

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
  if (y8 && h8 && y8_scale == h8_scale) return MP_ERR_RANGE;
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
  return static_cast<size_t>(backward_plan(rows, d).parts) * d * sizeof(float);
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
