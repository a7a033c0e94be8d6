// mp_gated.cu — the gated activation, forward and backward, and rows put away in
// 8 bits with a power of two for every 32 columns, and read back.
//
//   act(a) = a sigma(v),  v = a (silu) or 2 sqrt(2 / pi) (a + 0.044715 a^3) (gelu:
//   (1 + tanh(v / 2)) / 2 = sigma(v)),  act'(a) = sigma + a sigma (1 - sigma) v'
//
// Nothing is summed over rows or columns: every element goes through registers
// once, and HBM is the bound (16-bit: 6 B an element forward, 8 with both kept in 8 bits;
// 10 B backward, 8 from 8 bits). A thread takes the same eight columns of several rows.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_units.cuh"

namespace mpk {
namespace {

// 8192 x 14336 bf16, backward from 8 bits 142 us, with 256 threads 149; 1021 x 2731
// fp16 5.6 and 6.0; packing 16384 x 4096 with 64 34.3 instead of 31.8.
constexpr int kAcrossMost = 7, kThreadsG = 1 << kAcrossMost;

struct GatedArgs {
  void* y;
  void* dgate;
  void* dup;
  const void* dy;
  const void* gate;  // in the type or in 8 bits
  const void* up;
  const uint8_t* gate_scale;
  const uint8_t* up_scale;
  uint8_t* gate8;
  uint8_t* up8;
  uint8_t* gate8_scale;
  uint8_t* up8_scale;
  int64_t rows, d;
  int64_t y_stride, dgate_stride, dup_stride, dy_stride, gate_stride, up_stride, gate8_stride, up8_stride;
};

// How a block lies over the matrix: 2^across threads along a row, the rest down the
// rows. The grid's x covers a row, y and z (y has no more than 65535) the rows.
struct Tiling {
  int across;
  int chunks;
};

struct Place {
  int64_t r;  // of the thread's first unit; its rows are `down` apart
  int base, l, down;
};

__device__ __forceinline__ Place place(const Tiling& g, int rows_a_thread) {
  const int down = kThreadsG >> g.across, t = static_cast<int>(threadIdx.x), run = min(1 << g.across, 32);
  const int64_t strip = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
  const int l = t & (run - 1), first = (t & ((1 << g.across) - 1)) - l;
  return {strip * (down * rows_a_thread) + (t >> g.across), 8 * ((static_cast<int>(blockIdx.x) << g.across) + first),
          l, down};
}

constexpr float kGelu = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// sigma(v(a)) = 1 / (1 + exp(-v)); what would be below 2^-126 (v under -87.3) is 0.
template <int Act>
__device__ __forceinline__ F8 sigma8(const F8& a) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v = a.p[i];
    if (Act == MP_ACT_GELU)
      v = mul2(mul2(v, both(kGelu)), fma2(both(0.044715f), mul2(v, v), both(1.0f)));
    v = mul2(v, both(-kLog2E));
    v = add2(make_float2(exp2_fast(v.x), exp2_fast(v.y)), both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.p[i].x) : "f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.p[i].y) : "f"(v.y));
  }
  return r;
}

// act'(a) = sigma + a v' sigma (1 - sigma), with s = sigma(v(a)). Far out a v' may
// overflow where sigma (1 - sigma) is 0: the product is then left out.
template <int Act>
__device__ __forceinline__ F8 slope8(const F8& a, const F8& s) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = mul2(s.p[i], fma2(s.p[i], both(-1.0f), both(1.0f)));
    float2 v = a.p[i];
    if (Act == MP_ACT_GELU)
      v = mul2(mul2(v, both(kGelu)), fma2(both(3.0f * 0.044715f), mul2(v, v), both(1.0f)));
    r.p[i] = fma2(t, v, s.p[i]);
    r.p[i].x = t.x > 0.0f ? r.p[i].x : s.p[i].x;
    r.p[i].y = t.y > 0.0f ? r.p[i].y : s.p[i].y;
  }
  return r;
}

// ---- forward ----------------------------------------------------------------------
template <int T, bool Wide, int Act, int R>
__global__ void __launch_bounds__(kThreadsG) gated_forward_kernel(GatedArgs a, Tiling g) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const auto [r0, base, l, down] = place(g, R);
  const int d = static_cast<int>(a.d);
  const int64_t blocks = (d + 31) / 32;
  const E* gate = static_cast<const E*>(a.gate) + r0 * a.gate_stride;
  const E* up = a.up ? static_cast<const E*>(a.up) + r0 * a.up_stride : nullptr;
  Raw<T, Wide> ga[R], ua[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int n = r0 + i * down < a.rows ? d : 0;
    ga[i].load(gate + i * down * a.gate_stride, base, l, n);
    if (up) ua[i].load(up + i * down * a.up_stride, base, l, n);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * down;
    const bool live = r < a.rows;
    float m[8 / kShare<T, Wide>];
    Pack8<T> w = ga[i].unit();
    F8 f = get8(w), u;
    if (a.gate8) {
      blocks_amax<T, Wide>(m, w);
      put_block8<T, T, Wide>(f, m, a.gate8 + r * a.gate8_stride, a.gate8_scale + r * blocks, base, l, d, live);
    }
    if (up) {
      w = ua[i].unit();
      u = get8(w);
      if (a.up8) {
        blocks_amax<T, Wide>(m, w);
        put_block8<T, T, Wide>(u, m, a.up8 + r * a.up8_stride, a.up8_scale + r * blocks, base, l, d, live);
      }
    }
    f = mul8(f, sigma8<Act>(f));
    if (up) f = mul8(f, u);
    put8(w, f);
    if (live) store_unit<T, Wide>(w, static_cast<E*>(a.y) + r * a.y_stride, base, l, d);
  }
}

// ---- backward ---------------------------------------------------------------------
template <int T, bool Wide, bool Kept, int Act, int R>
__global__ void __launch_bounds__(kThreadsG, Wide && T != MP_FP32 ? 7 : 0) gated_backward_kernel(GatedArgs a, Tiling g) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const auto [r0, base, l, down] = place(g, R);
  const int d = static_cast<int>(a.d);
  const int64_t blocks = (d + 31) / 32;
  Raw<T, Wide> dy[R], ga[Kept ? 1 : R], ua[Kept ? 1 : R];
  Raw8<T, Wide> g8[Kept ? R : 1], u8[Kept ? R : 1];
  RawScales<T, Wide> gs[Kept ? R : 1], us[Kept ? R : 1];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * down;
    const int n = r < a.rows ? d : 0;
    dy[i].load(static_cast<const E*>(a.dy) + r * a.dy_stride, base, l, n);
    if constexpr (Kept) {
      g8[i].load(static_cast<const uint8_t*>(a.gate) + r * a.gate_stride, base, l, n);
      gs[i].load(a.gate_scale + r * blocks, base, l, n);
      if (a.up) {
        u8[i].load(static_cast<const uint8_t*>(a.up) + r * a.up_stride, base, l, n);
        us[i].load(a.up_scale + r * blocks, base, l, n);
      }
    } else {
      ga[i].load(static_cast<const E*>(a.gate) + r * a.gate_stride, base, l, n);
      if (a.up) ua[i].load(static_cast<const E*>(a.up) + r * a.up_stride, base, l, n);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * down;
    const bool live = r < a.rows;
    if (!Wide && !live) break;
    F8 f, u;
    if constexpr (Kept) {
      f = gs[i].values(g8[i].unit(), 1.0f);
      if (a.up) u = us[i].values(u8[i].unit(), 1.0f);
    } else {
      f = get8(ga[i].unit());
      if (a.up) u = get8(ua[i].unit());
    }
    const F8 d0 = get8(dy[i].unit()), s = sigma8<Act>(f), act = mul8(f, s);
    Pack8<T> w;
    put8(w, mul8(a.up ? mul8(d0, u) : d0, slope8<Act>(f, s)));
    if (live) store_unit<T, Wide>(w, static_cast<E*>(a.dgate) + r * a.dgate_stride, base, l, d);
    if (a.dup && live) {
      put8(w, mul8(d0, act));
      store_unit<T, Wide>(w, static_cast<E*>(a.dup) + r * a.dup_stride, base, l, d);
    }
    if (a.y && live) {
      put8(w, a.up ? mul8(act, u) : act);
      store_unit<T, Wide>(w, static_cast<E*>(a.y) + r * a.y_stride, base, l, d);
    }
  }
}

// ---- 8 bits -------------------------------------------------------------------------
struct Rows8Args {
  void* x;
  const void* x_in;
  uint8_t* q;
  const uint8_t* q_in;
  void* scale;
  int64_t rows, d, x_stride, q_stride;
  int kind;
};

template <int T, bool Wide, int R>
__global__ void __launch_bounds__(kThreadsG) pack_blocks_kernel(Rows8Args a, Tiling g) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const auto [r0, base, l, down] = place(g, R);
  const int d = static_cast<int>(a.d);
  const int64_t blocks = (d + 31) / 32;
  const E* from = static_cast<const E*>(a.x_in) + r0 * a.x_stride;
  uint8_t* to = a.q + r0 * a.q_stride;
  uint8_t* scales = static_cast<uint8_t*>(a.scale) + r0 * blocks;
  Raw<T, Wide> x[R];
#pragma unroll
  for (int i = 0; i < R; ++i) x[i].load(from + i * down * a.x_stride, base, l, r0 + i * down < a.rows ? d : 0);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float m[8 / kShare<T, Wide>];
    const Pack8<T> u = x[i].unit();
    blocks_amax<T, Wide>(m, u);
    put_block8<T, T, Wide>(get8(u), m, to + i * down * a.q_stride, scales + i * down * blocks, base, l, d,
                           r0 + i * down < a.rows);
  }
}

// A scale for each row: G warps a row, NV units a thread in registers from the
// row's largest magnitude to its 8 bits.
constexpr int kPackUnits = 4;

template <int T, bool Wide, int NV>
__global__ void __launch_bounds__(512) pack_rows_kernel(Rows8Args a, int G) {
  pdl_enter();
  using E = typename Elem<T>::type;
  __shared__ float red[16];
  const int warp = threadIdx.x / 32, l = threadIdx.x % 32, group = warp / G, w = warp - group * G;
  const int d = static_cast<int>(a.d);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32 / G) + group;
  if (r >= a.rows) return;  // the group's warps together
  const E* x = static_cast<const E*>(a.x_in) + r * a.x_stride;
  Raw<T, Wide> raw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) raw[v].load(x, 256 * (w + v * G), l, d);
  Pack8<T> u[NV];
  float m = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    u[v] = raw[v].unit();
    m = amax8(m, get8(u[v]));
  }
  m = warp_max(m);
  if (G > 1) {
    if (l == 0) red[warp] = m;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * G) : "memory");
    for (int i = 0; i < G; ++i) m = max_nan(m, red[group * G + i]);
  }
  const float scale = row_scale(m);
  float inverse;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inverse) : "f"(scale));
  if (w == 0 && l == 0) static_cast<float*>(a.scale)[r] = scale;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    store_unit8<T, Wide>(e4m3_pack(mul8(get8(u[v]), inverse)), a.q + r * a.q_stride, 256 * (w + v * G), l, d);
}

// Rows longer than that: read twice.
template <int T>
__global__ void __launch_bounds__(512) pack_long_rows_kernel(Rows8Args a) {
  pdl_enter();
  using E = Elem<T>;
  __shared__ float red[16];
  const int64_t r = blockIdx.x;
  const typename E::type* x = static_cast<const typename E::type*>(a.x_in) + r * a.x_stride;
  float m = 0.0f;
  for (int64_t j = threadIdx.x; j < a.d; j += 512) m = max_nan(m, fabsf(E::get(x[j])));
  m = warp_max(m);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
  __syncthreads();
  for (int i = 0; i < 16; ++i) m = max_nan(m, red[i]);
  const float scale = row_scale(m);
  float inverse;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inverse) : "f"(scale));
  if (threadIdx.x == 0) static_cast<float*>(a.scale)[r] = scale;
  for (int64_t j = threadIdx.x; j < a.d; j += 512)
    a.q[r * a.q_stride + j] = static_cast<uint8_t>(e4m3_pair(__fmul_rn(E::get(x[j]), inverse), 0.0f));
}

template <int T, bool Wide, int R>
__global__ void __launch_bounds__(kThreadsG) unpack_kernel(Rows8Args a, Tiling g) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const auto [r0, base, l, down] = place(g, R);
  const int d = static_cast<int>(a.d);
  const int64_t blocks = (d + 31) / 32;
  const bool row = a.kind == MP_SCALE_ROW;
  const uint8_t* from = a.q_in + r0 * a.q_stride;
  E* to = static_cast<E*>(a.x) + r0 * a.x_stride;
  Raw8<T, Wide> q[R];
  RawScales<T, Wide> s[R];
  float rs[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * down;
    const int n = r < a.rows ? d : 0;
    q[i].load(from + i * down * a.q_stride, base, l, n);
    if (!row)
      s[i].load(static_cast<const uint8_t*>(a.scale) + r * blocks, base, l, n);
    else
      rs[i] = n ? static_cast<const float*>(a.scale)[r] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    Pack8<T> x;
    put8(x, row ? mul8(e4m3_unpack(q[i].unit()), rs[i]) : s[i].values(q[i].unit(), 1.0f));
    if (r0 + i * down < a.rows) store_unit<T, Wide>(x, to + i * down * a.x_stride, base, l, d);
  }
}

// ---- launches -----------------------------------------------------------------------

// Threads of a block along a row of d elements: the fewest lanes left over, more
// of them along the row where that is equal; at least 2^least, so that lanes that
// share a scale are of one run.
Tiling tiling(int64_t d, int least) {
  const int units = static_cast<int>((d + 31) / 32 * 4);
  Tiling best = {};
  for (int across = kAcrossMost; across >= least; --across) {
    const int chunks = (units + (1 << across) - 1) >> across;
    if (across == kAcrossMost || (chunks << across) < (best.chunks << best.across)) best = {across, chunks};
  }
  return best;
}

template <int R, typename Args>
cudaError_t launch_tiled(void (*kernel)(Args, Tiling), const Args& a, int least, cudaStream_t s) {
  const Tiling g = tiling(a.d, least);
  const int64_t per_block = static_cast<int64_t>(kThreadsG >> g.across) * R;
  const int64_t strips = (a.rows + per_block - 1) / per_block, y = std::min<int64_t>(strips, 65535);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(g.chunks), static_cast<unsigned>(y), static_cast<unsigned>((strips + y - 1) / y));
  cfg.blockDim = dim3(kThreadsG);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, g);
}

// Rows a thread: two for the activation, whose three and four streams take the
// registers, four for the two streams of 8 bits. On the grid fewer cost every
// kernel of many rows (the backward pass of 8192 x 14336 bf16 162 us, with one row
// 190; packing 16384 x 4096 31.7, with two 34.5). A unit off the grid is loaded
// as several words, which hold more registers until they are put together: its
// backward pass takes one row (32768 x 2731 bf16 in 151 us instead of 162 with two,
// 1021 x 2731 fp16 in 5.6 instead of 6.2), its 8 bits two (unpacking 16384 x
// 4097 into fp32 in 71 us instead of 77 with four, packing 2047 x 1365 bf16 in 4.2
// instead of 5.8, though 16384 x 4097 in 61 instead of 59; with one 72). The forward
// pass keeps two there (32768 x 2731 in 91 us instead of 98 with one).
constexpr int kRows = 2, kBackwardRowsOther = 1, kRows8 = 4, kRows8Other = 2;

template <int T, int Act>
cudaError_t gated_forward(const GatedArgs& a, cudaStream_t s) {
  const bool wide = wide_rows(a.y, a.d, a.y_stride, a.rows, T) && wide_rows(a.gate, a.d, a.gate_stride, a.rows, T) &&
                    (!a.up || wide_rows(a.up, a.d, a.up_stride, a.rows, T)) &&
                    (!a.gate8 || wide_rows8(a.gate8, a.d, a.gate8_stride, a.rows)) &&
                    (!a.up8 || wide_rows8(a.up8, a.d, a.up8_stride, a.rows));
  return wide ? launch_tiled<kRows>(gated_forward_kernel<T, true, Act, kRows>, a, 3, s)
              : launch_tiled<kRows>(gated_forward_kernel<T, false, Act, kRows>, a, 5, s);
}

template <int T, int Act>
cudaError_t gated_backward(const GatedArgs& a, cudaStream_t s) {
  const bool kept = a.gate_scale;
  const auto source = [&](const void* p, int64_t stride) {
    return !p || (kept ? wide_rows8(p, a.d, stride, a.rows) : wide_rows(p, a.d, stride, a.rows, T));
  };
  const bool wide = wide_rows(a.dy, a.d, a.dy_stride, a.rows, T) && source(a.gate, a.gate_stride) &&
                    source(a.up, a.up_stride) && (!a.dgate || wide_rows(a.dgate, a.d, a.dgate_stride, a.rows, T)) &&
                    (!a.dup || wide_rows(a.dup, a.d, a.dup_stride, a.rows, T)) &&
                    (!a.y || wide_rows(a.y, a.d, a.y_stride, a.rows, T));
  if (kept)
    return wide ? launch_tiled<kRows>(gated_backward_kernel<T, true, true, Act, kRows>, a, 3, s)
                : launch_tiled<kBackwardRowsOther>(gated_backward_kernel<T, false, true, Act, kBackwardRowsOther>, a, 5, s);
  return wide ? launch_tiled<kRows>(gated_backward_kernel<T, true, false, Act, kRows>, a, 3, s)
              : launch_tiled<kBackwardRowsOther>(gated_backward_kernel<T, false, false, Act, kBackwardRowsOther>, a, 5, s);
}

template <int T>
cudaError_t pack_blocks(const Rows8Args& a, cudaStream_t s) {
  const bool wide = wide_rows(a.x_in, a.d, a.x_stride, a.rows, T) && wide_rows8(a.q, a.d, a.q_stride, a.rows);
  return wide ? launch_tiled<kRows8>(pack_blocks_kernel<T, true, kRows8>, a, 3, s)
              : launch_tiled<kRows8Other>(pack_blocks_kernel<T, false, kRows8Other>, a, 5, s);
}

template <int T, bool Wide>
cudaError_t pack_rows_wide(const Rows8Args& a, cudaStream_t s) {
  // four units a thread; one where a row is short
  const int units = static_cast<int>((a.d + 7) / 8), nv = units <= 32 ? 1 : kPackUnits;
  const int G = (units + 32 * nv - 1) / (32 * nv), groups = std::max(1, 8 / G);
  const unsigned blocks = static_cast<unsigned>((a.rows + groups - 1) / groups);
  return launch_pdl(nv == 1 ? pack_rows_kernel<T, Wide, 1> : pack_rows_kernel<T, Wide, kPackUnits>, blocks,
                    static_cast<unsigned>(32 * G * groups), s, a, G);
}

template <int T>
cudaError_t pack_rows(const Rows8Args& a, cudaStream_t s) {
  if (a.d > 512 * 8 * kPackUnits)
    return launch_pdl(pack_long_rows_kernel<T>, static_cast<unsigned>(a.rows), 512, s, a);
  const bool wide = wide_rows(a.x_in, a.d, a.x_stride, a.rows, T) && wide_rows8(a.q, a.d, a.q_stride, a.rows);
  return wide ? pack_rows_wide<T, true>(a, s) : pack_rows_wide<T, false>(a, s);
}

template <int T>
cudaError_t unpack(const Rows8Args& a, cudaStream_t s) {
  const bool wide = wide_rows(a.x, a.d, a.x_stride, a.rows, T) && wide_rows8(a.q_in, a.d, a.q_stride, a.rows);
  return wide ? launch_tiled<kRows8>(unpack_kernel<T, true, kRows8>, a, 3, s)
              : launch_tiled<kRows8Other>(unpack_kernel<T, false, kRows8Other>, a, 5, s);
}

// Rows whose blocks a grid can count.
bool tiled_ok(int64_t rows, int64_t d) { return unit_shape_ok(rows, d) && rows <= INT32_MAX; }

bool act_ok(int32_t act) { return act == MP_ACT_SILU || act == MP_ACT_GELU; }

}  // namespace

}  // namespace mpk

extern "C" int mp_gated_forward(void* y, void* gate8, void* gate8_scale, void* up8, void* up8_scale,
                                const void* gate, const void* up, int64_t rows, int64_t d, int64_t y_stride,
                                int64_t gate8_stride, int64_t up8_stride, int64_t gate_stride, int64_t up_stride,
                                int32_t activation, int32_t type, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !act_ok(activation) || !tiled_ok(rows, d) || !stride_ok(y_stride, d) ||
      !stride_ok(gate_stride, d) || (up && !stride_ok(up_stride, d)) || (gate8 && !stride_ok(gate8_stride, d)) ||
      (up8 && !stride_ok(up8_stride, d)))
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!y || !gate || (gate8 && !gate8_scale) || (up8 && (!up8_scale || !up))) return MP_ERR_NULL;
  if (!alias_ok(y, y_stride, gate, gate_stride) || !alias_ok(y, y_stride, up, up_stride) ||
      (gate8 && (gate8 == up8 || gate8 == y || gate8 == gate || gate8 == up)) ||
      (up8 && (up8 == y || up8 == gate || up8 == up)))
    return MP_ERR_RANGE;
  if (!type_aligned(y, type) || !type_aligned(gate, type) || !type_aligned(up, type)) return MP_ERR_ALIGN;
  if (gate8 && up8 && gate8_scale == up8_scale) return MP_ERR_RANGE;
  GatedArgs a = {};
  a.y = y;
  a.gate = gate;
  a.up = up;
  a.gate8 = static_cast<uint8_t*>(gate8);
  a.up8 = static_cast<uint8_t*>(up8);
  a.gate8_scale = static_cast<uint8_t*>(gate8_scale);
  a.up8_scale = static_cast<uint8_t*>(up8_scale);
  a.rows = rows;
  a.d = d;
  a.y_stride = y_stride;
  a.gate_stride = gate_stride;
  a.up_stride = up_stride;
  a.gate8_stride = gate8_stride;
  a.up8_stride = up8_stride;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (activation == MP_ACT_SILU)
    e = type == MP_BF16   ? gated_forward<MP_BF16, MP_ACT_SILU>(a, s)
        : type == MP_FP16 ? gated_forward<MP_FP16, MP_ACT_SILU>(a, s)
                          : gated_forward<MP_FP32, MP_ACT_SILU>(a, s);
  else
    e = type == MP_BF16   ? gated_forward<MP_BF16, MP_ACT_GELU>(a, s)
        : type == MP_FP16 ? gated_forward<MP_FP16, MP_ACT_GELU>(a, s)
                          : gated_forward<MP_FP32, MP_ACT_GELU>(a, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}

extern "C" int mp_gated_backward(void* dgate, void* dup, void* y, const void* dy, const void* gate,
                                 const void* gate_scale, const void* up, const void* up_scale, int64_t rows,
                                 int64_t d, int64_t dgate_stride, int64_t dup_stride, int64_t y_stride,
                                 int64_t dy_stride, int64_t gate_stride, int64_t up_stride, int32_t activation,
                                 int32_t type, void* stream) {
  using namespace mpk;
  if (!type_ok(type) || !act_ok(activation) || !tiled_ok(rows, d) || !stride_ok(dgate_stride, d) ||
      !stride_ok(dy_stride, d) || !stride_ok(gate_stride, d) || (up && !stride_ok(up_stride, d)) ||
      (dup && !stride_ok(dup_stride, d)) || (y && !stride_ok(y_stride, d)))
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!dgate || !dy || !gate || !up != !dup || (up && !gate_scale != !up_scale) || (!up && up_scale))
    return MP_ERR_NULL;
  const bool kept = gate_scale;
  const auto over = [&](const void* out, int64_t stride) {
    return alias_ok(out, stride, dy, dy_stride) &&
           (kept ? !out || (out != gate && out != up)
                 : alias_ok(out, stride, gate, gate_stride) && alias_ok(out, stride, up, up_stride));
  };
  if (!over(dgate, dgate_stride) || !over(dup, dup_stride) || !over(y, y_stride) || dgate == dup || dgate == y ||
      (dup && dup == y))
    return MP_ERR_RANGE;
  if (!type_aligned(dgate, type) || !type_aligned(dup, type) || !type_aligned(y, type) || !type_aligned(dy, type) ||
      (!kept && (!type_aligned(gate, type) || !type_aligned(up, type))))
    return MP_ERR_ALIGN;
  GatedArgs a = {};
  a.dgate = dgate;
  a.dup = dup;
  a.y = y;
  a.dy = dy;
  a.gate = gate;
  a.up = up;
  a.gate_scale = static_cast<const uint8_t*>(gate_scale);
  a.up_scale = static_cast<const uint8_t*>(up_scale);
  a.rows = rows;
  a.d = d;
  a.dgate_stride = dgate_stride;
  a.dup_stride = dup_stride;
  a.y_stride = y_stride;
  a.dy_stride = dy_stride;
  a.gate_stride = gate_stride;
  a.up_stride = up_stride;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (activation == MP_ACT_SILU)
    e = type == MP_BF16   ? gated_backward<MP_BF16, MP_ACT_SILU>(a, s)
        : type == MP_FP16 ? gated_backward<MP_FP16, MP_ACT_SILU>(a, s)
                          : gated_backward<MP_FP32, MP_ACT_SILU>(a, s);
  else
    e = type == MP_BF16   ? gated_backward<MP_BF16, MP_ACT_GELU>(a, s)
        : type == MP_FP16 ? gated_backward<MP_FP16, MP_ACT_GELU>(a, s)
                          : gated_backward<MP_FP32, MP_ACT_GELU>(a, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}

namespace {

int rows8_check(const void* q, const void* scale, const void* x, int64_t rows, int64_t d, int64_t q_stride,
                int64_t x_stride, int32_t type, int32_t kind) {
  using namespace mpk;
  if (!type_ok(type) || !scale8_ok(kind) || !tiled_ok(rows, d) || !stride_ok(q_stride, d) ||
      !stride_ok(x_stride, d))
    return MP_ERR_RANGE;
  if (rows == 0) return MP_OK;
  if (!q || !scale || !x) return MP_ERR_NULL;
  if (q == x) return MP_ERR_RANGE;
  return type_aligned(x, type) && scale8_aligned(scale, kind) ? MP_OK : MP_ERR_ALIGN;
}

}  // namespace

extern "C" int mp_pack8(void* q, void* scale, const void* x, int64_t rows, int64_t d, int64_t q_stride,
                        int64_t x_stride, int32_t type, int32_t kind, void* stream) {
  using namespace mpk;
  const int st = rows8_check(q, scale, x, rows, d, q_stride, x_stride, type, kind);
  if (st != MP_OK || rows == 0) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  Rows8Args a = {};
  a.x_in = x;
  a.q = static_cast<uint8_t*>(q);
  a.scale = scale;
  a.rows = rows;
  a.d = d;
  a.x_stride = x_stride;
  a.q_stride = q_stride;
  cudaError_t e;
  if (kind == MP_SCALE_ROW)
    e = type == MP_BF16 ? pack_rows<MP_BF16>(a, s)
                        : type == MP_FP16 ? pack_rows<MP_FP16>(a, s) : pack_rows<MP_FP32>(a, s);
  else
    e = type == MP_BF16 ? pack_blocks<MP_BF16>(a, s)
                        : type == MP_FP16 ? pack_blocks<MP_FP16>(a, s) : pack_blocks<MP_FP32>(a, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}

extern "C" int mp_unpack8(void* x, const void* q, const void* scale, int64_t rows, int64_t d, int64_t x_stride,
                          int64_t q_stride, int32_t type, int32_t kind, void* stream) {
  using namespace mpk;
  const int st = rows8_check(q, scale, x, rows, d, q_stride, x_stride, type, kind);
  if (st != MP_OK || rows == 0) return st;
  Rows8Args a = {};
  a.x = x;
  a.q_in = static_cast<const uint8_t*>(q);
  a.scale = const_cast<void*>(scale);
  a.rows = rows;
  a.d = d;
  a.x_stride = x_stride;
  a.q_stride = q_stride;
  a.kind = kind;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == MP_BF16   ? unpack<MP_BF16>(a, s)
                        : type == MP_FP16 ? unpack<MP_FP16>(a, s) : unpack<MP_FP32>(a, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}
