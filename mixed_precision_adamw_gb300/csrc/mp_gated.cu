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

constexpr int kThreadsG = 256;

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
  int c, down;
  int run;  // neighbouring lanes of a row
};

__device__ __forceinline__ Place place(const Tiling& g, int rows_a_thread) {
  const int down = kThreadsG >> g.across, t = static_cast<int>(threadIdx.x);
  const int64_t strip = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
  return {strip * (down * rows_a_thread) + (t >> g.across),
          8 * ((static_cast<int>(blockIdx.x) << g.across) + (t & ((1 << g.across) - 1))), down, min(1 << g.across, 32)};
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
  const Place at = place(g, R);
  const int d = static_cast<int>(a.d), c = at.c;
  const int64_t blocks = (d + 31) / 32;
  const E* gate = static_cast<const E*>(a.gate) + at.r * a.gate_stride;
  const E* up = a.up ? static_cast<const E*>(a.up) + at.r * a.up_stride : nullptr;
  Pack8<T> ga[R], ua[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int ci = at.r + i * at.down < a.rows ? c : d;
    load_unit<T, Wide>(ga[i], gate + i * at.down * a.gate_stride, ci, d);
    if (up) load_unit<T, Wide>(ua[i], up + i * at.down * a.up_stride, ci, d);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = at.r + i * at.down;
    const bool live = r < a.rows;
    F8 f = get8(ga[i]), u;
    if (a.gate8)
      put_block8<T, Wide>(f, quad_amax(ga[i]), a.gate8 + r * a.gate8_stride, a.gate8_scale + r * blocks, c, d, live,
                          at.run);
    if (up) {
      u = get8(ua[i]);
      if (a.up8)
        put_block8<T, Wide>(u, quad_amax(ua[i]), a.up8 + r * a.up8_stride, a.up8_scale + r * blocks, c, d, live,
                            at.run);
    }
    f = mul8(f, sigma8<Act>(f));
    if (up) f = mul8(f, u);
    put8(ga[i], f);
    store_unit<T, Wide>(ga[i], static_cast<E*>(a.y) + r * a.y_stride, c, d, live, at.run);
  }
}

// ---- backward ---------------------------------------------------------------------
template <int T, bool Wide, bool Kept, int Act, int R>
__global__ void __launch_bounds__(kThreadsG) gated_backward_kernel(GatedArgs a, Tiling g) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const Place at = place(g, R);
  const int d = static_cast<int>(a.d), c = at.c;
  const int64_t blocks = (d + 31) / 32;
  Pack8<T> dy[R], ga[Kept ? 1 : R], ua[Kept ? 1 : R];
  uint2 g8[Kept ? R : 1], u8[Kept ? R : 1];
  uint32_t gs[Kept ? R : 1], us[Kept ? R : 1];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = at.r + i * at.down;
    const int ci = r < a.rows ? c : d;
    load_unit<T, Wide>(dy[i], static_cast<const E*>(a.dy) + r * a.dy_stride, ci, d);
    if constexpr (Kept) {
      const bool in = ci < d;
      g8[i] = load_unit8<Wide>(static_cast<const uint8_t*>(a.gate) + r * a.gate_stride, ci, d);
      gs[i] = in ? a.gate_scale[r * blocks + c / 32] : 127u;
      if (a.up) {
        u8[i] = load_unit8<Wide>(static_cast<const uint8_t*>(a.up) + r * a.up_stride, ci, d);
        us[i] = in ? a.up_scale[r * blocks + c / 32] : 127u;
      }
    } else {
      load_unit<T, Wide>(ga[i], static_cast<const E*>(a.gate) + r * a.gate_stride, ci, d);
      if (a.up) load_unit<T, Wide>(ua[i], static_cast<const E*>(a.up) + r * a.up_stride, ci, d);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = at.r + i * at.down;
    const bool live = r < a.rows;
    F8 f, u;
    if constexpr (Kept) {
      f = mul8(e4m3_unpack(g8[i]), block_scale_value(gs[i]));
      if (a.up) u = mul8(e4m3_unpack(u8[i]), block_scale_value(us[i]));
    } else {
      f = get8(ga[i]);
      if (a.up) u = get8(ua[i]);
    }
    const F8 d0 = get8(dy[i]), s = sigma8<Act>(f), act = mul8(f, s);
    Pack8<T> w;
    put8(w, mul8(a.up ? mul8(d0, u) : d0, slope8<Act>(f, s)));
    store_unit<T, Wide>(w, static_cast<E*>(a.dgate) + r * a.dgate_stride, c, d, live, at.run);
    if (a.dup) {
      put8(w, mul8(d0, act));
      store_unit<T, Wide>(w, static_cast<E*>(a.dup) + r * a.dup_stride, c, d, live, at.run);
    }
    if (a.y) {
      put8(w, a.up ? mul8(act, u) : act);
      store_unit<T, Wide>(w, static_cast<E*>(a.y) + r * a.y_stride, c, d, live, at.run);
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
  const Place at = place(g, R);
  const int d = static_cast<int>(a.d), c = at.c;
  const int64_t blocks = (d + 31) / 32;
  const E* from = static_cast<const E*>(a.x_in) + at.r * a.x_stride;
  uint8_t* to = a.q + at.r * a.q_stride;
  uint8_t* scales = static_cast<uint8_t*>(a.scale) + at.r * blocks;
  Pack8<T> x[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    load_unit<T, Wide>(x[i], from + i * at.down * a.x_stride, at.r + i * at.down < a.rows ? c : d, d);
#pragma unroll
  for (int i = 0; i < R; ++i)
    put_block8<T, Wide>(get8(x[i]), quad_amax(x[i]), to + i * at.down * a.q_stride, scales + i * at.down * blocks, c,
                        d, at.r + i * at.down < a.rows, at.run);
}

template <int T, bool Wide, int R>
__global__ void __launch_bounds__(kThreadsG) unpack_kernel(Rows8Args a, Tiling g) {
  pdl_enter();
  using E = typename Elem<T>::type;
  const Place at = place(g, R);
  const int d = static_cast<int>(a.d), c = at.c;
  const int64_t blocks = (d + 31) / 32;
  const bool row = a.kind == MP_SCALE_ROW;
  uint2 q[R];
  float s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = at.r + i * at.down;
    const int ci = r < a.rows ? c : d;
    q[i] = load_unit8<Wide>(a.q_in + r * a.q_stride, ci, d);
    s[i] = ci >= d ? 0.0f
           : row   ? static_cast<const float*>(a.scale)[r]
                   : block_scale_value(static_cast<const uint8_t*>(a.scale)[r * blocks + c / 32]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = at.r + i * at.down;
    Pack8<T> x;
    put8(x, mul8(e4m3_unpack(q[i]), s[i]));
    store_unit<T, Wide>(x, static_cast<E*>(a.x) + r * a.x_stride, c, d, r < a.rows, at.run);
  }
}

// ---- launches -----------------------------------------------------------------------

// Threads of a block along a row of d elements: the fewest lanes left over, more
// of them along the row where that is equal. Whole quads of lanes (32 columns).
Tiling tiling(int64_t d) {
  const int units = static_cast<int>((d + 31) / 32 * 4);
  Tiling best = {};
  for (int across = 8; across >= 3; --across) {
    const int chunks = (units + (1 << across) - 1) >> across;
    if (across == 8 || (chunks << across) < (best.chunks << best.across)) best = {across, chunks};
  }
  return best;
}

template <int R, typename Args>
cudaError_t launch_tiled(void (*kernel)(Args, Tiling), const Args& a, cudaStream_t s) {
  const Tiling g = tiling(a.d);
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
// registers, four for the two streams of 8 bits.
template <int T, int Act>
cudaError_t gated_forward(const GatedArgs& a, cudaStream_t s) {
  constexpr int R = 2;
  const bool wide = wide_rows(a.y, a.d, a.y_stride, a.rows, T) && wide_rows(a.gate, a.d, a.gate_stride, a.rows, T) &&
                    (!a.up || wide_rows(a.up, a.d, a.up_stride, a.rows, T)) &&
                    (!a.gate8 || wide_rows8(a.gate8, a.d, a.gate8_stride, a.rows)) &&
                    (!a.up8 || wide_rows8(a.up8, a.d, a.up8_stride, a.rows));
  return launch_tiled<R>(wide ? gated_forward_kernel<T, true, Act, R> : gated_forward_kernel<T, false, Act, R>, a, s);
}

template <int T, int Act>
cudaError_t gated_backward(const GatedArgs& a, cudaStream_t s) {
  constexpr int R = 2;
  const bool kept = a.gate_scale;
  const auto source = [&](const void* p, int64_t stride) {
    return !p || (kept ? wide_rows8(p, a.d, stride, a.rows) : wide_rows(p, a.d, stride, a.rows, T));
  };
  const bool wide = wide_rows(a.dy, a.d, a.dy_stride, a.rows, T) && source(a.gate, a.gate_stride) &&
                    source(a.up, a.up_stride) && (!a.dgate || wide_rows(a.dgate, a.d, a.dgate_stride, a.rows, T)) &&
                    (!a.dup || wide_rows(a.dup, a.d, a.dup_stride, a.rows, T)) &&
                    (!a.y || wide_rows(a.y, a.d, a.y_stride, a.rows, T));
  const auto kernel = kept ? (wide ? gated_backward_kernel<T, true, true, Act, R> : gated_backward_kernel<T, false, true, Act, R>)
                           : (wide ? gated_backward_kernel<T, true, false, Act, R> : gated_backward_kernel<T, false, false, Act, R>);
  return launch_tiled<R>(kernel, a, s);
}

template <int T>
cudaError_t pack_blocks(const Rows8Args& a, cudaStream_t s) {
  constexpr int R = 4;
  const bool wide = wide_rows(a.x_in, a.d, a.x_stride, a.rows, T) && wide_rows8(a.q, a.d, a.q_stride, a.rows);
  return launch_tiled<R>(wide ? pack_blocks_kernel<T, true, R> : pack_blocks_kernel<T, false, R>, a, s);
}

template <int T>
cudaError_t unpack(const Rows8Args& a, cudaStream_t s) {
  constexpr int R = 4;
  const bool wide = wide_rows(a.x, a.d, a.x_stride, a.rows, T) && wide_rows8(a.q_in, a.d, a.q_stride, a.rows);
  return launch_tiled<R>(wide ? unpack_kernel<T, true, R> : unpack_kernel<T, false, R>, a, s);
}

// Rows whose blocks a grid can count.
bool tiled_ok(int64_t rows, int64_t d) { return unit_shape_ok(rows, d) && rows <= INT32_MAX; }

bool act_ok(int32_t act) { return act == MP_ACT_SILU || act == MP_ACT_GELU; }

}  // namespace

cudaError_t launch_pack8_rows(uint8_t* q, float* scale, const void* x, int64_t rows, int64_t d, int64_t q_stride,
                              int64_t x_stride, int32_t type, const DeviceInfo& dev, cudaStream_t s);

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
  cudaError_t e;
  if (kind == MP_SCALE_ROW) {
    DeviceInfo dev;
    e = device_info(&dev);
    if (e == cudaSuccess)
      e = launch_pack8_rows(static_cast<uint8_t*>(q), static_cast<float*>(scale), x, rows, d, q_stride, x_stride, type,
                            dev, s);
  } else {
    Rows8Args a = {};
    a.x_in = x;
    a.q = static_cast<uint8_t*>(q);
    a.scale = scale;
    a.rows = rows;
    a.d = d;
    a.x_stride = x_stride;
    a.q_stride = q_stride;
    e = type == MP_BF16 ? pack_blocks<MP_BF16>(a, s)
                        : type == MP_FP16 ? pack_blocks<MP_FP16>(a, s) : pack_blocks<MP_FP32>(a, s);
  }
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
