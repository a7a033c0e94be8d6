// mp_rope.cu — rotary positions of queries and keys, forward and inverse, and
// their frequencies.
//
// Angles are kept in turns, as 64-bit fractions: position * turns[i] modulo 2^64
// is the exact fraction of a turn, whatever the position, so there is no range
// reduction and no angle loses bits far into a context. The two leading bits are
// the quadrant; the rest, within an eighth of a turn of it, goes to fp32. A
// block takes a few tokens: their sines and cosines are computed once for all
// heads, into shared memory, and the rest is bound by HBM: 4 B a 16-bit element.
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_units.cuh"

namespace mpk {
namespace {

constexpr int kRopeThreads = 256;
constexpr int64_t kRopeSms = 152;
constexpr int kMaxHeads = 1024;    // of queries, and of keys
constexpr int kMaxHeadDim = 1024;  // so that heads * items * items < 2^32 (divisions by items)

struct RopeSide {  // queries or keys
  void* out;
  const void* in;
  int64_t out_token, out_head, in_token, in_head;
};

struct RopeArgs {
  RopeSide q, k;
  const uint64_t* turns;
  const void* positions;
  int64_t first, tokens;
  int q_heads, heads;  // heads: of queries and keys
  int pairs;           // rotary_dim / 2
  int items;           // of a head
  int per_block;       // tokens
  uint32_t by_items, by_token;  // multipliers of the divisions by items and by heads * items
  float factor;
  int index_type;
  int inverse;
};

// n / d with m = ceil(2^32 / d), for n d < 2^32; d = 1 has m = 0.
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t m) { return m ? __umulhi(n, m) : n; }
inline uint32_t divisor(uint32_t d) { return d == 1 ? 0u : static_cast<uint32_t>((uint64_t{1} << 32) / d + 1); }

// (cos, sin) of `turn` / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(uint64_t turn) {
  const uint64_t shifted = turn + (uint64_t{1} << 61);  // by an eighth of a turn
  const uint32_t quadrant = static_cast<uint32_t>(shifted >> 62);
  const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(quadrant) << 62));
  float s, c;
  sincospif(__fmul_rn(static_cast<float>(rest), 0x1p-63f), &s, &c);
  if (quadrant & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  return quadrant & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// Items of a head: with Wide, first the rotated units, then units that are
// copied. Half layout: a rotated unit is eight columns and their partners half a
// rotation further; interleaved: eight columns, four pairs. Otherwise an item is
// a pair, or a copied column.
template <int T, bool Wide, bool Interleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  pdl_enter();
  using E = Elem<T>;
  using S = typename E::type;
  extern __shared__ float2 angle[];  // [token of the block][pair]
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.per_block;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.per_block), a.tokens - t0));
  for (int i = threadIdx.x; i < tokens * a.pairs; i += kRopeThreads) {
    const int token = i / a.pairs;
    const int64_t p = a.positions ? load_index(a.positions, t0 + token, a.index_type) : a.first + t0 + token;
    float2 cs = cos_sin(static_cast<uint64_t>(p) * a.turns[i - token * a.pairs]);
    if (a.inverse) cs.y = -cs.y;
    angle[i] = make_float2(__fmul_rn(cs.x, a.factor), __fmul_rn(cs.y, a.factor));
  }
  __syncthreads();
  const uint32_t per_token = static_cast<uint32_t>(a.heads) * a.items;
  const int rotated = Wide ? (Interleaved ? a.pairs / 4 : a.pairs / 8) : a.pairs;
  for (uint32_t n = threadIdx.x; n < tokens * per_token; n += kRopeThreads) {
    const uint32_t token = a.per_block == 1 ? 0u : divide(n, a.by_token), rest = n - token * per_token;
    int head = static_cast<int>(divide(rest, a.by_items));
    const int item = static_cast<int>(rest - static_cast<uint32_t>(head) * a.items);
    const bool is_k = head >= a.q_heads;
    if (is_k) head -= a.q_heads;
    const RopeSide& side = is_k ? a.k : a.q;
    const S* in = static_cast<const S*>(side.in) + (t0 + token) * side.in_token + head * side.in_head;
    S* out = static_cast<S*>(side.out) + (t0 + token) * side.out_token + head * side.out_head;
    const float2* cs = angle + token * a.pairs;
    if (Wide) {
      Pack8<T> x;
      if (item >= rotated) {
        if (in == out) continue;
        const int c = 2 * a.pairs + 8 * (item - rotated);
        x.load(in + c);
        x.store(out + c);
        continue;
      }
      float f[8];
      x.load(in + 8 * item);
      if (Interleaved) {
        x.get(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 w = cs[4 * item + i];
          const float u = f[2 * i], v = f[2 * i + 1];
          f[2 * i] = __fmaf_rn(u, w.x, -__fmul_rn(v, w.y));
          f[2 * i + 1] = __fmaf_rn(u, w.y, __fmul_rn(v, w.x));
        }
        x.put(f);
        x.store(out + 8 * item);
      } else {
        Pack8<T> y;
        float g[8];
        y.load(in + a.pairs + 8 * item);
        x.get(f);
        y.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 w = cs[8 * item + i];
          const float u = f[i], v = g[i];
          f[i] = __fmaf_rn(u, w.x, -__fmul_rn(v, w.y));
          g[i] = __fmaf_rn(u, w.y, __fmul_rn(v, w.x));
        }
        x.put(f);
        y.put(g);
        x.store(out + 8 * item);
        y.store(out + a.pairs + 8 * item);
      }
    } else {
      if (item >= rotated) {
        if (in != out) out[a.pairs + item] = in[a.pairs + item];
        continue;
      }
      const int i = Interleaved ? 2 * item : item, j = Interleaved ? i + 1 : item + a.pairs;
      const float2 w = cs[item];
      const float u = E::get(in[i]), v = E::get(in[j]);
      out[i] = E::put(__fmaf_rn(u, w.x, -__fmul_rn(v, w.y)));
      out[j] = E::put(__fmaf_rn(u, w.y, __fmul_rn(v, w.x)));
    }
  }
}

// Distances of [tokens, heads, head_dim] without overlaps, tokens or heads outermost.
bool side_ok(const RopeSide& s, int64_t tokens, int64_t heads, int64_t head_dim) {
  const auto fits = [&](int64_t token, int64_t head) {
    if (tokens <= 1) token = head_dim;
    if (heads <= 1) head = head_dim;
    if (!stride_ok(head, head_dim) || !stride_ok(token, head_dim)) return false;
    const auto outer = [&](int64_t far, int64_t near, int64_t n) {
      return n <= 1 || (far - head_dim) / (n - 1) >= near;
    };
    return outer(token, head, heads) || outer(head, token, tokens);
  };
  return heads == 0 || (fits(s.out_token, s.out_head) && fits(s.in_token, s.in_head));
}

bool side_alias_ok(const RopeSide& s, int64_t tokens, int heads) {
  return heads == 0 || s.out != s.in ||
         ((tokens == 1 || s.out_token == s.in_token) && (heads == 1 || s.out_head == s.in_head));
}

bool side_aligned(const RopeSide& s, int heads, int32_t type) {
  return heads == 0 || (type_aligned(s.out, type) && type_aligned(s.in, type));
}

bool side_wide(const RopeSide& s, int heads, int64_t tokens, int32_t type) {
  const int64_t unit = type == MP_FP32 ? 4 : 8;
  const auto ok = [&](const void* p, int64_t token, int64_t head) {
    return aligned_to(p, 16) && (tokens <= 1 || token % unit == 0) && (heads <= 1 || head % unit == 0);
  };
  return heads == 0 || (ok(s.out, s.out_token, s.out_head) && ok(s.in, s.in_token, s.in_head));
}

template <int T>
cudaError_t rope(RopeArgs& a, int head_dim, int k_heads, bool interleaved, cudaStream_t s) {
  const bool wide = side_wide(a.q, a.q_heads, a.tokens, T) && side_wide(a.k, k_heads, a.tokens, T) &&
                    head_dim % 8 == 0 && a.pairs % (interleaved ? 4 : 8) == 0;
  const int rest = head_dim - 2 * a.pairs;
  a.items = wide ? (interleaved ? a.pairs / 4 : a.pairs / 8) + rest / 8 : a.pairs + rest;
  const int64_t per_token = static_cast<int64_t>(a.heads) * a.items;
  // Tokens of a block: several rounds of its threads, angles within 16 KB.
  a.per_block = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({(4 * kRopeThreads + per_token - 1) / per_token, 2048 / a.pairs, a.tokens / (2 * kRopeSms)})));
  a.by_items = divisor(static_cast<uint32_t>(a.items));
  a.by_token = divisor(static_cast<uint32_t>(per_token));
  const int64_t blocks = (a.tokens + a.per_block - 1) / a.per_block;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = static_cast<size_t>(a.per_block) * a.pairs * sizeof(float2);
  const auto kernel = wide ? (interleaved ? rope_kernel<T, true, true> : rope_kernel<T, true, false>)
                           : (interleaved ? rope_kernel<T, false, true> : rope_kernel<T, false, false>);
  return launch_pdl_smem(kernel, static_cast<unsigned>(blocks), kRopeThreads, smem, s, a);
}

}  // namespace
}  // namespace mpk

extern "C" int mp_rope(void* q_out, const void* q, void* k_out, const void* k, const uint64_t* turns,
                       const void* positions, int64_t first_position, int64_t tokens, int32_t q_heads,
                       int32_t k_heads, int32_t head_dim, int32_t rotary_dim, int64_t q_out_token_stride,
                       int64_t q_out_head_stride, int64_t q_token_stride, int64_t q_head_stride,
                       int64_t k_out_token_stride, int64_t k_out_head_stride, int64_t k_token_stride,
                       int64_t k_head_stride, float factor, int32_t interleaved, int32_t inverse, int32_t type,
                       int32_t index_type, void* stream) {
  using namespace mpk;
  RopeArgs a = {};
  a.q = {q_out, q, q_out_token_stride, q_out_head_stride, q_token_stride, q_head_stride};
  a.k = {k_out, k, k_out_token_stride, k_out_head_stride, k_token_stride, k_head_stride};
  if (!type_ok(type) || !index_type_ok(index_type) || tokens < 0 || tokens > INT32_MAX || q_heads < 0 || q_heads > kMaxHeads ||
      k_heads < 0 || k_heads > kMaxHeads || q_heads + k_heads == 0 || head_dim < 2 || head_dim > kMaxHeadDim ||
      rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2 || !std::isfinite(factor) ||
      !side_ok(a.q, tokens, q_heads, head_dim) || !side_ok(a.k, tokens, k_heads, head_dim))
    return MP_ERR_RANGE;
  if (tokens == 0) return MP_OK;
  if (!turns || (q_heads && (!q_out || !q)) || (k_heads && (!k_out || !k))) return MP_ERR_NULL;
  if (!side_alias_ok(a.q, tokens, q_heads) || !side_alias_ok(a.k, tokens, k_heads) || (q_heads && k_heads && q_out == k_out))
    return MP_ERR_RANGE;
  if (!side_aligned(a.q, q_heads, type) || !side_aligned(a.k, k_heads, type) || !aligned_to(turns, 8) ||
      !index_aligned(positions, index_type))
    return MP_ERR_ALIGN;
  a.turns = turns;
  a.positions = positions;
  a.first = first_position;
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.heads = q_heads + k_heads;
  a.pairs = rotary_dim / 2;
  a.factor = factor;
  a.index_type = index_type;
  a.inverse = inverse != 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == MP_BF16   ? rope<MP_BF16>(a, head_dim, k_heads, interleaved != 0, s)
                        : type == MP_FP16 ? rope<MP_FP16>(a, head_dim, k_heads, interleaved != 0, s)
                                          : rope<MP_FP32>(a, head_dim, k_heads, interleaved != 0, s);
  return e == cudaSuccess ? MP_OK : record_cuda_error(e);
}

extern "C" int mp_rope_frequencies(uint64_t* turns, float* factor, int32_t rotary_dim, double base,
                                   const mp_rope_scaling_t* scaling) {
  using namespace mpk;
  constexpr double kTurn = 6.283185307179586476925;
  const int kind = scaling ? scaling->kind : MP_ROPE_NONE;
  if (rotary_dim < 2 || rotary_dim > kMaxHeadDim || rotary_dim % 2 || !(base > 1.0) || !std::isfinite(base) ||
      kind < MP_ROPE_NONE || kind > MP_ROPE_RAMP)
    return MP_ERR_RANGE;
  const mp_rope_scaling_t by = scaling ? *scaling : mp_rope_scaling_t{};
  if (kind != MP_ROPE_NONE && (!(by.factor >= 1.0) || !std::isfinite(by.factor))) return MP_ERR_RANGE;
  if ((kind == MP_ROPE_BANDS || kind == MP_ROPE_RAMP) &&
      (!(by.context > 0.0) || !std::isfinite(by.context) || !(by.low > 0.0) || !(by.high > by.low) ||
       !std::isfinite(by.high)))
    return MP_ERR_RANGE;
  if (!turns) return MP_ERR_NULL;
  const double r = rotary_dim;
  if (kind == MP_ROPE_BASE && rotary_dim > 2) base *= std::pow(by.factor, r / (r - 2.0));
  if (!std::isfinite(base)) return MP_ERR_RANGE;
  // the pair of the frequency that makes u turns in the context
  const auto pair_of = [&](double u) { return r * std::log(by.context / (u * kTurn)) / (2.0 * std::log(base)); };
  const double lo = kind == MP_ROPE_RAMP ? std::max(0.0, std::floor(pair_of(by.high))) : 0.0;
  const double hi = kind == MP_ROPE_RAMP ? std::min(r - 1.0, std::ceil(pair_of(by.low))) : 0.0;
  const auto limited = [](double s) { return std::min(1.0, std::max(0.0, s)); };
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (kind == MP_ROPE_LINEAR) f /= by.factor;
    if (kind == MP_ROPE_BANDS) {
      const double s = limited((by.context * f / kTurn - by.low) / (by.high - by.low));
      f *= (1.0 - s) / by.factor + s;
    }
    if (kind == MP_ROPE_RAMP) {
      const double s = limited((i - lo) / std::max(hi - lo, 0.001));
      f *= s / by.factor + 1.0 - s;
    }
    turns[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f / kTurn, 64)));  // f <= 1
  }
  if (factor) *factor = kind == MP_ROPE_RAMP ? static_cast<float>(0.1 * std::log(by.factor) + 1.0) : 1.0f;
  return MP_OK;
}
