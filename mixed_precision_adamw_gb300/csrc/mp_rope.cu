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
constexpr int kMaxHeads = 1024;  // of queries, and of keys
constexpr int kMaxHeadDim = 1024;

struct RopeSide {  // queries or keys
  void* out;
  const void* in;
  int64_t out_token, out_head, in_token, in_head;
};

struct RopeArgs {
  RopeSide side[2];
  int heads[2];
  const uint64_t* turns;
  const void* positions;
  int64_t first, tokens;
  int head_dim, pairs;   // pairs: rotary_dim / 2
  int items;             // of a head, each a lane's
  int angles;            // in shared memory, of a token
  int tokens_per_block;
  uint32_t by_items, by_heads;  // multipliers of the divisions by items and by the number of heads
  float factor;
  int index_type;
  int inverse;
};

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

// The angles of `tokens` tokens from t0 on, in shared memory: (cos, sin) * factor,
// put(token's, pair, (cos, sin)).
template <typename Put>
__device__ __forceinline__ void make_angles(float2* angle, const RopeArgs& a, int64_t t0, int tokens, Put put) {
  for (int i = threadIdx.x; i < tokens * a.pairs; i += kRopeThreads) {
    const int token = i / a.pairs;
    const int64_t p = a.positions ? load_index(a.positions, t0 + token, a.index_type) : a.first + t0 + token;
    float2 cs = cos_sin(static_cast<uint64_t>(p) * a.turns[i - token * a.pairs]);
    if (a.inverse) cs.y = -cs.y;
    put(angle + token * a.angles, i - token * a.pairs, make_float2(__fmul_rn(cs.x, a.factor), __fmul_rn(cs.y, a.factor)));
  }
}

// One for each pair.
struct PairAngles {
  static __host__ __device__ int angles(const RopeArgs& a) { return a.pairs; }
  static __device__ __forceinline__ void put(const RopeArgs&, float2* angle, int pair, float2 w) { angle[pair] = w; }
};

// A pair's column rotated by (cos, sin): the first with its partner's sign turned.
__device__ __forceinline__ float turned(float own, float other, float2 w) {
  return __fmaf_rn(other, w.y, __fmul_rn(own, w.x));
}
__device__ __forceinline__ void rotate(float& x, float& y, float2 w) {
  const float u = x, v = y;
  x = turned(u, -v, w);
  y = turned(v, u, w);
}

// What a lane has of a head at a time, eight columns an access, on the 16-byte grid.
//
// Half layout, whole vectors of pairs: two vectors, eight pairs (or of the copied columns).
template <int T>
struct HalfItem : PairAngles {
  using E = typename Elem<T>::type;
  static constexpr int kBlocks = T == MP_FP32 ? 6 : 8;  // of an SM
  static constexpr int kRounds = T == MP_FP32 ? 2 : 4;  // of a block's threads
  Pack8<T> x, y;

  static __device__ __forceinline__ int rest(const RopeArgs& a) { return (a.head_dim - 2 * a.pairs) / 8; }
  // columns of the second vector after the first's, 0 if there is none
  static __device__ __forceinline__ int first(const RopeArgs& a, int item) {
    const int j = item - a.pairs / 8;
    return j < 0 ? 8 * item : 2 * a.pairs + 8 * j;
  }
  static __device__ __forceinline__ int apart(const RopeArgs& a, int item) {
    const int j = item - a.pairs / 8, n = rest(a), half = (n + 1) / 2;
    return j < 0 ? a.pairs : j + half < n ? 8 * half : 0;
  }
  __device__ __forceinline__ void load(const RopeArgs& a, const E* head, int item) {
    const E* p = head + first(a, item);
    const int q = apart(a, item);
    x.load(p);
    if (q) y.load(p + q);
  }
  __device__ __forceinline__ void finish(const RopeArgs& a, E* head, const float2* cs, int item) {
    E* p = head + first(a, item);
    const int q = apart(a, item);
    if (item < a.pairs / 8) {
      float f[8], g[8];
      x.get(f);
      y.get(g);
      const float4* w = reinterpret_cast<const float4*>(cs + 8 * item);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = w[i];
        rotate(f[2 * i], g[2 * i], make_float2(v.x, v.y));
        rotate(f[2 * i + 1], g[2 * i + 1], make_float2(v.z, v.w));
      }
      x.put(f);
      y.put(g);
    }
    x.store(p);
    if (q) y.store(p + q);
  }
};

// The partners of columns c to c + 7, c a multiple of 8 below 2 h, h = pairs, in the
// half layout: what lies h after the columns up to h and h before the others, cut out of
// the 16-byte pieces that it is in. Only of columns on both sides of h are three
// pieces needed: two after, and the head's first. A piece is of the head
// altogether or not at all. Columns past the rotation get anything.
template <int T>
struct Partners {
  uint4 lo, hi, first;

  __device__ __forceinline__ void load(const RopeArgs& a, const uint16_t* head, int c) {
    const int h = a.pairs, q = c < h ? c + h : c - h;
    const uint4* base = reinterpret_cast<const uint4*>(head);
    lo = base[q / 8];
    hi = q % 8 && q / 8 + 1 < a.head_dim / 8 ? base[q / 8 + 1] : make_uint4(0u, 0u, 0u, 0u);
    if (c < h && c + 8 > h) first = base[0];
  }
  __device__ __forceinline__ F8 get(const RopeArgs& a, int c) const {
    const int h = a.pairs, m = h - c;
    Pack8<T> y;
    y.across(place(c < h ? c + h : c - h), lo, hi);
    if (m > 0 && m < 8) {
      Pack8<T> z;
      z.across(place(8 - m), make_uint4(0u, 0u, 0u, 0u), first);
      y.v = make_uint4(joined(y.v.x, z.v.x, m), joined(y.v.y, z.v.y, m - 2), joined(y.v.z, z.v.z, m - 4),
                       joined(y.v.w, z.v.w, m - 6));
    }
    return get8(y);
  }
  // A column's place on the grid that the pieces lie on.
  static __device__ __forceinline__ const uint16_t* place(int column) {
    return reinterpret_cast<const uint16_t*>(static_cast<uintptr_t>(2 * column));
  }
  // The first m of a's two columns, the others of b.
  static __device__ __forceinline__ uint32_t joined(uint32_t a, uint32_t b, int m) {
    return m >= 2 ? a : m <= 0 ? b : __byte_perm(a, b, 0x7610);
  }
};

template <>
struct Partners<MP_FP32> {
  float p[8];

  __device__ __forceinline__ void load(const RopeArgs& a, const float* head, int c) {
    const int h = a.pairs;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = c + e;
      p[e] = k < 2 * h ? head[k < h ? k + h : k - h] : 0.0f;
    }
  }
  __device__ __forceinline__ F8 get(const RopeArgs&, int) const {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = make_float2(p[2 * i], p[2 * i + 1]);
    return r;
  }
};

// Half layout, any number of pairs: eight columns, and their partners, which lie
// off the grid.
template <int T>
struct AnyHalfItem {
  using E = typename Elem<T>::type;
  static constexpr int kBlocks = 5, kRounds = T == MP_FP32 ? 4 : 8;
  Pack8<T> x;
  Partners<T> partners;

  // One angle for each column, the sine with the sign that the partner has in its sum:
  // (cos, cos, sin, sin) of two neighbours, those that the items have at one place
  // side by side, for access without bank conflicts (16384 x 40 heads of 80, 50
  // columns rotated, bf16: 71 us with the pairs' angles in a row, 56 this way; a pair at
  // a time 139).
  static __host__ __device__ int angles(const RopeArgs& a) { return a.head_dim; }
  static __device__ __forceinline__ void put(const RopeArgs& a, float2* angle, int pair, float2 w) {
    const auto at = [&](int c, float sine) {
      float* p = reinterpret_cast<float*>(angle) + 4 * (c % 8 / 2 * a.items + c / 8) + c % 2;
      p[0] = w.x;
      p[2] = sine;
    };
    at(pair, -w.y);
    at(pair + a.pairs, w.y);
  }

  __device__ __forceinline__ void load(const RopeArgs& a, const E* head, int item) {
    x.load(head + 8 * item);
    if (8 * item < 2 * a.pairs) partners.load(a, head, 8 * item);
  }
  __device__ __forceinline__ void finish(const RopeArgs& a, E* head, const float2* cs, int item) {
    const int c = 8 * item, n = 2 * a.pairs;
    if (c < n) {
      const F8 f = get8(x), g = partners.get(a, c);
      const float4* w = reinterpret_cast<const float4*>(cs) + item;
      F8 r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = w[i * a.items];
        const float2 t = fma2(g.p[i], make_float2(v.z, v.w), mul2(f.p[i], make_float2(v.x, v.y)));
        r.p[i] = T != MP_FP32 || c + 2 * i < n ? t : f.p[i];
      }
      if constexpr (T == MP_FP32) {
        put8(x, r);
      } else {  // what is past the rotation stays bit by bit
        Pack8<T> y;
        put8(y, r);
        x.v = make_uint4(y.v.x, c + 2 < n ? y.v.y : x.v.y, c + 4 < n ? y.v.z : x.v.z, c + 6 < n ? y.v.w : x.v.w);
      }
    }
    x.store(head + c);
  }
};

// Interleaved: two vectors, four pairs each.
template <int T>
struct InterleavedItem : PairAngles {
  using E = typename Elem<T>::type;
  static constexpr int kBlocks = T == MP_FP32 ? 6 : 8, kRounds = 2;
  Pack8<T> x[2];

  static __device__ __forceinline__ bool second(const RopeArgs& a, int item) {
    return 8 * (item + a.items) < a.head_dim;
  }
  __device__ __forceinline__ void load(const RopeArgs& a, const E* head, int item) {
    x[0].load(head + 8 * item);
    if (second(a, item)) x[1].load(head + 8 * (item + a.items));
  }
  __device__ __forceinline__ void finish(const RopeArgs& a, E* head, const float2* cs, int item) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = item + k * a.items;
      if (k && !second(a, item)) break;
      if (4 * j < a.pairs) {
        if constexpr (T == MP_FP32) {
          float f[8];
          x[k].get(f);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * j + i < a.pairs) rotate(f[2 * i], f[2 * i + 1], cs[4 * j + i]);
          x[k].put(f);
        } else {  // a pair a word; what is past the rotation stays bit by bit
          const int most = min(a.pairs - 4 * j, 4);
          const float2* c = cs + 4 * j;
          uint32_t w[4] = {x[k].v.x, x[k].v.y, x[k].v.z, x[k].v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < most) {
              float f = Elem<T>::get(static_cast<uint16_t>(w[i])), g = Elem<T>::get(static_cast<uint16_t>(w[i] >> 16));
              rotate(f, g, c[i]);
              w[i] = T == MP_BF16 ? pack2_bf16(f, g) : pack2_fp16(f, g);
            }
          x[k].v = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      x[k].store(head + 8 * j);
    }
  }
};

// n / d with m = floor(2^32 / d) + 1, for n d < 2^32; d = 1 has m = 0.
__device__ __forceinline__ int divide(int n, uint32_t m) {
  return m ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), m)) : n;
}
inline uint32_t divisor(int d) { return d == 1 ? 0u : static_cast<uint32_t>((uint64_t{1} << 32) / d + 1); }

// A block takes a few tokens, a lane one item at a time of all their heads, those of
// queries and keys counted together. With 32 to 40 registers six to eight blocks an SM
// hide each other's angles and loads: 16384 x (32 + 8) x 128 bf16 in 52 us; holding
// four items a lane, loaded before the angles, 67.
template <int T, typename Item>
__global__ void __launch_bounds__(kRopeThreads, Item::kBlocks) rope_kernel(RopeArgs a) {
  pdl_enter();
  using S = typename Elem<T>::type;
  extern __shared__ __align__(16) float2 angle[];  // [token of the block][angles]
  const int heads = a.heads[0] + a.heads[1];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tokens_per_block), a.tokens - t0));
  make_angles(angle, a, t0, tokens, [&](float2* of, int pair, float2 w) { Item::put(a, of, pair, w); });
  __syncthreads();
  for (int n = threadIdx.x; n < tokens * heads * a.items; n += kRopeThreads) {
    const int row = divide(n, a.by_items), item = n - row * a.items;
    const int token = a.tokens_per_block == 1 ? 0 : divide(row, a.by_heads);
    int head = row - token * heads;
    const bool is_k = head >= a.heads[0];
    if (is_k) head -= a.heads[0];
    const RopeSide& s = a.side[is_k];
    Item part;
    part.load(a, static_cast<const S*>(s.in) + (t0 + token) * s.in_token + head * s.in_head, item);
    part.finish(a, static_cast<S*>(s.out) + (t0 + token) * s.out_token + head * s.out_head, angle + token * a.angles,
                item);
  }
}

// Heads off the 16-byte grid: a pair, or two columns that are copied, at a time. A
// thread has one of every slots-th head of a block's tokens, queries first, so that
// per head it only moves its pointers on.
template <int T, bool Interleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_pairs_kernel(RopeArgs a) {
  pdl_enter();
  using E = Elem<T>;
  using S = typename E::type;
  extern __shared__ __align__(16) float2 angle[];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tokens_per_block), a.tokens - t0));
  make_angles(angle, a, t0, tokens, [&](float2* of, int pair, float2 w) { of[pair] = w; });
  __syncthreads();
  const int lanes = min(a.items, kRopeThreads), slots = kRopeThreads / lanes, slot = threadIdx.x / lanes;
  if (slot >= slots) return;
  const int rest = a.head_dim - 2 * a.pairs, half = (rest + 1) / 2;
  for (int item = threadIdx.x - slot * lanes; item < a.items; item += lanes) {
    const int j = item - a.pairs;
    const bool turns = j < 0, second = turns || j + half < rest;
    const int c0 = turns ? (Interleaved ? 2 * item : item) : 2 * a.pairs + j;
    const int c1 = turns ? (Interleaved ? c0 + 1 : c0 + a.pairs) : c0 + half;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const RopeSide& s = a.side[k];
      const int heads = a.heads[k];
      if (heads == 0 || (!turns && s.in == s.out)) continue;
      int token = slot / heads, head = slot - token * heads;
      const int dt = slots / heads, dh = slots - dt * heads;
      const S* in = static_cast<const S*>(s.in) + (t0 + token) * s.in_token + head * s.in_head;
      S* out = static_cast<S*>(s.out) + (t0 + token) * s.out_token + head * s.out_head;
      const int64_t in_step = dt * s.in_token + dh * s.in_head, in_wrap = s.in_token - heads * s.in_head;
      const int64_t out_step = dt * s.out_token + dh * s.out_head, out_wrap = s.out_token - heads * s.out_head;
      while (token < tokens) {
        S x = in[c0], y = {};
        if (second) y = in[c1];
        if (turns) {
          float f = E::get(x), g = E::get(y);
          rotate(f, g, angle[token * a.pairs + item]);
          x = E::put(f);
          y = E::put(g);
        }
        out[c0] = x;
        if (second) out[c1] = y;
        token += dt;
        head += dh;
        in += in_step;
        out += out_step;
        if (head >= heads) {
          head -= heads;
          ++token;
          in += in_wrap;
          out += out_wrap;
        }
      }
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

// Whether a side's heads lie on the 16-byte grid.
bool side_wide(const RopeSide& s, int64_t tokens, int heads, int32_t type) {
  const int64_t unit = type == MP_FP32 ? 4 : 8;
  const auto ok = [&](const void* p, int64_t token, int64_t head) {
    return aligned_to(p, 16) && (tokens <= 1 || token % unit == 0) && (heads <= 1 || head % unit == 0);
  };
  return heads == 0 || (ok(s.out, s.out_token, s.out_head) && ok(s.in, s.in_token, s.in_head));
}

// Tokens of a block: `rounds` rounds of its threads, angles within 16 KB, and one
// wave of blocks where there are few tokens (4097 x 40 heads of 128 bf16 in 16.5 us,
// rounded down 17.7; 5110 x 2 heads of 96 in 3.1 instead of 3.7; 4097 x 24 of 64 fp32 in
// 11.1 instead of 10.9).
//
// More rounds make the angles of more tokens at once and have fewer starts, fewer
// overlap one block's angles with another's loads (us with 2 / 4 / 8 rounds, 16384 x 40
// heads, 8192 of fp32): half layout bf16 128 54.6 / 53.2 / 54.3, 80 39.3 / 37.8 / 40.2,
// fp32 128 52.0 / 57.1 / 63.0; interleaved bf16 128 51.4 / 52.5 / 54.8; 50 of 80 columns
// bf16 62.9 / 58.5 / 55.8, 34 of 64 fp32 59.9 / 57.1 / 59.4.
int tokens_of_block(const RopeArgs& a, int rounds) {
  const int64_t per_token = static_cast<int64_t>(a.heads[0] + a.heads[1]) * a.items, wave = 8 * kRopeSms;
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({(rounds * kRopeThreads + per_token - 1) / per_token, 2048 / a.angles,
                            (a.tokens + wave - 1) / wave})));
}

cudaError_t rope_launch(void (*kernel)(RopeArgs), RopeArgs& a, int items, int angles, int rounds, cudaStream_t s) {
  a.items = items;
  a.angles = angles;
  a.tokens_per_block = tokens_of_block(a, rounds);
  // n < tokens heads items, below 2048 + heads items: n items < 2^32
  a.by_items = divisor(items);
  a.by_heads = divisor(a.heads[0] + a.heads[1]);
  const int64_t blocks = (a.tokens + a.tokens_per_block - 1) / a.tokens_per_block;
  const size_t smem = static_cast<size_t>(a.tokens_per_block) * a.angles * sizeof(float2);
  return launch_pdl_smem(kernel, static_cast<unsigned>(blocks), kRopeThreads, smem, s, a);
}

template <int T, typename Item>
cudaError_t rope_items(RopeArgs& a, int items, cudaStream_t s) {
  return rope_launch(rope_kernel<T, Item>, a, items, Item::angles(a), Item::kRounds, s);
}

template <int T>
cudaError_t rope(RopeArgs& a, bool interleaved, cudaStream_t s) {
  const int rest = a.head_dim - 2 * a.pairs;
  const bool over = (a.heads[0] && a.side[0].in == a.side[0].out) || (a.heads[1] && a.side[1].in == a.side[1].out);
  if (a.head_dim % 8 == 0 && side_wide(a.side[0], a.tokens, a.heads[0], T) &&
      side_wide(a.side[1], a.tokens, a.heads[1], T)) {
    if (interleaved) return rope_items<T, InterleavedItem<T>>(a, (a.head_dim / 8 + 1) / 2, s);
    if (a.pairs % 8 == 0) return rope_items<T, HalfItem<T>>(a, a.pairs / 8 + (rest / 8 + 1) / 2, s);
    // over its input a pair has to be one lane's
    if (!over) return rope_items<T, AnyHalfItem<T>>(a, a.head_dim / 8, s);
  }
  return rope_launch(interleaved ? rope_pairs_kernel<T, true> : rope_pairs_kernel<T, false>, a,
                     a.pairs + (rest + 1) / 2, a.pairs, 4, s);
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
  a.side[0] = {q_out, q, q_out_token_stride, q_out_head_stride, q_token_stride, q_head_stride};
  a.side[1] = {k_out, k, k_out_token_stride, k_out_head_stride, k_token_stride, k_head_stride};
  if (!type_ok(type) || !index_type_ok(index_type) || tokens < 0 || tokens > INT32_MAX || q_heads < 0 ||
      q_heads > kMaxHeads || k_heads < 0 || k_heads > kMaxHeads || q_heads + k_heads == 0 || head_dim < 2 ||
      head_dim > kMaxHeadDim || rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2 || !std::isfinite(factor) ||
      !side_ok(a.side[0], tokens, q_heads, head_dim) || !side_ok(a.side[1], tokens, k_heads, head_dim))
    return MP_ERR_RANGE;
  if (tokens == 0) return MP_OK;
  if (!turns || (q_heads && (!q_out || !q)) || (k_heads && (!k_out || !k))) return MP_ERR_NULL;
  if (!side_alias_ok(a.side[0], tokens, q_heads) || !side_alias_ok(a.side[1], tokens, k_heads) ||
      (q_heads && k_heads && (q_out == k_out || q_out == k || k_out == q)))
    return MP_ERR_RANGE;
  if (!side_aligned(a.side[0], q_heads, type) || !side_aligned(a.side[1], k_heads, type) || !aligned_to(turns, 8) ||
      !index_aligned(positions, index_type))
    return MP_ERR_ALIGN;
  a.heads[0] = q_heads;
  a.heads[1] = k_heads;
  a.turns = turns;
  a.positions = positions;
  a.first = first_position;
  a.tokens = tokens;
  a.head_dim = head_dim;
  a.pairs = rotary_dim / 2;
  a.factor = factor;
  a.index_type = index_type;
  a.inverse = inverse != 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == MP_BF16   ? rope<MP_BF16>(a, interleaved != 0, s)
                        : type == MP_FP16 ? rope<MP_FP16>(a, interleaved != 0, s)
                                          : rope<MP_FP32>(a, interleaved != 0, s);
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
