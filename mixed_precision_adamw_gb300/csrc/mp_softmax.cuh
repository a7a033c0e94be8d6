// mp_softmax.cuh — one pass over a row of logits (or a segment of one): the
// sum of exponentials relative to a running reference, and with it the sum
// that gives the entropy.
//
// With c = scale * log2(e), a reference R in log2 units and t = c x - R (one
// FMA, rounded once):
//   s = sum 2^t,   u = sum t 2^t
// and with delta = c m - R for the largest element m and L = log2(s / 2^delta)
//   lse = scale m + L ln 2,   entropy = (delta + L - u / s) ln 2
//   log p(x) = scale (x - m) - L ln 2
// (L is exactly 0, and with it the largest element's log p, where one element
// has all the probability.) R is whatever rounded value is subtracted, so its
// own rounding costs nothing as long as it is small against 1, which is what
// delta is then: |R| stays below 2^24, where half a step of fp32 is 1/2. A
// maximum below that range takes R = -2^24, whose terms are 0 beside those of
// any row that is not wholly down there; rows whose reference ends outside it
// (masked throughout with -1e9, say) are summed again from differences. The
// rounding of c is a relative change of the scale by at most 2^-24. R follows
// the running maximum lazily: it moves only when a chunk's maximum exceeds the
// one it was taken from by 8 / c, so a rescale is rare and no term grows past
// 2^9. Against t = (x - m) c it saves an operation of eight an element (8192 x
// 50304 bf16 with entropy: 133 us, 148 with the difference).
#pragma once

#include <cooperative_groups.h>

#include "mp_rows.cuh"

namespace mpk {

constexpr float kSlack = 8.0f;       // log2 units R may lag behind the maximum
constexpr float kFar = 16777216.0f;  // 2^24: bound of |R|
constexpr float kLowest = -200.0f;   // 2^-200 is 0: t below it counts as it (its product with 2^t is 0)

struct RowStats {
  float R;    // reference in log2 units; -inf: no element yet (s and u mean nothing)
  float lim;  // a maximum above this moves R
  float s, u;
  float m;    // largest element

  __device__ __forceinline__ void clear() {
    R = lim = m = -kInf;
    s = u = 0.0f;
  }
};

// Brings the sums from their reference to R.
__device__ __forceinline__ void rebase(RowStats& a, float R) {
  if (a.R == -kInf) {
    a.s = a.u = 0.0f;
  } else {
    const float d = max_nan(__fsub_rn(a.R, R), kLowest), f = exp2_fast(d);
    a.u = __fmul_rn(f, __fmaf_rn(d, a.s, a.u));
    a.s = __fmul_rn(f, a.s);
  }
  a.R = R;
}

// Takes note of a maximum, and moves the reference to it if it has to.
__device__ __forceinline__ void note_maximum(RowStats& a, float top, float c, float slack) {
  a.m = max_nan(a.m, top);
  if (top <= a.lim) return;
  rebase(a, max_nan(__fmul_rn(top, c), -kFar));
  a.lim = __fadd_rn(top, slack);
}

// Adds `n` of U units from the q0-th on; the reference has been moved.
template <int T, int U, bool Entropy>
__device__ __forceinline__ void add_units(RowStats& a, const Pack8<T> (&x)[U], int q0, int n, float c) {
  const float R = a.R;
#pragma unroll
  for (int q = 0; q < U; ++q) {
    if (q < q0 || q >= q0 + n) continue;
    float f[8];
    x[q].get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float t = __fmaf_rn(f[e], c, -R);
      if (Entropy) t = max_nan(t, kLowest);
      const float p = exp2_fast(t);
      a.s = __fadd_rn(a.s, p);
      if (Entropy) a.u = __fmaf_rn(p, t, a.u);
    }
  }
}

// A row, or the part [first, last) of its units, as the threads of a block
// read it: whole units on 16-B boundaries, and the fewer than 16 elements
// before and after them one by one (read by the first part's threads).
template <int T>
struct RowPart {
  using E = typename Elem<T>::type;
  const E* row;
  const E* body;        // row + head, 16-B aligned
  int64_t first, last;  // units
  int head, extra;      // elements before the units; before and after them (0 unless this is part 0)
  int64_t units, n;

  __device__ __forceinline__ RowPart(const E* p, int64_t length, int part, int parts) : row(p), n(length) {
    constexpr int kAlign = 16 / sizeof(E);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) / sizeof(E) % kAlign);
    head = off ? kAlign - off : 0;
    if (head > n) head = static_cast<int>(n);
    units = (n - head) / 8;
    body = p + head;
    first = units * part / parts;
    last = units * (part + 1) / parts;
    extra = part == 0 ? static_cast<int>(n - 8 * units) : 0;
  }
  // whether element j is this part's
  __device__ __forceinline__ bool holds(int64_t j) const {
    if (j < head || j >= head + 8 * units) return extra > 0;
    return j >= head + 8 * first && j < head + 8 * last;
  }
  // index of the i-th extra element
  __device__ __forceinline__ int64_t extra_index(int i) const { return i < head ? i : 8 * units + i; }
};

template <int T, int U>
__device__ __forceinline__ void load_units(Pack8<T> (&x)[U], const RowPart<T>& p, int64_t unit, int64_t step) {
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int64_t i = unit + q * step;
    if (i < p.last)
      x[q].load(p.body + 8 * i);
    else
      x[q].fill(Elem<T>::kMinusInf);
  }
}

// Units a thread has in flight: 64 B.
template <int T>
constexpr int kUnits = T == MP_FP32 ? 2 : 4;

// U units of eight elements of a row of n, `step` elements apart, the first
// from element j on, as far as they start before element `end`. Where they
// start on a 16-B boundary: one 16-B load each (two for fp32). Where not, with
// Across and 16-bit types the two 16-B pieces that a unit lies in, all loaded
// before the first are shifted together; units at the row's ends, whose pieces
// may reach beyond it, and the others are loaded element by element. 8192 x
// 50304 bf16 in rows of 50307: the distillation 476 us across, 590 by elements;
// the log probabilities' gradient 342 and 337, and its aligned rows 256 and 249,
// for the registers that the pieces take.
template <int T, bool Across, int U>
__device__ __forceinline__ void load_any(Pack8<T> (&x)[U], const typename Elem<T>::type* row, int64_t j, int64_t step,
                                         int64_t end, int64_t n, bool aligned) {
  if (aligned) {
#pragma unroll
    for (int q = 0; q < U; ++q)
      if (j + q * step < end) x[q].load(row + j + q * step);
    return;
  }
  constexpr bool kAcross = Across && T != MP_FP32;
  if constexpr (kAcross) {
    uint4 a[U], b[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int64_t k = j + q * step;
      a[q] = b[q] = make_uint4(0u, 0u, 0u, 0u);
      if (k < end && k >= 7 && k + 15 <= n) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row + k) & ~uintptr_t{15});
        a[q] = p[0];
        b[q] = p[1];
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) x[q].across(row + j, a[q], b[q]);  // one alignment: step is a multiple of 8
  }
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int64_t k = j + q * step;
    if (k < end && (!kAcross || k < 7 || k + 15 > n)) x[q].load_stepped(row + k, 0, 1, 8);
  }
}

// Writes f(x[j]) for a part of a row: `out` divides dx (its alignment), x is
// read to match (Across: load_any). Each thread reads what it writes, so dx
// may be x.
template <int T, bool Across, typename F>
__device__ __forceinline__ void map_row(const RowPart<T>& out, typename Elem<T>::type* dx,
                                        const typename Elem<T>::type* x, F&& f) {
  using E = typename Elem<T>::type;
  constexpr int U = kUnits<T>;
  const int threads = blockDim.x;
  const bool aligned = reinterpret_cast<uintptr_t>(x + out.head) % 16 == 0;
  for (int64_t i = out.first + threadIdx.x; i < out.last; i += static_cast<int64_t>(U) * threads) {
    Pack8<T> u[U];
    load_any<T, Across>(u, x, out.head + 8 * i, 8 * threads, out.head + 8 * out.last, out.n, aligned);
#pragma unroll
    for (int q = 0; q < U; ++q)
      if (i + q * threads < out.last) {
        float v[8];
        u[q].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f(v[e]);
        u[q].put(v);
        u[q].store(dx + out.head + 8 * (i + q * threads));
      }
  }
  if (threadIdx.x < out.extra) {
    const int64_t j = out.extra_index(threadIdx.x);
    dx[j] = Elem<T>::put(f(Elem<T>::get(x[j])));
  }
}

template <int T>
__device__ __forceinline__ void zero_row(const RowPart<T>& out, typename Elem<T>::type* dx) {
  Pack8<T> z;
  z.zero();
  for (int64_t i = out.first + threadIdx.x; i < out.last; i += blockDim.x) z.store(dx + out.head + 8 * i);
  if (threadIdx.x < out.extra) dx[out.extra_index(threadIdx.x)] = Elem<T>::put(0.0f);
}

// A part's first chunk, to be loaded before scan_row.
template <int T>
__device__ __forceinline__ void first_chunk(Pack8<T> (&x)[kUnits<T>], const RowPart<T>& p, int t, int threads) {
  load_units(x, p, p.first + t, threads);
}

// The whole part, by `threads` threads, of which this is the t-th; x holds its
// first chunk. chunk(top) is called with each chunk's maximum, in the order of the
// chunks: chunk i of the thread is the units first + (i U + q) threads + t,
// q < U. ahead(x) is called once, before the last chunk is added, to load what
// comes after the part.
template <int T, bool Entropy, typename Chunk, typename Ahead>
__device__ __forceinline__ void scan_row(RowStats& a, Pack8<T> (&x)[kUnits<T>], const RowPart<T>& p, int t, int threads,
                                         float c, float slack, Chunk&& chunk, Ahead&& ahead) {
  constexpr int U = kUnits<T>;
  const int64_t step = static_cast<int64_t>(U) * threads;
  a.clear();
  if (t < p.extra) {
    Pack8<T> one[1];
    float f[8] = {-kInf, -kInf, -kInf, -kInf, -kInf, -kInf, -kInf, -kInf};
    f[0] = Elem<T>::get(p.row[p.extra_index(t)]);
    one[0].put(f);
    note_maximum(a, f[0], c, slack);
    add_units<T, 1, Entropy>(a, one, 0, 1, c);
  }
  Pack8<T> next[U];
  int64_t i = p.first;
  for (; i + step < p.last; i += step) {
    load_units(next, p, i + step + t, threads);
    const float top = max_of<T, U>(x);
    chunk(top);
    note_maximum(a, top, c, slack);
    add_units<T, U, Entropy>(a, x, 0, U, c);
#pragma unroll
    for (int q = 0; q < U; ++q) x[q] = next[q];
  }
  ahead(next);
  if (i < p.last) {  // the last chunk, only as many units as the block still has
    const float top = max_of<T, U>(x);
    chunk(top);
    note_maximum(a, top, c, slack);
#pragma unroll
    for (int q = 0; q < U; ++q)
      if (i + q * threads < p.last) add_units<T, U, Entropy>(a, x, q, 1, c);
  }
#pragma unroll
  for (int q = 0; q < U; ++q) x[q] = next[q];
}

// Sum of a warp's statistics, to each lane.
__device__ __forceinline__ RowStats join_warp(RowStats a) {
  rebase(a, warp_max(a.R));
  a.m = warp_max(a.m);
  a.s = warp_sum(a.s);
  a.u = warp_sum(a.u);
  return a;
}

// Sum of `n` joined statistics at at(i).
template <typename At>
__device__ __forceinline__ RowStats join_all(int n, At&& at) {
  float R = at(0)->R;
#pragma unroll 1
  for (int i = 1; i < n; ++i) R = max_nan(R, at(i)->R);
  RowStats a = *at(0);
  rebase(a, R);
#pragma unroll 1
  for (int i = 1; i < n; ++i) {
    RowStats b = *at(i);
    rebase(b, R);
    a.m = max_nan(a.m, b.m);
    a.s = __fadd_rn(a.s, b.s);
    a.u = __fadd_rn(a.u, b.u);
  }
  return a;
}

// The block's statistics, to every thread. `red` has one entry per warp.
__device__ __forceinline__ RowStats join_block(RowStats a, RowStats* red) {
  a = join_warp(a);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = a;
  __syncthreads();
  return join_all(blockDim.x / 32, [&](int i) { return red + i; });
}

// The threads that finish a row: a whole block, or one warp of it.
struct BlockTeam {
  __device__ __forceinline__ static int thread() { return threadIdx.x; }
  __device__ __forceinline__ static int threads() { return blockDim.x; }
  __device__ __forceinline__ static RowStats join(const RowStats& a, RowStats* red) { return join_block(a, red); }
};

struct WarpTeam {
  __device__ __forceinline__ static int thread() { return threadIdx.x % 32; }
  __device__ __forceinline__ static int threads() { return 32; }
  __device__ __forceinline__ static RowStats join(const RowStats& a, RowStats*) { return join_warp(a); }
};

// Whether the row's finite maximum left the range of R: its statistics have to
// be taken from differences instead (difference_stats).
__device__ __forceinline__ bool out_of_range(const RowStats& a) {
  return isfinite(a.m) && !(fabsf(a.R) < kFar);
}

// The second pass over such rows, by a team over the whole row: t = (x - m) c.
// On return R is 0 and t = (x - m) c replaces c x - R. 8192 x 50304 bf16 with
// entropy: 135 us; with one row of 16, or every row, at -1e9 throughout, 288 and
// 395.
template <int T, bool Entropy, typename Team>
__device__ __noinline__ RowStats difference_stats(const typename Elem<T>::type* row, int64_t n, float m, float c,
                                                  RowStats* red) {
  constexpr int U = kUnits<T>;
  const RowPart<T> p(row, n, 0, 1);
  const int threads = Team::threads();
  RowStats a;
  a.R = 0.0f;
  a.lim = 0.0f;
  a.s = a.u = 0.0f;
  a.m = m;
  auto add = [&](float x) {
    const float t = max_nan(__fmul_rn(__fsub_rn(x, m), c), kLowest);
    const float p = exp2_fast(t);
    a.s = __fadd_rn(a.s, p);
    if (Entropy) a.u = __fmaf_rn(p, t, a.u);
  };
  if (Team::thread() < p.extra) add(Elem<T>::get(p.row[p.extra_index(Team::thread())]));
#pragma unroll 1
  for (int64_t i = Team::thread(); i < p.last; i += U * threads) {
    Pack8<T> x[U];
    load_units(x, p, i, threads);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      float f[8];
      x[q].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) add(f[e]);
    }
  }
  return Team::join(a, red);
}

// The logarithms of a row's joined statistics.
struct RowLog {
  float m, scale, log_sum, entropy, lse;
  bool empty;

  __device__ __forceinline__ RowLog(const RowStats& a, bool difference, float c, float scale_)
      : m(a.m), scale(scale_), empty(a.m == -kInf) {
    const float delta = difference ? 0.0f : __fmaf_rn(m, c, -a.R);
    const float p = exp2_fast(delta);
    const float L = log2f(__fdiv_rn(a.s, p));
    const float own = __fmul_rn(p, delta);
    // sums that hold the largest element's terms alone: one token has all the probability
    entropy = empty || (a.s == p && a.u == own)
                  ? 0.0f
                  : __fmul_rn(__fadd_rn(__fsub_rn(delta, __fdiv_rn(a.u, a.s)), L), kLn2);
    log_sum = __fmul_rn(L, kLn2);
    lse = empty ? -kInf : __fmaf_rn(m, scale, log_sum);
  }
  // log p(x) of an element of the row
  __device__ __forceinline__ float log_p(float x) const {
    return empty ? -kInf : __fmaf_rn(__fsub_rn(x, m), scale, -log_sum);
  }
};

}  // namespace mpk
