// Scores of given tokens: log probability, entropy, rank and the most likely
// alternatives of a row of logits, and the gradient.
//
// z = scale * x, p_j = exp(z_j - lse), lse = log sum exp z.  One pass over the
// row: every thread keeps the largest element so far, the sum of weights
// w_j = exp(z_j - max) and the sum of w_j (x_j - max), which give
//   log p_id = scale (x_id - max) - log sum w
//   entropy  = log sum w - scale sum w (x - max) / sum w
// with no difference of large numbers.  A token's rank counts the elements
// above it, and the equal ones before it.
//
// Gradient: with G = g_logprob + sum g_top - g_lse,
//   dz_j = -p_j (G + g_entropy (log p_j + entropy))
//          + g_logprob [j = id] + sum_t g_top_t [j = top_t].
#include "bbpe_rows.h"

#include <algorithm>

namespace bbpe {
namespace {

constexpr uint32_t TOP_MAX = 256;      // alternatives at most
constexpr uint32_t TOP_ROOM = 2048;    // candidates for them at most
static_assert(TOP_ROOM >= ROW_STEP && TOP_ROOM >= 8 * TOP_MAX, "");

struct ScoreArgs {
  const void *x;
  int64_t stride;
  uint64_t row0;
  uint32_t vocab, k;
  float scale, c;
  uint32_t index_bits;  // of a place in the row
  const int32_t *ids;
  float *logprobs, *entropy, *lse;
  int32_t *ranks;
  int32_t *top_ids;
  float *top_logprobs;
  float2 *stats;
};

// ---- order ----
// Larger elements first, and the lower place among equals: as one whole number,
// the element's bits in order above the place counted from the end.  Elements of
// 16 bits leave the lowest bits of a float the same, so those are left out.
template <typename T> struct Order {
  static constexpr uint32_t LOW = std::is_same<T, float>::value ? 0 : std::is_same<T, _Float16>::value ? 13 : 16;
};
template <typename T>
__device__ __forceinline__ uint64_t order_key(float v, uint32_t place, uint32_t bits) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // (-0 is 0)
  const uint32_t up = (b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u)) >> Order<T>::LOW;
  return uint64_t(up) << bits | (((1u << bits) - 1) - place);
}
template <typename T>
__device__ __forceinline__ float key_value(uint64_t key, uint32_t bits) {
  constexpr uint32_t ones = (1u << Order<T>::LOW) - 1;
  uint32_t up = uint32_t(key >> bits) << Order<T>::LOW;
  up = up >> 31 ? up ^ 0x80000000u : ~(up | ones);
  return __uint_as_float(up);
}
__device__ __forceinline__ uint32_t key_place(uint64_t key, uint32_t bits) {
  return ((1u << bits) - 1) - (uint32_t(key) & ((1u << bits) - 1));
}

// A number that exactly k of the n keys in LDS reach, by one wave; 1 if there
// are no more than k.  Keys differ from each other, but for absent ones, which are 0.
__device__ uint64_t kth_key(const uint64_t *keys, uint32_t n, uint32_t k) {
  const uint32_t lane = threadIdx.x & 63;
  uint64_t lo = ~uint64_t(0), hi = 0;
  uint32_t there = 0;
  for (uint32_t i = 0; i < n; i += 64) {
    const uint64_t v = i + lane < n ? keys[i + lane] : 0;
    there += uint32_t(__popcll(__ballot(v != 0)));
    if (v > hi) hi = v;
    if (v && v < lo) lo = v;
  }
  if (there <= k) return 1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t l = __shfl_xor(lo, d, 64), h = __shfl_xor(hi, d, 64);
    if (l < lo) lo = l;
    if (h > hi) hi = h;
  }
  // k or more reach lo, fewer than k reach hi + 1
  while (lo < hi) {
    const uint64_t mid = lo + (hi - lo + 1) / 2;
    uint32_t reach = 0;
    for (uint32_t i = 0; i < n; i += 64) reach += uint32_t(__popcll(__ballot(i + lane < n && keys[i + lane] >= mid)));
    if (reach == k) return mid;
    if (reach > k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The largest number below v in the order of floats; below minus infinity: NaN.
__device__ __forceinline__ float next_below(float v) {
  const uint32_t b = __float_as_uint(v);
  if (v == -INFINITY) return __uint_as_float(0x7FC00000u);
  if (v == 0.0f) return __uint_as_float(0x80000001u);
  return __uint_as_float(v > 0.0f ? b - 1 : b + 1);
}

// One workgroup a row.
//
// Alternatives.  A thread's step takes ROW_UNROLL pieces; the pieces at one
// place of all steps are a group, of which the thread keeps the largest element
// and the first piece that has it.  An element among the row's first k lies in
// one of the k groups whose largest come first: k groups without it would have
// k elements before it.  Those groups are read once more, and what reaches the
// k-th group's largest are the candidates, seldom many more than k.
template <typename T, bool TOP>
__global__ __launch_bounds__(ROW_THREADS) void k_scores(ScoreArgs a) {
  typedef Piece<T> P;
  typedef typename P::raw Raw;
  __shared__ Partial sh[ROW_WAVES];
  __shared__ uint32_t sh_rank[ROW_WAVES];
  __shared__ uint64_t keys[TOP ? TOP_ROOM : 1];
  __shared__ uint16_t chosen[TOP ? TOP_MAX : 1];
  __shared__ uint32_t n_chosen, n_found;
  __shared__ uint64_t reach;
  const uint64_t row = a.row0 + blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  const Row<const T> r(x, a.vocab);
  const uint32_t tid = threadIdx.x, pieces = r.pieces();
  const int32_t id = a.ids[row];
  const bool given = id >= 0 && uint32_t(id) < a.vocab;
  const float at_id = given ? float(x[id]) : INFINITY;  // nothing is above infinity
  const uint32_t id_piece = given ? (r.lead + uint32_t(id)) / P::N : 0;
  const float at_least = given ? next_below(at_id) : INFINITY;

  Partial s{-INFINITY, 0.0f, 0.0f};
  float ref = 0.0f;
  uint32_t above = 0;  // the wave's
  float best[ROW_UNROLL];
  uint32_t step_of[ROW_UNROLL];
  for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
    best[u] = -INFINITY;
    step_of[u] = 0;
  }
  const auto work = [&](const Raw (&raw)[ROW_UNROLL], uint32_t step) {
    typename P::val v[ROW_UNROLL];
    float m = -INFINITY;
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      v[u] = values<T>(raw[u]);
      float pm = v[u][0];
#pragma unroll
      for (uint32_t e = 1; e < P::N; ++e) pm = fmaxf(pm, v[u][e]);
      if (TOP && pm > best[u]) {
        best[u] = pm;
        step_of[u] = step;
      }
      m = fmaxf(m, pm);
    }
    if (m > s.max) {
      s = s.max == -INFINITY ? Partial{m, s.sum, 0.0f} : relative(s, m, a.c);
      ref = m;
    }
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      const uint32_t p = step * ROW_STEP + u * ROW_THREADS + tid;
      const float bar = p < id_piece ? at_least : at_id;
#pragma unroll
      for (uint32_t e = 0; e < P::N; ++e) {
        const float d = v[u][e] - ref, w = __builtin_amdgcn_exp2f(d * a.c);
        s.sum += w;
        s.mean += w * fmaxf(d, LOWEST);  // (0 times minus infinity is to be 0)
        above += uint32_t(__popcll(__ballot(!(v[u][e] <= bar))));
      }
    }
  };
  const uint32_t steps = (pieces + ROW_STEP - 1) / ROW_STEP;
  for (uint32_t i = 0; i < steps; ++i) {
    Raw raw[ROW_UNROLL];
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) raw[u] = r.load(i * ROW_STEP + u * ROW_THREADS + tid);
    work(raw, i);
  }
  if ((tid & 63) == 0) sh_rank[tid >> 6] = above;
  if (TOP) {
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      const uint32_t g = u * ROW_THREADS + tid;
      keys[g] = g < pieces ? order_key<T>(best[u], (step_of[u] * ROW_STEP + g) * P::N, a.index_bits) : 0;
    }
    if (tid == 0) n_chosen = n_found = 0;
  }
  s = row_partial(s, a.c, sh);  // (with a barrier)
  const bool none = s.max == -INFINITY && s.sum == 0.0f, bad = !(s.sum == s.sum) || s.max == INFINITY;
  const double log_sum = none ? -INFINITY : log(double(s.sum));
  if (tid == 0) {
    const float nan = __uint_as_float(0x7FC00000u);
    float lp = 0.0f;
    int32_t rank = 0;
    if (given) {
      for (uint32_t w = 0; w < ROW_WAVES; ++w) rank += int32_t(sh_rank[w]);
      for (uint32_t j = max(r.lead, id_piece * P::N); j < r.lead + uint32_t(id); ++j) rank += float(r.at[j]) == at_id;
      // (places before the row have been taken for equal ones)
      if (at_id == -INFINITY && id_piece > 0) rank -= int32_t(r.lead);
      rank = bad ? 0 : rank + 1;
      lp = bad ? nan : none ? -INFINITY : float((double(at_id) - s.max) * a.scale - log_sum);
    } else if (id >= 0) {
      lp = nan;
    }
    a.logprobs[row] = lp;
    a.ranks[row] = rank;
    a.entropy[row] = bad ? nan : none ? 0.0f : float(log_sum - double(s.mean) / s.sum * a.scale);
    a.lse[row] = bad ? nan : none ? -INFINITY : float(double(s.max) * a.scale + log_sum);
    a.stats[row] = bad ? make_float2(0.0f, nan) : make_float2(s.max, float(log_sum));
  }
  if (!TOP) return;

  const auto put = [&](uint32_t rank, uint64_t key) {
    const float v = key_value<T>(key, a.index_bits);
    a.top_ids[row * a.k + rank] = int32_t(key_place(key, a.index_bits) - r.lead);
    a.top_logprobs[row * a.k + rank] = none ? -INFINITY : float((double(v) - s.max) * a.scale - log_sum);
  };
  if (bad) {
    for (uint32_t t = tid; t < a.k; t += ROW_THREADS) {
      a.top_ids[row * a.k + t] = -1;
      a.top_logprobs[row * a.k + t] = __uint_as_float(0x7FC00000u);
    }
    return;
  }
  if (tid < 64) {
    const uint64_t bar = kth_key(keys, ROW_STEP, a.k);
    if (tid == 0) reach = bar;
  }
  __syncthreads();
  for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
    const uint32_t g = u * ROW_THREADS + tid;
    if (keys[g] >= reach) chosen[atomicAdd(&n_chosen, 1u)] = uint16_t(g);  // (k at most; their order does not matter)
  }
  __syncthreads();
  // Every element of the chosen groups that is no later in order than the k-th
  // group's largest (as that key has it: by its piece's place) and reaches `low`.
  const uint32_t n_pieces = n_chosen * steps;
  const uint64_t group_bar = reach;
  const auto each = [&](uint64_t low, auto take) {
    for (uint32_t i = tid; i < n_pieces; i += ROW_THREADS) {
      const uint32_t p = (i % steps) * ROW_STEP + chosen[i / steps];
      if (p >= pieces) continue;
      const typename P::val v = values<T>(r.load(p));
#pragma unroll
      for (uint32_t e = 0; e < P::N; ++e) {
        const uint32_t j = p * P::N + e;
        if (j < r.lead || j >= r.end || order_key<T>(v[e], p * P::N, a.index_bits) < group_bar) continue;
        const uint64_t key = order_key<T>(v[e], j, a.index_bits);
        if (key >= low) take(key);
      }
    }
  };
  const auto collect = [&](uint64_t low) {
    each(low, [&](uint64_t key) {
      const uint32_t to = atomicAdd(&n_found, 1u);
      if (to < TOP_ROOM) keys[to] = key;
    });
    __syncthreads();
  };
  collect(0);
  if (n_found > TOP_ROOM) {
    // Large elements crowd in a few groups: halve what is between until a bar
    // leaves k or more, and no more than there is room for.  (Keys differ, so
    // there is one that leaves k.)
    uint64_t lo = 0, hi = ~uint64_t(0) >> 1;
    for (;;) {
      const uint64_t mid = lo + (hi - lo + 1) / 2;
      __syncthreads();  // n_found has been read
      if (tid == 0) n_found = 0;
      __syncthreads();
      each(mid, [&](uint64_t) { atomicAdd(&n_found, 1u); });
      __syncthreads();
      const uint32_t n = n_found;
      if (n < a.k) {
        hi = mid - 1;
      } else {
        lo = mid;
        if (n <= TOP_ROOM) break;
      }
    }
    __syncthreads();
    if (tid == 0) n_found = 0;
    __syncthreads();
    collect(lo);
  }
  const uint32_t n = n_found;
  for (uint32_t i = tid; i < n; i += ROW_THREADS) {
    const uint64_t mine = keys[i];
    uint32_t before = 0;
    for (uint32_t j = 0; j < n; ++j) before += keys[j] > mine;
    if (before < a.k) put(before, mine);
  }
}

struct ScoreBackArgs {
  const void *x;
  int64_t stride;
  void *dx;
  int64_t dx_stride;
  uint64_t block0;
  uint32_t vocab, k, parts, part;  // parts of a row, and pieces of one
  float scale, c;
  const int32_t *ids, *top_ids;
  const float *entropy;
  const float2 *stats;
  const float *g_logprobs, *g_entropy, *g_lse, *g_top;  // null: zeros
};

// One workgroup a part of a row.  Elements that have a term of their own are
// written once more when the part is done, from what was there before (dx may
// be x): each by one thread, or by several with the same value.
template <typename T>
__global__ __launch_bounds__(ROW_THREADS) void k_scores_back(ScoreBackArgs a) {
  typedef Piece<T> P;
  __shared__ int32_t own_id[TOP_MAX + 1];
  __shared__ float own_g[TOP_MAX + 1];
  __shared__ float sh_g[ROW_WAVES];
  const uint32_t tid = threadIdx.x;
  const uint64_t block = a.block0 + blockIdx.x, row = block / a.parts;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  T *dx = static_cast<T *>(a.dx) + int64_t(row) * a.dx_stride;
  const Row<T> r(dx, a.vocab);  // pieces as they are written
  const uint32_t from = uint32_t(block % a.parts) * a.part, to = min(r.pieces(), from + a.part);
  if (from >= to) return;  // (parts are counted for rows that begin anywhere)
  // terms of single elements: the given token's, and the alternatives'
  const uint32_t n = 1 + (a.g_top ? a.k : 0);
  float mine = 0.0f;
  for (uint32_t t = tid; t < n; t += ROW_THREADS) {
    int32_t id = t ? a.top_ids[row * a.k + t - 1] : a.ids[row];
    if (id < 0 || uint32_t(id) >= a.vocab) id = -1;
    const float *g = t ? a.g_top : a.g_logprobs;
    const float v = id < 0 || !g ? 0.0f : t ? g[row * a.k + t - 1] : g[row];
    own_id[t] = id;
    own_g[t] = v;
    mine += v;
  }
  mine = wave_sum(mine);
  if ((tid & 63) == 0) sh_g[tid >> 6] = mine;
  __syncthreads();
  float g = 0.0f;
  for (uint32_t w = 0; w < ROW_WAVES; ++w) g += sh_g[w];
  bool any = false;
  for (uint32_t t = tid; t < n; t += ROW_THREADS) any |= own_g[t] != 0.0f;
  any = __syncthreads_or(any);
  if (a.g_lse) g -= a.g_lse[row];
  const float gh = a.g_entropy ? a.g_entropy[row] : 0.0f;
  const float2 st = a.stats[row];
  // p (g + gh (log p + entropy)) = w (alpha + beta d), d = x - max, w = exp2(c d)
  const bool zero = st.x == -INFINITY || (g == 0.0f && gh == 0.0f && !any);
  const float inv = a.scale * __builtin_amdgcn_exp2f(-st.y * LOG2E);
  const float alpha = -inv * (g + gh * (a.entropy[row] - st.y)), beta = -inv * gh * a.scale;
  const auto of = [&](float v) {
    const float d = fmaxf(v - st.x, LOWEST);
    return __builtin_amdgcn_exp2f(d * a.c) * (alpha + beta * d);
  };
  constexpr uint32_t TERMS = (TOP_MAX + ROW_THREADS) / ROW_THREADS;
  float before[TERMS];
  for (uint32_t i = 0; i < TERMS; ++i) {
    const uint32_t t = tid + i * ROW_THREADS;
    before[i] = t < n && own_id[t] >= 0 && (r.lead + uint32_t(own_id[t])) / P::N - from < to - from ? float(x[own_id[t]]) : 0.0f;
  }
  __syncthreads();
  for (uint32_t p0 = from + tid; p0 < to; p0 += ROW_STEP) {
    typename P::raw raw[ROW_UNROLL];
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u)
      if (p0 + u * ROW_THREADS < to && !zero) raw[u] = r.load(x - r.lead, p0 + u * ROW_THREADS);
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      if (p0 + u * ROW_THREADS >= to) break;
      typename P::val v = 0.0f;
      if (!zero) {
        v = values<T>(raw[u]);
#pragma unroll
        for (uint32_t e = 0; e < P::N; ++e) v[e] = of(v[e]);
      }
      r.store(p0 + u * ROW_THREADS, v);
    }
  }
  __syncthreads();
  if (zero) return;
  for (uint32_t i = 0; i < TERMS; ++i) {
    const uint32_t t = tid + i * ROW_THREADS;
    if (t >= n || own_id[t] < 0 || (r.lead + uint32_t(own_id[t])) / P::N - from >= to - from) continue;
    float sum = 0.0f;
    for (uint32_t j = 0; j < n; ++j) sum += own_id[j] == own_id[t] ? own_g[j] : 0.0f;
    dx[own_id[t]] = T(of(before[i]) + a.scale * sum);
  }
}

uint32_t bits_of(uint32_t vocab) {
  uint32_t b = 1;
  while (b < 31 && (1u << b) < vocab) ++b;
  return b;
}

constexpr uint64_t MAX_GROUPS = 1u << 23;  // workgroups of a launch: fewer than 2^32 threads

}  // namespace
}  // namespace bbpe

using namespace bbpe;

extern "C" {

int bbpe_token_logprobs(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                        const int32_t *d_ids, uint32_t top_k, float scale, float *d_logprobs, float *d_entropy,
                        float *d_lse, int32_t *d_ranks, int32_t *d_top_ids, float *d_top_logprobs, float *d_stats,
                        void *hip_stream) {
  if (bad_logits(dtype, logits, row_stride, n_rows, vocab, false) || top_k > TOP_MAX || top_k > vocab || !(scale > 0.0f) ||
      !std::isfinite(scale))
    return BBPE_E_INVALID_ARG;
  if (n_rows && (!d_ids || !d_logprobs || !d_entropy || !d_lse || !d_ranks || !d_stats ||
                 (top_k && (!d_top_ids || !d_top_logprobs))))
    return BBPE_E_INVALID_ARG;
  if ((address(d_ids) | address(d_logprobs) | address(d_entropy) | address(d_lse) | address(d_ranks) | address(d_top_ids) |
       address(d_top_logprobs)) & 3 || (address(d_stats) & 7))
    return BBPE_E_INVALID_ARG;
  if (n_rows == 0) return BBPE_OK;
  ScoreArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.vocab = vocab;
  a.k = top_k;
  a.scale = scale;
  a.c = scale * LOG2E;
  a.index_bits = bits_of(vocab + 8);  // places begin up to 7 before the row
  a.ids = d_ids;
  a.logprobs = d_logprobs;
  a.entropy = d_entropy;
  a.lse = d_lse;
  a.ranks = d_ranks;
  a.top_ids = d_top_ids;
  a.top_logprobs = d_top_logprobs;
  a.stats = reinterpret_cast<float2 *>(d_stats);
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  for (; a.row0 < n_rows; a.row0 += MAX_GROUPS)
    with_element(dtype, [&](auto t) {
      const uint32_t grid = uint32_t(std::min(n_rows - a.row0, MAX_GROUPS));
      if (top_k) k_scores<decltype(t), true><<<grid, ROW_THREADS, 0, st>>>(a);
      else k_scores<decltype(t), false><<<grid, ROW_THREADS, 0, st>>>(a);
    });
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

int bbpe_token_logprobs_backward(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                                 const int32_t *d_ids, uint32_t top_k, float scale, const float *d_entropy,
                                 const int32_t *d_top_ids, const float *d_stats, const float *g_logprobs,
                                 const float *g_entropy, const float *g_lse, const float *g_top, void *d_logits,
                                 int64_t dl_stride, void *hip_stream) {
  if (bad_logits(dtype, logits, row_stride, n_rows, vocab, false) || bad_logits(dtype, d_logits, dl_stride, n_rows, vocab, true) ||
      top_k > TOP_MAX || top_k > vocab || !(scale > 0.0f) || !std::isfinite(scale))
    return BBPE_E_INVALID_ARG;
  if (n_rows && (!d_ids || !d_entropy || !d_stats || (g_top && top_k && !d_top_ids))) return BBPE_E_INVALID_ARG;
  if ((address(d_ids) | address(d_entropy) | address(d_top_ids) | address(g_logprobs) | address(g_entropy) | address(g_lse) |
       address(g_top)) & 3 || (address(d_stats) & 7))
    return BBPE_E_INVALID_ARG;
  if (n_rows == 0) return BBPE_OK;
  ScoreBackArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.dx = d_logits;
  a.dx_stride = dl_stride;
  a.vocab = vocab;
  a.k = top_k;
  a.scale = scale;
  a.c = scale * LOG2E;
  a.ids = d_ids;
  a.top_ids = d_top_ids;
  a.entropy = d_entropy;
  a.stats = reinterpret_cast<const float2 *>(d_stats);
  a.g_logprobs = g_logprobs;
  a.g_entropy = g_entropy;
  a.g_lse = g_lse;
  a.g_top = top_k ? g_top : nullptr;
  a.part = 2 * ROW_STEP;
  a.parts = (most_pieces(dtype, vocab) + a.part - 1) / a.part;
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const uint64_t blocks = n_rows * a.parts;
  for (; a.block0 < blocks; a.block0 += MAX_GROUPS)
    with_element(dtype, [&](auto t) {
      k_scores_back<decltype(t)><<<uint32_t(std::min(blocks - a.block0, MAX_GROUPS)), ROW_THREADS, 0, st>>>(a);
    });
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

}  // extern "C"
