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

constexpr uint32_t TOP_MAX = 256;   // alternatives at most
// What a bar may let through besides the first k: the halving ends some steps
// earlier for it (4,096 rows of 200,064, 64 alternatives: 324 us, without 333).
__host__ __device__ constexpr uint32_t with_slack(uint32_t k) { return k + k / 4 + 16; }
constexpr uint32_t TOP_ROOM = with_slack(TOP_MAX);
// Alternatives up to which a wave may take a row: of a wave's 256 groups, 96 reach
// the bar at most, and 5.3 KB of LDS let 28 waves (all that its registers do) onto a CU.
constexpr uint32_t SMALL_TOP = 64;
constexpr uint32_t KEPT_ROOM = (TOP_ROOM + 63) / 64 * 64;
constexpr uint32_t JOIN_KEYS = 4096;  // alternatives of all parts at most: 32 KB of LDS in the kernel that joins them

struct ScorePart {
  Partial p;
  uint32_t above;
};

struct ScoreArgs {
  const void *x;
  int64_t stride;
  uint64_t block0;
  uint32_t vocab, k, parts, part;  // parts of a row, and pieces of one
  float scale;
  Exponent x2;
  uint32_t index_bits;  // of a place in the row
  const int32_t *ids;
  float *logprobs, *entropy, *lse;
  int32_t *ranks;
  int32_t *top_ids;
  float *top_logprobs;
  float2 *stats;
  ScorePart *parted;     // [rows][parts]
  uint64_t *parted_top;  // [rows][parts][k], 0 where a part has fewer
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

// A number that k of the keys reach, and no more than `most`, by one wave; 1 if
// there are no more than k.  get(i): the lane's i-th of N, or of n where N is 0.
// Keys differ from each other, but for absent ones, which are 0.
template <uint32_t N, typename G>
__device__ __forceinline__ uint64_t top_bar(G get, uint32_t n, uint32_t k, uint32_t most) {
  const auto each = [&](auto f) {
    if constexpr (N > 0) {
#pragma unroll
      for (uint32_t i = 0; i < N; ++i) f(get(i));
    } else {
      for (uint32_t i = 0; i < n; ++i) f(get(i));
    }
  };
  uint64_t lo = ~uint64_t(0), hi = 0;
  uint32_t there = 0;
  each([&](uint64_t v) {
    there += uint32_t(__popcll(__ballot(v != 0)));
    if (v > hi) hi = v;
    if (v && v < lo) lo = v;
  });
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
    each([&](uint64_t v) { reach += uint32_t(__popcll(__ballot(v >= mid))); });
    if (reach < k) {
      hi = mid - 1;
    } else {
      if (reach <= most) return mid;
      lo = mid;
    }
  }
  return lo;
}

// Puts n different keys in order, the first k of them: put(place, key).  keys: in
// LDS, with room for as many (in sixty-fours) from `half` on.  Sixty-four at a
// time are ranked by counting and laid there in order; a key's place among the
// others is found by halving, in several sixty-fours at once.
template <uint32_t WAVES, typename F>
__device__ __forceinline__ void put_in_order(uint64_t *keys, uint32_t half, uint32_t n, uint32_t k, F put) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, blocks = (n + 63) / 64;
  for (uint32_t b = wave; b < blocks; b += WAVES) {
    const uint64_t *own = keys + b * 64;
    const uint32_t there = min(64u, n - b * 64);
    const uint64_t mine = lane < there ? own[lane] : 0;
    uint32_t place = 0;
#pragma unroll 8
    for (uint32_t j = 0; j < there; ++j) place += own[j] > mine;
    keys[half + b * 64 + (lane < there ? place : lane)] = mine;
  }
  __syncthreads();
  for (uint32_t b = wave; b < blocks; b += WAVES) {
    const uint64_t mine = keys[half + b * 64 + lane];
    uint32_t at = lane;
#pragma unroll 4
    for (uint32_t o = 0; o < blocks; ++o) {
      const uint64_t *others = keys + half + o * 64;
      uint32_t before = 0;
#pragma unroll
      for (uint32_t step = 32; step; step /= 2) before += others[before + step - 1] > mine ? step : 0;
      before += others[before] > mine;
      at += o == b ? 0 : before;
    }
    if (b * 64 + lane < n && at < k) put(at, mine);
  }
}

// The largest number below v in the order of floats; below minus infinity: NaN.
__device__ __forceinline__ float next_below(float v) {
  const uint32_t b = __float_as_uint(v);
  if (v == -INFINITY) return __uint_as_float(0x7FC00000u);
  if (v == 0.0f) return __uint_as_float(0x80000001u);
  return __uint_as_float(v > 0.0f ? b - 1 : b + 1);
}

// What a row's weights come to.
struct RowEnd {
  Partial p;
  bool none, bad;  // nothing but minus infinity; a NaN or plus infinity
  double log_sum;

  __device__ __forceinline__ explicit RowEnd(Partial s) : p(s) {
    none = s.max == -INFINITY && s.sum == 0.0;
    bad = !(s.sum == s.sum) || s.max == INFINITY;
    log_sum = none ? -INFINITY : log(s.sum);
  }
  __device__ __forceinline__ float logprob(float v, float scale) const {
    return bad ? __uint_as_float(0x7FC00000u) : none ? -INFINITY : float((double(v) - p.max) * scale - log_sum);
  }
};

// The row's given token.
template <typename T> struct Given {
  bool there;
  float value;      // infinity where there is none: nothing is above it
  uint32_t place;
  __device__ __forceinline__ Given(const ScoreArgs &a, const Row<const T> &r, int32_t id) {
    there = id >= 0 && uint32_t(id) < a.vocab;
    place = r.lead + (there ? uint32_t(id) : 0);
    value = there ? float(r.at[place]) : INFINITY;
  }
  __device__ __forceinline__ uint32_t piece() const { return place / Piece<T>::N; }
  // Elements before it in its piece that are equal to it.  Places before the row
  // count as minus infinity in all pieces before its own, and are taken off.
  __device__ __forceinline__ int32_t equal_before(const Row<const T> &r) const {
    constexpr uint32_t N = Piece<T>::N;
    const typename Piece<T>::val v = values<T>(r.load(piece()));
    int32_t n = value == -INFINITY && piece() > 0 ? -int32_t(r.lead) : 0;
#pragma unroll
    for (uint32_t e = 0; e < N; ++e) n += piece() * N + e >= r.lead && piece() * N + e < place && v[e] == value;
    return n;
  }
};

// The row's numbers, by one thread.  above: elements before the given one in order.
template <typename T>
__device__ __forceinline__ void write_row(const ScoreArgs &a, uint64_t row, const RowEnd &end, int32_t id, const Given<T> &given, int32_t above) {
  const float nan = __uint_as_float(0x7FC00000u);
  const double inv = 1.0 / end.p.sum;
  a.logprobs[row] = given.there ? end.logprob(given.value, a.scale) : id < 0 ? 0.0f : nan;
  a.ranks[row] = given.there && !end.bad ? above + 1 : 0;
  a.entropy[row] = end.bad ? nan : end.none ? 0.0f : float(end.log_sum - double(end.p.mean) * inv * a.scale);
  a.lse[row] = end.bad ? nan : end.none ? -INFINITY : float(double(end.p.max) * a.scale + end.log_sum);
  a.stats[row] = end.bad ? make_float2(0.0f, nan) : make_float2(end.p.max, float(inv));
}
template <typename T>
__device__ __forceinline__ void write_top(const ScoreArgs &a, uint64_t row, uint32_t lead, const RowEnd &end, uint32_t t, uint64_t key) {
  a.top_ids[row * a.k + t] = end.bad ? -1 : int32_t(key_place(key, a.index_bits) - lead);
  a.top_logprobs[row * a.k + t] = end.logprob(key_value<T>(key, a.index_bits), a.scale);
}

// KEEP: pieces of a group whose places a thread keeps; 0 without alternatives.
template <uint32_t WAVES, uint32_t KEEP> struct ScoreShared {
  static constexpr bool TOP = KEEP > 0;
  static constexpr uint32_t GROUPS = 64 * WAVES * ROW_UNROLL;
  // Candidates that can be put in order; twice as many can be held.  Where no more
  // than k groups have pieces, all of their elements are.
  static constexpr uint32_t LIST = with_slack(KEEP < 2 ? SMALL_TOP : TOP_MAX);  // groups that reach the bar
  static constexpr uint32_t ROOM = GROUPS;
  static_assert(ROOM >= LIST && 2 * ROOM >= 8 * (WAVES == 1 ? SMALL_TOP : TOP_MAX), "");
  Partial sums[WAVES];
  uint32_t above[WAVES];
  uint64_t keys[TOP ? 2 * ROOM : 1];
  uint32_t chosen[TOP ? KEEP * LIST : 1];  // pieces
  uint32_t deep[TOP ? LIST : 1][TOP ? 1 + KEEP : 1];  // a group, and its pieces among the chosen ones
  uint32_t n_chosen, n_deep, n_found;
  uint64_t reach;
};

// Pieces [first, last) of a row by a workgroup: the whole row, or a part of it
// (`part`: where its numbers go).
//
// Alternatives.  A thread's step takes ROW_UNROLL pieces; the pieces at one
// place of all steps are a group, of which the thread keeps the largest element,
// the first piece that has it, and the largest element of all other pieces.  A
// bar that the largest of k groups or more reach keeps the first k elements: one
// below it has k before it.  Of the groups that reach it the pieces with the
// largest are read once more, and the others only where their largest reaches it
// too: seldom, of 1,024 groups, for 20 alternatives, but of one group in six for
// 256.  Workgroups (KEEP 2) keep the second piece's place and the largest of the
// third too (4,096 rows of 200,064, 256 alternatives: 437 -> 372 us, 20: the same;
// a wave by itself, whose rows have few steps, does not).  What reaches the bar are
// the candidates, not many more than k.
template <typename T, uint32_t WAVES, uint32_t KEEP, bool WHOLE>
__device__ __forceinline__ void score_pieces(const ScoreArgs &a, uint64_t row, uint32_t first, uint32_t last, uint64_t part,
                                             ScoreShared<WAVES, KEEP> &sh) {
  typedef Piece<T> P;
  constexpr bool TOP = KEEP > 0;
  constexpr uint32_t THREADS = 64 * WAVES, STEP = THREADS * ROW_UNROLL, ROOM = ScoreShared<WAVES, KEEP>::ROOM;
  const Row<const T> r(static_cast<const T *>(a.x) + int64_t(row) * a.stride, a.vocab);
  const uint32_t tid = threadIdx.x;
  last = min(last, r.pieces());
  const int32_t id = a.ids[row];
  const Given<T> given(a, r, id);
  const uint32_t before_id = given.there ? min(last, given.piece()) : 0;  // pieces, where equal ones count too
  const float at_least = given.there ? next_below(given.value) : INFINITY;
  const int32_t beside = WHOLE && given.there ? given.equal_before(r) : 0;

  Partial s{0.0, -INFINITY, 0.0f};
  float ref = 0.0f;
  uint32_t above = 0;  // the wave's
  float best[ROW_UNROLL], second[ROW_UNROLL], third[ROW_UNROLL];
  uint32_t best_at[ROW_UNROLL], second_at[ROW_UNROLL];  // the piece's step
#pragma unroll
  for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
    best[u] = second[u] = third[u] = -INFINITY;
    best_at[u] = second_at[u] = ~0u;  // none
  }
  for (uint32_t p0 = first; p0 < last; p0 += STEP) {
    typename P::raw raw[ROW_UNROLL];
    r.template load_step<THREADS>(raw, r.at, p0 + tid, last);
    typename P::val v[ROW_UNROLL];
    float m = -INFINITY;
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      v[u] = values<T>(raw[u]);
      float pm = v[u][0];
#pragma unroll
      for (uint32_t e = 1; e < P::N; ++e) pm = fmaxf(pm, v[u][e]);
      if (TOP) {
        const bool more = pm > best[u];
        if (KEEP > 1) {
          // (a piece of nothing but minus infinity is no second one; third covers it)
          third[u] = __builtin_amdgcn_fmed3f(third[u], second[u], pm);
          second_at[u] = more ? best_at[u] : pm > second[u] ? p0 : second_at[u];
        }
        second[u] = __builtin_amdgcn_fmed3f(second[u], best[u], pm);  // (they are in order)
        best[u] = more ? pm : best[u];
        best_at[u] = more ? p0 : best_at[u];
      }
      m = fmaxf(m, pm);
    }
    if (m > s.max) {
      const float d = s.max - m;
      s = s.max == -INFINITY ? Partial{s.sum, m, 0.0f} : scaled(s, m, d, fine_weight(d, Exponent{a.x2.c, 0.0f}));
      ref = m;
    }
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      const float bar = p0 + u * THREADS + tid < before_id ? at_least : given.value;
#pragma unroll
      for (uint32_t e = 0; e < P::N; ++e) {
        const float d = v[u][e] - ref, w = __builtin_amdgcn_exp2f(d * a.x2.c);
        s.mean += w * fmaxf(d, LOWEST);  // (0 times minus infinity is to be 0)
        above += uint32_t(__popcll(__ballot(!(v[u][e] <= bar))));
        v[u][e] = w;
      }
      s.sum += double(piece_sum<P::N>(v[u]));
    }
  }
  // (the exponent's second part, to first order: each weight times LN2 * low * (x - max))
  s.sum += LN2 * double(a.x2.low) * double(s.mean);
  if ((tid & 63) == 0) sh.above[tid >> 6] = above;
  const RowEnd end(row_partial<WAVES>(s, a.x2, sh.sums));  // (with a barrier)
  if (tid == THREADS - 1) {  // (the first wave has the bar to find)
    above = 0;
    for (uint32_t w = 0; w < WAVES; ++w) above += sh.above[w];
    if (WHOLE) write_row<T>(a, row, end, id, given, int32_t(above) + beside);
    else a.parted[part] = ScorePart{end.p, above};
  }
  if (!TOP) return;

  const auto put = [&](uint32_t t, uint64_t key) {
    if (WHOLE) write_top<T>(a, row, r.lead, end, t, key);
    else a.parted_top[part * a.k + t] = key;
  };
  if (end.bad) {
    for (uint32_t t = tid; t < a.k; t += THREADS) put(t, 0);
    return;
  }
  // Every element of the chosen groups that reaches the bar (by its piece's place,
  // as groups do) and `low`.
  const uint32_t deep_steps = (last - first + STEP - 1) / STEP;
  uint32_t n_pieces, n_deep_pieces;
  uint64_t group_bar;
  const auto each = [&](uint64_t low, auto take) {
    for (uint32_t i = tid; i < (n_pieces + n_deep_pieces) * P::N; i += THREADS) {  // an element a thread
      uint32_t p = i / P::N;
      if (p < n_pieces) {
        p = sh.chosen[p];
      } else {
        p -= n_pieces;
        const uint32_t *of = sh.deep[p / deep_steps];
        p = first + p % deep_steps * STEP + of[0];
        if (p >= last || p == of[1] || (KEEP > 1 && p == of[2])) continue;
      }
      const uint32_t j = p * P::N + i % P::N;
      if (j < r.lead || j >= r.end) continue;
      const float v = float(r.at[j]);
      if (order_key<T>(v, p * P::N, a.index_bits) < group_bar) continue;
      const uint64_t key = order_key<T>(v, j, a.index_bits);
      if (key >= low) take(key);
    }
  };
  const auto collect = [&](uint64_t low) {
    each(low, [&](uint64_t key) {
      const uint32_t to = atomicAdd(&sh.n_found, 1u);
      if (to < 2 * ROOM) sh.keys[to] = key;
    });
    __syncthreads();
  };
  for (uint32_t most = with_slack(a.k);; most = a.k) {
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      const uint32_t g = u * THREADS + tid;
      if (best_at[u] == ~0u) best_at[u] = first;  // nothing but minus infinity
      // (keys made ahead of the loop take 18 registers: 4 waves a SIMD, not 5, and 4% of the time)
      asm("" : "+v"(best[u]), "+v"(second[u]), "+v"(third[u]));
      sh.keys[g] = first + g < last ? order_key<T>(best[u], (best_at[u] + g) * P::N, a.index_bits) : 0;
    }
    if (tid == 0) sh.n_chosen = sh.n_deep = sh.n_found = 0;
    __syncthreads();
    if (tid < 64) {
      uint64_t mine[STEP / 64];
#pragma unroll
      for (uint32_t i = 0; i < STEP / 64; ++i) mine[i] = sh.keys[i * 64 + tid];
      const uint64_t bar = top_bar<STEP / 64>([&](uint32_t i) { return mine[i]; }, 0, a.k, most);
      if (tid == 0) sh.reach = bar;
    }
    __syncthreads();
    group_bar = sh.reach;
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      const uint32_t g = u * THREADS + tid;
      if (sh.keys[g] < group_bar) continue;
      // (their order does not matter)
      sh.chosen[atomicAdd(&sh.n_chosen, 1u)] = best_at[u] + g;
      float rest = second[u];
      if (KEEP > 1) {
        const bool two = second_at[u] != ~0u && order_key<T>(rest, (second_at[u] + g) * P::N, a.index_bits) >= group_bar;
        if (two) {
          sh.chosen[atomicAdd(&sh.n_chosen, 1u)] = second_at[u] + g;
          rest = third[u];
        } else {
          second_at[u] = ~0u;
        }
      }
      // the others' key is no larger than that of their largest at the first of them
      uint32_t other = first;
      if (other == best_at[u]) other += STEP;
      if (KEEP > 1 && other == second_at[u]) other += other + STEP == best_at[u] ? 2 * STEP : STEP;
      if (other + g < last && order_key<T>(rest, (other + g) * P::N, a.index_bits) >= group_bar) {
        uint32_t *to = sh.deep[atomicAdd(&sh.n_deep, 1u)];
        to[0] = g;
        to[1] = best_at[u] + g;
        if (KEEP > 1) to[2] = second_at[u] == ~0u ? ~0u : second_at[u] + g;
      }
    }
    __syncthreads();
    n_pieces = sh.n_chosen;
    n_deep_pieces = sh.n_deep * deep_steps;
    collect(0);
    // Among equal elements a bar lets through whole pieces: with the smallest bar
    // that is 8 k elements, with some slack it may be more than there is room for.
    if (sh.n_found <= 2 * ROOM || most == a.k) break;
    __syncthreads();  // the lists have been read
  }
  if (sh.n_found > 2 * ROOM) {
    // Large elements crowd in a few groups: halve what is between until a bar
    // leaves k or more, and no more than there is room for.  (Keys differ, so
    // there is one that leaves k.)
    uint64_t lo = 0, hi = ~uint64_t(0) >> 1;
    for (;;) {
      const uint64_t mid = lo + (hi - lo + 1) / 2;
      __syncthreads();  // n_found has been read
      if (tid == 0) sh.n_found = 0;
      __syncthreads();
      each(mid, [&](uint64_t) { atomicAdd(&sh.n_found, 1u); });
      __syncthreads();
      const uint32_t n = sh.n_found;
      if (n < a.k) {
        hi = mid - 1;
      } else {
        lo = mid;
        if (n <= 2 * ROOM) break;
      }
    }
    __syncthreads();
    if (tid == 0) sh.n_found = 0;
    __syncthreads();
    collect(lo);
  }
  uint32_t n = sh.n_found;
  __syncthreads();  // n_found has been read
  if (n > ROOM) {
    // more than can be put in order: those that reach a bar among them, moved to the front
    if (tid < 64) {
      const uint64_t bar = top_bar<0>([&](uint32_t i) { return i * 64 + tid < n ? sh.keys[i * 64 + tid] : 0; }, (n + 63) / 64, a.k, with_slack(a.k));
      if (tid == 0) {
        sh.reach = bar;
        sh.n_found = 0;
      }
    }
    __syncthreads();
    for (uint32_t i = 0; i < n; i += THREADS) {
      const uint64_t mine = i + tid < n ? sh.keys[i + tid] : 0;
      __syncthreads();  // (no more are moved than have been read)
      if (mine >= sh.reach) sh.keys[atomicAdd(&sh.n_found, 1u)] = mine;
    }
    __syncthreads();
    n = sh.n_found;
  }
  put_in_order<WAVES>(sh.keys, ROOM, n, a.k, put);
  if (!WHOLE)
    for (uint32_t t = n + tid; t < a.k; t += THREADS) put(t, 0);  // a part of fewer elements
}

// A workgroup a row or, SPLIT, a part of one.
//
// Bound by the one read of the row: bfloat16, 8,192 rows of 100,277 in 290 us, 5.65
// TB/s where a sum of as many bytes by itself reaches 3.9 and a copy's two ways 5.0;
// 4,096 of 200,064 with 20 alternatives 319 us (5.1), float32 580 without and 612
// with.  Entropy, rank and the sum in 64 bits fit under the loads: leaving them out
// changes nothing.  A thread has four loads of 16 bytes in flight and a CU 32 waves
// (20 with alternatives, for the groups' registers; forced to 24 they spill, 368 us).
// Aligned pieces, whatever element a row begins at: 346 -> 296 us for 100,277.
// Workgroups that stay and take equal runs over all rows were slower (308 us), and
// so with alternatives (350).
template <typename T, uint32_t WAVES, uint32_t KEEP, bool SPLIT>
__global__ __launch_bounds__(64 * WAVES) void k_scores(ScoreArgs a) {
  __shared__ ScoreShared<WAVES, KEEP> sh;
  const uint64_t block = a.block0 + blockIdx.x, row = SPLIT ? block / a.parts : block;
  const uint32_t first = SPLIT ? uint32_t(block % a.parts) * a.part : 0;
  score_pieces<T, WAVES, KEEP, !SPLIT>(a, row, first, SPLIT ? first + a.part : ~0u, block, sh);
}

// Joins a row's parts.  Bound by its launch and a chain of barriers: 5 us, 7 for 20
// alternatives of each of 128 rows.
template <typename T, bool TOP>
__global__ __launch_bounds__(TOP ? ROW_THREADS : 64) void k_scores_join(ScoreArgs a) {
  __shared__ uint64_t keys[TOP ? JOIN_KEYS : 1];
  __shared__ uint64_t kept[TOP ? 2 * KEPT_ROOM : 1];
  __shared__ uint32_t n_kept;
  __shared__ uint64_t reach;
  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint64_t row = a.block0 + blockIdx.x;
  const Row<const T> r(static_cast<const T *>(a.x) + int64_t(row) * a.stride, a.vocab);
  ScorePart part{Partial{0.0, -INFINITY, 0.0f}, 0};
  if (lane < a.parts) part = a.parted[row * a.parts + lane];
  const RowEnd end(wave_partial(part.p, a.x2));
  const uint32_t above = wave_sum(part.above);
  const int32_t id = a.ids[row];
  const Given<T> given(a, r, id);
  if (tid == (TOP ? ROW_THREADS : 64) - 1)
    write_row<T>(a, row, end, id, given, int32_t(above) + (given.there ? given.equal_before(r) : 0));
  if (!TOP) return;
  const uint32_t n = a.parts * a.k;
  for (uint32_t i = tid; i < n; i += ROW_THREADS) keys[i] = a.parted_top[row * n + i];
  if (tid == 0) n_kept = 0;
  __syncthreads();
  if (end.bad) {
    for (uint32_t t = tid; t < a.k; t += ROW_THREADS) write_top<T>(a, row, r.lead, end, t, 0);
    return;
  }
  if (tid < 64) {
    const uint64_t bar = top_bar<0>([&](uint32_t i) { return i * 64 + lane < n ? keys[i * 64 + lane] : 0; }, (n + 63) / 64, a.k, with_slack(a.k));
    if (tid == 0) reach = bar;
  }
  __syncthreads();
  for (uint32_t i = tid; i < n; i += ROW_THREADS)
    if (keys[i] >= reach) kept[atomicAdd(&n_kept, 1u)] = keys[i];
  __syncthreads();
  put_in_order<ROW_WAVES>(kept, KEPT_ROOM, n_kept, a.k, [&](uint32_t t, uint64_t key) { write_top<T>(a, row, r.lead, end, t, key); });
}

struct ScoreBackArgs {
  const void *x;
  int64_t stride;
  void *dx;
  int64_t dx_stride;
  uint64_t block0;
  uint32_t vocab, k, parts, part;  // parts of a row, and pieces of one
  float scale;
  Exponent x2;
  const int32_t *ids, *top_ids;
  const float *entropy;
  const float2 *stats;
  const float *g_logprobs, *g_entropy, *g_lse, *g_top;  // null: zeros
};

// One workgroup a part of a row: two steps, so that rows of any length are many
// workgroups (4,096 rows of 100,277 in bfloat16: 288 us, 5.7 TB/s of what is read
// and written); a wave a row of up to 512 pieces (65,536 of 1,280: 148 -> 76 us; 512
// rows of 8,192 7.4 us, by a wave each 11.4).  Elements that have a term of their own are
// written once more when the part is done, from what was there before (dx may
// be x): each by one thread, or by several with the same value.
template <typename T, uint32_t WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_scores_back(ScoreBackArgs a) {
  constexpr uint32_t THREADS = 64 * WAVES, STEP = THREADS * ROW_UNROLL;
  typedef Piece<T> P;
  __shared__ int32_t own_id[TOP_MAX + 1];
  __shared__ float own_g[TOP_MAX + 1];
  __shared__ float sh_g[WAVES];
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
  for (uint32_t t = tid; t < n; t += THREADS) {
    int32_t id = t ? a.top_ids[row * a.k + t - 1] : a.ids[row];
    if (id < 0 || uint32_t(id) >= a.vocab) id = -1;
    // (alternatives count without their ids too: a row without probabilities names none, but what it returned depends
    // on its logits, and its gradient is NaN)
    const float v = t ? a.g_top[row * a.k + t - 1] : id < 0 || !a.g_logprobs ? 0.0f : a.g_logprobs[row];
    own_id[t] = id;
    own_g[t] = v;
    mine += v;
  }
  mine = wave_sum(mine);
  if ((tid & 63) == 0) sh_g[tid >> 6] = mine;
  __syncthreads();
  float g = 0.0f;
  for (uint32_t w = 0; w < WAVES; ++w) g += sh_g[w];
  bool any = false;
  for (uint32_t t = tid; t < n; t += THREADS) any |= own_g[t] != 0.0f;
  any = __syncthreads_or(any);
  if (a.g_lse) g -= a.g_lse[row];
  const float gh = a.g_entropy ? a.g_entropy[row] : 0.0f;
  const float2 st = a.stats[row];
  // p (g + gh (log p + entropy)) = w (alpha + beta t), t = scale log2(e) (x - max), w = exp2(t);
  // t is bounded where w is 0, so that their product is 0
  const bool zero = st.x == -INFINITY || (g == 0.0f && gh == 0.0f && !any);
  const float inv = a.scale * st.y;
  const float alpha = -inv * (g + gh * (a.entropy[row] + logf(st.y))), beta = -inv * gh * float(LN2);
  const auto of = [&](float v) {
    const float d = v - st.x, t = fmaxf(__builtin_fmaf(d, a.x2.low, d * a.x2.c), -16384.0f);
    return __builtin_amdgcn_exp2f(t) * (alpha + beta * t);
  };
  constexpr uint32_t TERMS = (TOP_MAX + THREADS) / THREADS;
  float before[TERMS];
  for (uint32_t i = 0; i < TERMS; ++i) {
    const uint32_t t = tid + i * THREADS;
    before[i] = t < n && own_id[t] >= 0 && (r.lead + uint32_t(own_id[t])) / P::N - from < to - from ? float(x[own_id[t]]) : 0.0f;
  }
  __syncthreads();
  for (uint32_t p0 = from; p0 < to; p0 += STEP) {
    typename P::raw raw[ROW_UNROLL];
    if (!zero) r.template load_step<THREADS>(raw, x - r.lead, p0 + tid, to);
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      const uint32_t p = p0 + u * THREADS + tid;
      if (p >= to) break;
      typename P::val v = 0.0f;
      if (!zero) {
        v = values<T>(raw[u]);
#pragma unroll
        for (uint32_t e = 0; e < P::N; ++e) v[e] = of(v[e]);
      }
      r.store(p, v);
    }
  }
  __syncthreads();
  if (zero) return;
  for (uint32_t i = 0; i < TERMS; ++i) {
    const uint32_t t = tid + i * THREADS;
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

struct ScoreCut : Cut {
  uint64_t parted_bytes, bytes;  // of the parts' numbers, and with their alternatives
};
ScoreCut cut_of(int dtype, uint64_t n_rows, uint32_t vocab, uint32_t k) {
  ScoreCut c{cut_rows(dtype, n_rows, vocab, k <= SMALL_TOP, k ? JOIN_KEYS / k : PARTS_MAX), 0, 0};
  if (c.parts > 1) {
    c.parted_bytes = (n_rows * c.parts * sizeof(ScorePart) + 255) / 256 * 256;
    c.bytes = c.parted_bytes + n_rows * c.parts * k * sizeof(uint64_t);
  }
  return c;
}

int check_scores(int dtype, const void *logits, int64_t stride, uint64_t n_rows, uint32_t vocab, uint32_t k, float scale) {
  return bad_logits(dtype, logits, stride, n_rows, vocab, false) || k > TOP_MAX || k > vocab || bad_scale(scale)
             ? BBPE_E_INVALID_ARG
             : BBPE_OK;
}

}  // namespace
}  // namespace bbpe

using namespace bbpe;

extern "C" {

int bbpe_token_logprobs_workspace_bytes(int dtype, uint64_t n_rows, uint32_t vocab, uint32_t top_k, uint64_t *out_bytes) {
  if (!out_bytes || bad_sizes(dtype, n_rows, vocab) || top_k > TOP_MAX || top_k > vocab) return BBPE_E_INVALID_ARG;
  *out_bytes = cut_of(dtype, n_rows, vocab, top_k).bytes;
  return BBPE_OK;
}

int bbpe_token_logprobs(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                        const int32_t *d_ids, uint32_t top_k, float scale, float *d_logprobs, float *d_entropy,
                        float *d_lse, int32_t *d_ranks, int32_t *d_top_ids, float *d_top_logprobs, float *d_stats,
                        void *d_workspace, uint64_t workspace_bytes, void *hip_stream) {
  const int rc = check_scores(dtype, logits, row_stride, n_rows, vocab, top_k, scale);
  if (rc) return rc;
  if (n_rows && (!d_ids || !d_logprobs || !d_entropy || !d_lse || !d_ranks || !d_stats ||
                 (top_k && (!d_top_ids || !d_top_logprobs))))
    return BBPE_E_INVALID_ARG;
  if ((address(d_ids) | address(d_logprobs) | address(d_entropy) | address(d_lse) | address(d_ranks) | address(d_top_ids) |
       address(d_top_logprobs)) & 3 || (address(d_stats) & 7))
    return BBPE_E_INVALID_ARG;
  if (n_rows == 0) return BBPE_OK;
  const ScoreCut cut = cut_of(dtype, n_rows, vocab, top_k);
  if (cut.bytes && (!d_workspace || (address(d_workspace) & 255) || workspace_bytes < cut.bytes)) return BBPE_E_WORKSPACE;
  ScoreArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.vocab = vocab;
  a.k = top_k;
  a.parts = cut.parts;
  a.part = cut.part;
  a.scale = scale;
  a.x2 = exponent_of(scale);
  a.index_bits = bits_of(vocab + 8);  // places begin up to 7 before the row
  a.ids = d_ids;
  a.logprobs = d_logprobs;
  a.entropy = d_entropy;
  a.lse = d_lse;
  a.ranks = d_ranks;
  a.top_ids = d_top_ids;
  a.top_logprobs = d_top_logprobs;
  a.stats = reinterpret_cast<float2 *>(d_stats);
  a.parted = static_cast<ScorePart *>(d_workspace);
  a.parted_top = reinterpret_cast<uint64_t *>(static_cast<char *>(d_workspace) + cut.parted_bytes);
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const auto launch = [&](uint64_t blocks, auto kernel, uint32_t threads) {
    for (a.block0 = 0; a.block0 < blocks; a.block0 += MAX_GROUPS)
      kernel<<<uint32_t(std::min(blocks - a.block0, MAX_GROUPS)), threads, 0, st>>>(a);
  };
  with_element(dtype, [&](auto t) {
    typedef decltype(t) T;
    constexpr uint32_t W = ROW_WAVES;
    if (cut.parts > 1) {
      launch(n_rows * cut.parts, top_k ? k_scores<T, W, 2, true> : k_scores<T, W, 0, true>, ROW_THREADS);
      launch(n_rows, top_k ? k_scores_join<T, true> : k_scores_join<T, false>, top_k ? ROW_THREADS : 64);
    } else if (cut.waves > 1) {
      launch(n_rows, top_k ? k_scores<T, W, 2, false> : k_scores<T, W, 0, false>, ROW_THREADS);
    } else {
      launch(n_rows, top_k ? k_scores<T, 1, 1, false> : k_scores<T, 1, 0, false>, 64);
    }
  });
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

int bbpe_token_logprobs_backward(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                                 const int32_t *d_ids, uint32_t top_k, float scale, const float *d_entropy,
                                 const int32_t *d_top_ids, const float *d_stats, const float *g_logprobs,
                                 const float *g_entropy, const float *g_lse, const float *g_top, void *d_logits,
                                 int64_t dl_stride, void *hip_stream) {
  const int rc = check_scores(dtype, logits, row_stride, n_rows, vocab, top_k, scale);
  if (rc) return rc;
  if (bad_logits(dtype, d_logits, dl_stride, n_rows, vocab, true) ||
      crossing(dtype, logits, row_stride, d_logits, dl_stride, n_rows, vocab))
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
  a.x2 = exponent_of(scale);
  a.ids = d_ids;
  a.top_ids = d_top_ids;
  a.entropy = d_entropy;
  a.stats = reinterpret_cast<const float2 *>(d_stats);
  a.g_logprobs = g_logprobs;
  a.g_entropy = g_entropy;
  a.g_lse = g_lse;
  a.g_top = top_k ? g_top : nullptr;
  const uint32_t pieces = most_pieces(dtype, vocab);
  const bool small = pieces <= 512;
  a.part = small ? pieces : 2 * ROW_STEP;
  a.parts = (pieces + a.part - 1) / a.part;
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const uint64_t blocks = n_rows * a.parts;
  for (; a.block0 < blocks; a.block0 += MAX_GROUPS)
    with_element(dtype, [&](auto t) {
      const uint32_t grid = uint32_t(std::min(blocks - a.block0, MAX_GROUPS));
      if (small) k_scores_back<decltype(t), 1><<<grid, 64, 0, st>>>(a);
      else k_scores_back<decltype(t), ROW_WAVES><<<grid, ROW_THREADS, 0, st>>>(a);
    });
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

}  // extern "C"
