// Distillation from a teacher's top log probabilities: divergence of a student's
// distribution from the teacher's listed tokens, and its gradient.
//
// p = softmax(scale * x) over the vocabulary; the teacher lists tokens t with
// log probabilities a_t.  Without a tail q_t = exp(a_t) / sum exp(a),
//   loss = sum_t q_t (log q_t - log p_t),   dz_j = p_j - sum_{t: t = j} q_t.
// With one, q_t = exp(a_t), and what they leave, q_r = max(0, 1 - sum q), is
// held against p_r, the student's sum over tokens that are not listed:
//   loss = sum_t q_t (log q_t - log p_t) + q_r (log q_r - log p_r),
//   dz_j = p_j (sum q + q_r) - [j not listed] q_r p_j / p_r - sum_{t: t = j} q_t.
// p_j / p_r is the softmax of the tokens that are not listed by themselves.  Where
// they lie far below the listed ones, as under a finite mask, p_j and p_r are below
// any float while that is not: so what concerns it is relative to their own largest
// element u.  With s = sum w and s_r of theirs, relative to the row's and to u,
//   dz_j = exp(z_j - u) ((sum q + q_r) exp(u - max) / s - q_r / s_r),   j not listed.
//
// One pass over the row for the largest element and the sum of weights relative
// to it; with a tail, over the tokens that are not listed alone, the listed
// ones' weights joined at the end: p_r as a difference would keep no digits
// where the list holds nearly everything.  Which tokens are listed is a bit each
// in LDS.  A row's few numbers are in 64 bits, since the loss is a difference of
// near ones where student and teacher agree.
#include "bbpe_rows.h"

#include <algorithm>

namespace bbpe {
namespace {

constexpr uint32_t LIST_MAX = 256;  // listed tokens at most
// What a list may leave of 1 by its rounding alone: each of its log probabilities a is
// off by |a| 2^-24, their q-weighted sum by log(256) 2^-24 at most, and all together by
// the log-sum that a teacher took off, 2^-18 for one of 64 in a float.  Where the
// student gives all other tokens minus infinity, as under the teacher's own mask, that
// much is nothing rather than a divergence of infinity (in every other row or so).
constexpr double ROUNDING_REST = 0x1p-18;
// Pieces that a thread holds from the loss to the gradient: 64 of the 128 registers
// that four waves a SIMD leave it.
constexpr uint32_t HELD = 16;
// Rows from which on loss and gradient of a long row are by one workgroup.  Fewer do
// not fill the card, and go to the kernels that cut rows (of 100,277 tokens in
// bfloat16, 128 rows: 29.4 us cut, 28.3 whole; 64: 24.2 and 26.2; 160: 34.7 and 29.7;
// 256: 43.9 and 33.4).
constexpr uint64_t STEP_ROWS = 160;

struct DistillArgs {
  const void *x;
  int64_t stride;
  void *dx;  // where the gradient is wanted too
  int64_t dx_stride;
  uint64_t block0;
  uint32_t vocab, k, tail, parts, part;  // parts of a row, and pieces of one
  float scale;
  Exponent x2;
  const int32_t *ids;
  const float *lp;
  float *loss, *lse;
  float4 *stats;
  const float *grad;
  Partial *parted;  // [rows][parts]
};

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmax(v, __shfl_xor(v, d, 64));
  return v;
}

// What the teacher lists for a row, and what comes of it before the row is read.
// By one wave, four entries a lane.
template <uint32_t LIST> struct ListShared {
  double q[LIST], log_q[LIST];
  alignas(16) int32_t ids[LIST];  // -1 where an entry names no token
  float own[LIST];                // the student's element; minus infinity where it is not there
  bool first[LIST], alone[LIST];  // the first entry that names this token, the only one
  double mass, rest, log_norm;
  int some;
};
template <uint32_t LIST> struct ListLoads {
  int32_t id[LIST / 64];
  float lp[LIST / 64];
};
template <uint32_t LIST>
__device__ __forceinline__ ListLoads<LIST> load_list(const DistillArgs &a, uint64_t row) {
  ListLoads<LIST> l;
#pragma unroll
  for (uint32_t i = 0; i < LIST / 64; ++i) {
    const uint32_t t = (threadIdx.x & 63) + 64 * i;
    const int32_t id = t < a.k ? a.ids[row * a.k + t] : -1;
    l.id[i] = id >= 0 && uint32_t(id) < a.vocab ? id : -1;
    l.lp[i] = l.id[i] >= 0 ? a.lp[row * a.k + t] : -INFINITY;
  }
  return l;
}
template <uint32_t LIST>
__device__ __forceinline__ void keep_ids(const ListLoads<LIST> &l, ListShared<LIST> &sh) {
#pragma unroll
  for (uint32_t i = 0; i < LIST / 64; ++i) sh.ids[(threadIdx.x & 63) + 64 * i] = l.id[i];
  __builtin_amdgcn_wave_barrier();  // the wave reads them below
}
// How a list names entry t's token: first, and nowhere else.  ids: 16-byte aligned
// in LDS, -1 from k on.
struct Named {
  bool first, alone;
};
__device__ __forceinline__ Named named(const int32_t *ids, uint32_t k, uint32_t t) {
  typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
  const int32_t id = ids[t];
  Named n{true, true};
#pragma unroll 4
  for (uint32_t s = 0; s < k; s += 4) {
    const i32x4 v = *reinterpret_cast<const i32x4 *>(ids + s);
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      n.alone &= v[e] != id || s + e == t;
      n.first &= v[e] != id || s + e >= t;
    }
  }
  return n;
}

// Of all entries, by the threads from `from` on.  (sh.ids are there)
template <uint32_t WAVES, uint32_t LIST>
__device__ __forceinline__ void read_names(const DistillArgs &a, uint32_t from, ListShared<LIST> &sh) {
  for (uint32_t t = threadIdx.x - from; t < a.k; t += 64 * WAVES - from) {
    const Named n = named(sh.ids, a.k, t);
    sh.first[t] = sh.ids[t] >= 0 && n.first;
    sh.alone[t] = n.alone;
  }
}

// What the row has for the list, and the teacher's sums, by one wave.
template <typename T, uint32_t LIST>
__device__ __forceinline__ void read_list(const DistillArgs &a, const T *x, const ListLoads<LIST> &l, ListShared<LIST> &sh) {
  constexpr uint32_t LIST_EACH = LIST / 64;
  const uint32_t lane = threadIdx.x & 63;
  float own[LIST_EACH];
  double top = -INFINITY;
  bool some = false;
#pragma unroll
  for (uint32_t i = 0; i < LIST_EACH; ++i) {
    own[i] = l.id[i] >= 0 ? float(x[l.id[i]]) : -INFINITY;
    some |= l.id[i] >= 0 && (a.tail || l.lp[i] != -INFINITY);
    top = fmax(top, double(l.lp[i]));
  }
  some = __any(some);
  double c = 0.0, mass = 0.0, rest = 0.0;
  if (!a.tail) c = wave_max(top);
#pragma unroll
  for (uint32_t i = 0; i < LIST_EACH; ++i)
    if (64 * i < a.k) mass += l.lp[i] == -INFINITY ? 0.0 : exp(double(l.lp[i]) - c);
  mass = wave_sum(mass);
  if (a.tail) rest = mass < 1.0 ? 1.0 - mass : mass == mass ? 0.0 : mass;
  else c += log(mass);
#pragma unroll
  for (uint32_t i = 0; i < LIST_EACH; ++i) {
    if (64 * i >= a.k) continue;
    const uint32_t t = lane + 64 * i;
    const double log_q = l.lp[i] == -INFINITY ? -INFINITY : double(l.lp[i]) - c;
    sh.log_q[t] = log_q;
    sh.q[t] = exp(log_q);
    sh.own[t] = own[i];
  }
  if (lane == 0) {
    sh.mass = mass;
    sh.rest = rest;
    sh.log_norm = c;
    sh.some = some;
  }
}

// The end of a row, by the wave that has read the list: p holds the weights of the
// whole row (with a tail: of the tokens that are not listed).
//
// stats: the row's maximum, and the factor of p_j in the gradient over the row's sum
// of weights (a quotient, not its logarithm, which in 32 bits would put every
// probability off by up to a millionth, all the same way).  Without a tail then the
// logarithm of the teacher's sum in two parts (any constant may be added to a list:
// in one, an offset of 10,000 would put all of q off by up to 5e-4); with one, for
// tokens that are not listed, their maximum and the factor of weights relative to that.
template <uint32_t LIST>
__device__ __forceinline__ float4 end_row(const DistillArgs &a, uint64_t row, bool tail, Partial p, const ListShared<LIST> &sh) {
  const uint32_t lane = threadIdx.x & 63;
  float high = p.max;
  if (tail) {
    for (uint32_t t = lane; t < a.k; t += 64) high = fmaxf(high, sh.own[t]);
    high = wave_max(high);
  }
  const float ref = finite_max(high);
  double others = p.sum, listed = 0.0;
  if (tail) {
    if (p.max != -INFINITY) others *= exp((double(p.max) - ref) * a.scale);
    for (uint32_t t = lane; t < a.k; t += 64) listed += sh.first[t] ? exp((double(sh.own[t]) - ref) * a.scale) : 0.0;
    listed = wave_sum(listed);
  }
  const double sum = others + listed, log_sum = log(sum);
  double loss = 0.0;
  for (uint32_t t = lane; t < a.k; t += 64) {
    const double log_q = sh.log_q[t], log_p = sh.own[t] == -INFINITY ? -INFINITY : (double(sh.own[t]) - ref) * a.scale - log_sum;
    if (sh.q[t] != 0.0) loss += sh.q[t] * (log_q - log_p);
  }
  loss = wave_sum(loss);
  const bool empty = p.max == -INFINITY && p.sum == 0.0;  // of tokens that are not listed
  const double rest = empty && sh.rest <= ROUNDING_REST ? 0.0 : sh.rest, mass = sh.mass;
  if (rest > 0.0) {
    // log p_r = -log(1 + listed / others): of the ratio, not of two logarithms, until
    // it leaves the range of numbers and 1 is nothing beside it
    // (__any: all lanes hold the same, and a branch leaves one of the logarithms out)
    loss += rest * (log(rest) + (__any(others > 1e-200) ? log1p(listed / others) : log(listed / p.sum) - (double(p.max) - ref) * a.scale));
  }
  const bool none = high == -INFINITY && sum == 0.0, bad = !(sum == sum) || high == INFINITY;
  const float nan = __uint_as_float(0x7FC00000u);
  float4 st = make_float4(high, float(1.0 / sum), float(sh.log_norm), float(sh.log_norm - double(float(sh.log_norm))));
  if (tail) {
    st.y = float((mass + rest) / sum);
    st.z = finite_max(p.max);
    st.w = empty ? 0.0f : float((mass + rest) / sum * (others / p.sum) - rest / p.sum);
  }
  if (!sh.some) {  // no teacher: no loss and no gradient, whatever the row holds
    loss = 0.0;
    st.x = -INFINITY;
  } else if (bad) {
    loss = nan;
    st = make_float4(0.0f, nan, nan, nan);
  } else if (none) {
    loss = INFINITY;
  }
  if (lane == 0) {
    a.loss[row] = float(loss);
    a.lse[row] = bad ? nan : none ? -INFINITY : float(double(high) * a.scale + log_sum);
    a.stats[row] = st;
  }
  return st;
}

// Tokens by which bits of the list are set at a time, 16 or (float32) 32 steps.
template <uint32_t WAVES> constexpr uint32_t BITS = 64 * WAVES * ROW_UNROLL * 8 * 16;

template <uint32_t WAVES, bool TAIL, uint32_t LIST> struct DistillShared {
  Partial sums[WAVES];
  ListShared<LIST> list;
  uint32_t bits[TAIL ? BITS<WAVES> / 32 : 1];
  float4 stats;
};

// Sets the bits of listed tokens among `pieces` pieces from `first` on.
template <typename T, uint32_t WAVES, bool TAIL, uint32_t LIST>
__device__ __forceinline__ void set_bits(const DistillArgs &a, const Row<const T> &r, uint32_t first, uint32_t pieces,
                                         DistillShared<WAVES, TAIL, LIST> &sh) {
  constexpr uint32_t THREADS = 64 * WAVES;
  const uint32_t tid = threadIdx.x, from = first * Piece<T>::N, words = (pieces * Piece<T>::N + 31) / 32;
  __syncthreads();
  for (uint32_t w = tid; w < words; w += THREADS) sh.bits[w] = 0;
  __syncthreads();
  for (uint32_t t = tid; t < a.k; t += THREADS) {
    const uint32_t place = sh.list.ids[t] >= 0 ? r.lead + uint32_t(sh.list.ids[t]) - from : ~0u;
    if (place < words * 32) atomicOr(&sh.bits[place / 32], 1u << place % 32);
  }
  __syncthreads();
}

// Adds a step's pieces to s; with a tail, their tokens that are not listed.  at:
// the thread's first piece, counted from where the bits begin.
template <typename T, uint32_t WAVES, bool TAIL, uint32_t LIST>
__device__ __forceinline__ void add_step(const DistillArgs &a, const typename Piece<T>::raw *raw, uint32_t at, DistillShared<WAVES, TAIL, LIST> &sh,
                                         Partial &s) {
  typedef Piece<T> P;
  typename P::val v[ROW_UNROLL];
  float m = -INFINITY;
#pragma unroll
  for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
    v[u] = values<T>(raw[u]);
    if (TAIL) {
      const uint32_t place = (at + u * 64 * WAVES) * P::N;  // (past the row: of old bits, and nothing to mask)
      const uint32_t mask = sh.bits[place / 32] >> place % 32 & ((1u << P::N) - 1);
      if (__any(mask)) {
#pragma unroll
        for (uint32_t e = 0; e < P::N; ++e) v[u][e] = mask >> e & 1 ? -INFINITY : v[u][e];
      }
    }
#pragma unroll
    for (uint32_t e = 0; e < P::N; ++e) m = fmaxf(m, v[u][e]);
  }
  if (m > s.max) {
    if (s.max != -INFINITY) s.sum *= double(fine_weight(s.max - m, a.x2));
    s.max = m;
  }
  const float ref = finite_max(s.max);
#pragma unroll
  for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
#pragma unroll
    for (uint32_t e = 0; e < P::N; ++e) v[u][e] = weight_of(v[u][e] - ref, a.x2);
    s.sum += double(piece_sum<P::N>(v[u]));
  }
}

// Adds pieces [first, last) of a row to s; with a tail, their tokens that are not
// listed.
template <typename T, uint32_t WAVES, bool TAIL, uint32_t LIST>
__device__ __forceinline__ void add_pieces(const DistillArgs &a, const Row<const T> &r, uint32_t first, uint32_t last,
                                           DistillShared<WAVES, TAIL, LIST> &sh, Partial &s) {
  constexpr uint32_t THREADS = 64 * WAVES, STEP = THREADS * ROW_UNROLL;
  constexpr uint32_t STRETCH = BITS<WAVES> / Piece<T>::N;  // pieces between two settings of the bits
  for (uint32_t p0 = first; p0 < last; p0 += STEP) {
    if (TAIL && (p0 - first) % STRETCH == 0) set_bits<T>(a, r, p0, min(last - p0, STRETCH), sh);
    typename Piece<T>::raw raw[ROW_UNROLL];
    r.template load_step<THREADS>(raw, r.at, p0 + threadIdx.x, last);
    add_step<T>(a, raw, (p0 - first) % STRETCH + threadIdx.x, sh, s);
  }
}

// The gradient of a row from its stats.
template <typename T, uint32_t WAVES> struct Gradient {
  static constexpr uint32_t THREADS = 64 * WAVES;
  float4 st;
  float g, base, factor;  // of tokens that are not listed: g * factor * exp(scale * (x - base))
  Exponent x2;
  bool zero;

  __device__ __forceinline__ Gradient(const DistillArgs &a, bool tail, float4 stats, float grad) : st(stats), g(grad * a.scale), x2(a.x2) {
    zero = st.x == -INFINITY || g == 0.0f;
    base = tail ? st.z : st.x;
    factor = tail ? st.w : st.y;
  }
  __device__ __forceinline__ typename Piece<T>::val of(typename Piece<T>::raw raw) const {
    typename Piece<T>::val v = 0.0f;
    if (zero) return v;
    const float all = g * factor;
    v = values<T>(raw);
#pragma unroll
    for (uint32_t e = 0; e < Piece<T>::N; ++e) v[e] = weight_of(v[e] - base, x2) * all;  // (of listed ones anything: they are written once more)
    return v;
  }
  // Pieces [from, to), as out has them.
  __device__ __forceinline__ void pieces(const T *x, const Row<T> &out, uint32_t from, uint32_t to) const {
    for (uint32_t p0 = from; p0 < to; p0 += THREADS * ROW_UNROLL) {
      typename Piece<T>::raw raw[ROW_UNROLL];
      if (!zero) out.template load_step<THREADS>(raw, x - out.lead, p0 + threadIdx.x, to);
#pragma unroll
      for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
        const uint32_t p = p0 + u * THREADS + threadIdx.x;
        if (p < to) out.store(p, of(raw[u]));
      }
    }
  }
  // The listed tokens among pieces [from, to), written once more when those are (a
  // barrier apart) from what was there before (dx may be x): each by one thread,
  // or by several with the same value.
  template <typename Q>
  __device__ __forceinline__ void listed(const DistillArgs &a, const Row<T> &out, uint32_t from, uint32_t to, const int32_t *ids, const bool *alone,
                                         const float *own, const Q *q) const {
    if (zero) return;
    for (uint32_t t = threadIdx.x; t < a.k; t += THREADS) {
      const int32_t id = ids[t];
      const uint32_t place = out.lead + uint32_t(id);
      if (id < 0 || place / Piece<T>::N - from >= to - from) continue;
      float sum = float(q[t]);
      if (!alone[t]) {
        sum = 0.0f;
        for (uint32_t i = 0; i < a.k; ++i) sum += ids[i] == id ? float(q[i]) : 0.0f;
      }
      out.at[place] = T(g * (st.y * fine_weight(own[t] - st.x, x2) - sum));
    }
  }
};

// The loss: a workgroup a row or, SPLIT, a part of one.
//
// Bound by the one read of the row: 4,096 rows of 100,277 in bfloat16 with a tail,
// 160 us (5.1 TB/s).  The listed tokens' bits cost a word of LDS a piece, and a
// branch that one piece in hundreds takes.
template <typename T, uint32_t WAVES, bool TAIL, bool SPLIT, uint32_t LIST>
__global__ __launch_bounds__(64 * WAVES) void k_distill(DistillArgs a) {
  __shared__ DistillShared<WAVES, TAIL, LIST> sh;
  const uint64_t block = a.block0 + blockIdx.x, row = SPLIT ? block / a.parts : block;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  const Row<const T> r(x, a.vocab);
  const uint32_t first = SPLIT ? uint32_t(block % a.parts) * a.part : 0;
  if ((TAIL || !SPLIT) && threadIdx.x < 64) {
    const ListLoads<LIST> l = load_list<LIST>(a, row);
    keep_ids(l, sh.list);
    if (!SPLIT) read_list(a, x, l, sh.list);
  }
  if (TAIL && !SPLIT) {
    __syncthreads();
    if (WAVES == 1 || threadIdx.x >= 64) read_names<WAVES>(a, WAVES == 1 ? 0 : 64, sh.list);
  }
  Partial s{0.0, -INFINITY, 0.0f};
  add_pieces<T>(a, r, first, SPLIT ? min(r.pieces(), first + a.part) : r.pieces(), sh, s);
  s = row_partial<WAVES>(s, a.x2, sh.sums);  // (with a barrier, for the list too)
  if (SPLIT) {
    if (threadIdx.x == 0) a.parted[block] = s;
  } else if (threadIdx.x < 64) {
    end_row(a, row, TAIL, s, sh.list);
  }
}

// Loss and gradient of a row by a workgroup.  A thread's first HELD pieces stay in
// its registers between the two and, of 16 waves, some more in LDS; what a row has
// besides is read again.
//
// Bound by the read and the write of a row where it is held (4,096 rows of 100,277
// in bfloat16 with a tail, 64 listed: 390 us, 4.2 TB/s; the two kernels apart 479), and by
// what is read again where it is not (2,048 rows of 200,005 in float32, 256 listed: 811
// us, 4.0 TB/s in two moves; of a row of 800 KB 384 are held or kept).  All of a
// workgroup loads before any of it stores, so a CU needs workgroups besides: that is
// why waves are no more than a row needs.  Rows that are not many times what the card
// holds at once leave it mostly idle in the end: of 8 waves two workgroups a CU, 512 in
// all, so 1,111 rows take three turns (68 us, where their bytes take 45).  Loading the next row's pieces ahead spilled (936 us for
// 403).
template <typename T, uint32_t WAVES, bool TAIL, uint32_t LIST>
__global__ __launch_bounds__(64 * WAVES, 4) void k_distill_step(DistillArgs a) {
  constexpr uint32_t THREADS = 64 * WAVES, STEP = THREADS * ROW_UNROLL;
  constexpr uint32_t KEPT = WAVES < 16 ? 0 : TAIL ? 4 : 8;
  static_assert(HELD % ROW_UNROLL == 0 && KEPT % ROW_UNROLL == 0 && THREADS * (HELD + KEPT) * Piece<T>::N <= BITS<WAVES>, "");
  __shared__ DistillShared<WAVES, TAIL, LIST> sh;
  __shared__ typename Piece<T>::raw kept[KEPT ? KEPT * THREADS : 1];
  const uint64_t row = a.block0 + blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  T *dx = static_cast<T *>(a.dx) + int64_t(row) * a.dx_stride;
  const Row<const T> r(x, a.vocab);
  const uint32_t tid = threadIdx.x, pieces = r.pieces(), held = min(pieces, THREADS * HELD), near = min(pieces, THREADS * (HELD + KEPT));
  const float weight = a.grad[row];
  ListLoads<LIST> l;
  if (tid < 64) l = load_list<LIST>(a, row);
  typename Piece<T>::raw raw[HELD / ROW_UNROLL][ROW_UNROLL];
#pragma unroll
  for (uint32_t i = 0; i < HELD / ROW_UNROLL; ++i) r.template load_step<THREADS>(raw[i], r.at, i * STEP + tid, held);
  if (tid < 64) keep_ids(l, sh.list);
  if (TAIL) set_bits<T>(a, r, 0, near, sh);
  else __syncthreads();
  if (tid < 64) read_list(a, x, l, sh.list);
  if (WAVES == 1 || tid >= 64) read_names<WAVES>(a, WAVES == 1 ? 0 : 64, sh.list);
  Partial s{0.0, -INFINITY, 0.0f};
#pragma unroll
  for (uint32_t i = 0; i < HELD / ROW_UNROLL; ++i)
    if (i * STEP < held) add_step<T>(a, raw[i], i * STEP + tid, sh, s);
#pragma unroll
  for (uint32_t i = 0; i < KEPT / ROW_UNROLL; ++i) {
    const uint32_t p = THREADS * HELD + i * STEP + tid;
    if (p - tid >= near) break;
    typename Piece<T>::raw more[ROW_UNROLL];
    r.template load_step<THREADS>(more, r.at, p, near);
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) kept[i * STEP + u * THREADS + tid] = more[u];
    add_step<T>(a, more, p, sh, s);
  }
  add_pieces<T>(a, r, near, pieces, sh, s);
  s = row_partial<WAVES>(s, a.x2, sh.sums);
  if (tid < 64) {
    const float4 st = end_row(a, row, TAIL, s, sh.list);
    if (tid == 0) sh.stats = st;
  }
  __syncthreads();
  const Gradient<T, WAVES> grad(a, TAIL, sh.stats, weight);
  const Row<T> out = r.over(dx);
#pragma unroll
  for (uint32_t i = 0; i < HELD; ++i) {
    const uint32_t p = i * THREADS + tid;
    if (p < held) out.store(p, grad.of(raw[i / ROW_UNROLL][i % ROW_UNROLL]));
  }
#pragma unroll
  for (uint32_t i = 0; i < KEPT; ++i) {
    const uint32_t p = (HELD + i) * THREADS + tid;
    if (p < near) out.store(p, grad.of(kept[i * THREADS + tid]));
  }
  grad.pieces(x, out, near, pieces);
  __syncthreads();
  grad.listed(a, out, 0, pieces, sh.list.ids, sh.list.alone, sh.list.own, sh.list.q);
}

// Joins a row's parts.
template <typename T>
__global__ __launch_bounds__(64) void k_distill_join(DistillArgs a) {
  __shared__ ListShared<LIST_MAX> sh;
  const uint64_t row = a.block0 + blockIdx.x;
  Partial p{0.0, -INFINITY, 0.0f};
  if (threadIdx.x < a.parts) p = a.parted[row * a.parts + threadIdx.x];
  const ListLoads<LIST_MAX> l = load_list<LIST_MAX>(a, row);
  keep_ids(l, sh);
  __syncthreads();
  read_list(a, static_cast<const T *>(a.x) + int64_t(row) * a.stride, l, sh);
  if (a.tail) read_names<1>(a, 0, sh);
  p = wave_partial(p, a.x2);
  __syncthreads();
  end_row(a, row, a.tail, p, sh);
}

// The gradient by itself: a workgroup a part of a row.
//
// Bound by the row's read and write (4,096 rows of 100,277 in bfloat16 with a tail: 309
// us, 5.3 TB/s).  A wave by itself is held to the registers of eight on a SIMD, which the
// list's exponentials in 64 bits would pass (65,536 rows of 1,280 76.1 us, with seven
// 83.5; of 1,024 60.3 and 68.8; of 2,048 119.7 and 117.1); workgroups of four are not (those
// 4,096 rows would take 324 us).
template <typename T, uint32_t WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 1 ? 8 : 1) void k_distill_back(DistillArgs a) {
  constexpr uint32_t THREADS = 64 * WAVES;
  __shared__ alignas(16) int32_t ids[LIST_MAX];
  __shared__ float own[LIST_MAX], q[LIST_MAX];
  __shared__ bool alone[LIST_MAX];
  const uint64_t block = a.block0 + blockIdx.x, row = block / a.parts;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  const Row<T> r(static_cast<T *>(a.dx) + int64_t(row) * a.dx_stride, a.vocab);
  const uint32_t from = uint32_t(block % a.parts) * a.part, to = min(r.pieces(), from + a.part);
  if (from >= to) return;  // (parts are counted for rows that begin anywhere)
  const Gradient<T, WAVES> grad(a, a.tail, a.stats[row], a.grad[row]);
  const double norm = a.tail ? 0.0 : double(grad.st.z) + grad.st.w;
  for (uint32_t t = threadIdx.x; t < (a.k + 3) / 4 * 4; t += THREADS) {  // (named() reads four at a time)
    const int32_t id = t < a.k ? a.ids[row * a.k + t] : -1;
    const bool there = id >= 0 && uint32_t(id) < a.vocab;
    ids[t] = there ? id : -1;
    if (t >= a.k) continue;
    q[t] = there ? float(exp(double(a.lp[row * a.k + t]) - norm)) : 0.0f;
    own[t] = there && (r.lead + uint32_t(id)) / Piece<T>::N - from < to - from ? float(x[id]) : 0.0f;
  }
  __syncthreads();
  // (of the entries that this part has: listed() looks at no others)
  for (uint32_t t = threadIdx.x; t < a.k; t += THREADS)
    if (ids[t] >= 0 && (r.lead + uint32_t(ids[t])) / Piece<T>::N - from < to - from) alone[t] = named(ids, a.k, t).alone;
  grad.pieces(x, r, from, to);
  __syncthreads();
  grad.listed(a, r, from, to, ids, alone, own, q);
}

int check(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab, const int32_t *ids, const float *lp,
          uint32_t k, int tail, float scale) {
  if (bad_logits(dtype, logits, row_stride, n_rows, vocab, false) || k == 0 || k > LIST_MAX || tail < 0 || tail > 1 ||
      k > vocab || (tail && k >= vocab) || bad_scale(scale))
    return BBPE_E_INVALID_ARG;
  if ((n_rows && (!ids || !lp)) || ((address(ids) | address(lp)) & 3)) return BBPE_E_INVALID_ARG;
  return BBPE_OK;
}

DistillArgs args_of(const void *logits, int64_t row_stride, uint32_t vocab, const int32_t *ids, const float *lp, uint32_t k, int tail, float scale) {
  DistillArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.vocab = vocab;
  a.k = k;
  a.tail = uint32_t(tail);
  a.scale = scale;
  a.x2 = exponent_of(scale);
  a.ids = ids;
  a.lp = lp;
  return a;
}

uint64_t parted_bytes(const Cut &cut, uint64_t n_rows) { return cut.parts > 1 ? n_rows * cut.parts * sizeof(Partial) : 0; }

// The gradient from rows' stats.
void launch_back(DistillArgs a, int dtype, uint64_t n_rows, hipStream_t st) {
  const uint32_t pieces = most_pieces(dtype, a.vocab);
  const bool small = pieces <= 512;
  a.part = small ? pieces : 2 * ROW_STEP;
  a.parts = (pieces + a.part - 1) / a.part;
  const uint64_t blocks = n_rows * a.parts;
  with_element(dtype, [&](auto t) {
    for (a.block0 = 0; a.block0 < blocks; a.block0 += MAX_GROUPS) {
      const uint32_t grid = uint32_t(std::min(blocks - a.block0, MAX_GROUPS));
      if (small) k_distill_back<decltype(t), 1><<<grid, 64, 0, st>>>(a);
      else k_distill_back<decltype(t), ROW_WAVES><<<grid, ROW_THREADS, 0, st>>>(a);
    }
  });
}

}  // namespace
}  // namespace bbpe

using namespace bbpe;

extern "C" {

int bbpe_distill_loss_workspace_bytes(int dtype, uint64_t n_rows, uint32_t vocab, uint64_t *out_bytes) {
  if (!out_bytes || bad_sizes(dtype, n_rows, vocab)) return BBPE_E_INVALID_ARG;
  // (a list's length decides whether short rows go to waves: the larger of both)
  *out_bytes = parted_bytes(cut_rows(dtype, n_rows, vocab, false, PARTS_MAX), n_rows);
  return BBPE_OK;
}

int bbpe_distill_loss_backward(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                               const int32_t *d_top_ids, const float *d_top_logprobs, uint32_t top_k, int tail, float scale,
                               const float *d_stats, const float *d_grad, void *d_logits, int64_t dl_stride, void *hip_stream) {
  const int rc = check(dtype, logits, row_stride, n_rows, vocab, d_top_ids, d_top_logprobs, top_k, tail, scale);
  if (rc) return rc;
  if (bad_logits(dtype, d_logits, dl_stride, n_rows, vocab, true) ||
      crossing(dtype, logits, row_stride, d_logits, dl_stride, n_rows, vocab) || (n_rows && (!d_stats || !d_grad)) ||
      (address(d_stats) & 15) || (address(d_grad) & 3))
    return BBPE_E_INVALID_ARG;
  if (n_rows == 0) return BBPE_OK;
  DistillArgs a = args_of(logits, row_stride, vocab, d_top_ids, d_top_logprobs, top_k, tail, scale);
  a.dx = d_logits;
  a.dx_stride = dl_stride;
  a.stats = reinterpret_cast<float4 *>(const_cast<float *>(d_stats));
  a.grad = d_grad;
  launch_back(a, dtype, n_rows, static_cast<hipStream_t>(hip_stream));
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

int bbpe_distill_loss(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                      const int32_t *d_top_ids, const float *d_top_logprobs, uint32_t top_k, int tail, float scale,
                      float *d_loss, float *d_lse, float *d_stats, const float *d_weights, void *d_logits, int64_t dl_stride,
                      void *d_workspace, uint64_t workspace_bytes, void *hip_stream) {
  const int rc = check(dtype, logits, row_stride, n_rows, vocab, d_top_ids, d_top_logprobs, top_k, tail, scale);
  if (rc) return rc;
  if ((n_rows && (!d_loss || !d_lse || !d_stats)) || ((address(d_loss) | address(d_lse) | address(d_weights)) & 3) ||
      (address(d_stats) & 15) || (d_weights == nullptr) != (d_logits == nullptr) ||
      (d_logits && (bad_logits(dtype, d_logits, dl_stride, n_rows, vocab, true) ||
                    crossing(dtype, logits, row_stride, d_logits, dl_stride, n_rows, vocab))))
    return BBPE_E_INVALID_ARG;
  if (n_rows == 0) return BBPE_OK;
  const Cut cut = cut_rows(dtype, n_rows, vocab, top_k <= 64, PARTS_MAX);
  const uint64_t need = parted_bytes(cut, n_rows);
  if (need && (!d_workspace || (address(d_workspace) & 255) || workspace_bytes < need)) return BBPE_E_WORKSPACE;
  DistillArgs a = args_of(logits, row_stride, vocab, d_top_ids, d_top_logprobs, top_k, tail, scale);
  a.dx = d_logits;
  a.dx_stride = dl_stride;
  a.parts = cut.parts;
  a.part = cut.part;
  a.loss = d_loss;
  a.lse = d_lse;
  a.stats = reinterpret_cast<float4 *>(d_stats);
  a.grad = d_weights;
  a.parted = static_cast<Partial *>(d_workspace);
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const auto launch = [&](uint64_t blocks, auto kernel, uint32_t threads) {
    for (a.block0 = 0; a.block0 < blocks; a.block0 += MAX_GROUPS)
      kernel<<<uint32_t(std::min(blocks - a.block0, MAX_GROUPS)), threads, 0, st>>>(a);
  };
  // Loss and gradient of a row by one workgroup, of as few waves as hold it:
  //   one, up to 1,024 pieces (8,192 rows of 8,192 in bfloat16: 61.5 us, four 81.7;
  //   of 16,384, more than it holds: 157 and 113);
  //   four, up to 3,584 (4,096 rows of 28,000: 104 us, eight 106; of 32,000, 119 and 113);
  //   eight, up to 8,192, and for 16-bit rows of any length (2,048 of 65,536: 115 us,
  //   four 146; of 100,277: 206, sixteen 230);
  //   sixteen for longer ones of float32 (2,048 of 100,277, 64 listed: 340 us, eight 427,
  //   256 listed 363 and 461; of 200,005: 773 and 955, 817 and 1,000).
  const uint32_t per = dtype == BBPE_F32 ? 4 : 8, pieces = (vocab + per - 1) / per;
  const bool whole = d_logits && (n_rows >= STEP_ROWS || pieces <= 256 * HELD);
  with_element(dtype, [&](auto t) {
    typedef decltype(t) T;
    const auto by_tail = [&](uint64_t blocks, uint32_t threads, auto without, auto with) { launch(blocks, tail ? with : without, threads); };
    constexpr uint32_t W = ROW_WAVES, L = LIST_MAX;
    if (whole) {
      if (pieces <= 64 * HELD && top_k <= 64) by_tail(n_rows, 64, k_distill_step<T, 1, false, 64>, k_distill_step<T, 1, true, 64>);
      else if (pieces <= 224 * HELD) by_tail(n_rows, 256, k_distill_step<T, 4, false, L>, k_distill_step<T, 4, true, L>);
      else if (pieces <= 512 * HELD || sizeof(T) == 2) by_tail(n_rows, 512, k_distill_step<T, 8, false, L>, k_distill_step<T, 8, true, L>);
      else if constexpr (sizeof(T) == 4) by_tail(n_rows, 1024, k_distill_step<T, 16, false, L>, k_distill_step<T, 16, true, L>);
    } else if (cut.parts > 1) {
      by_tail(n_rows * cut.parts, ROW_THREADS, k_distill<T, W, false, true, L>, k_distill<T, W, true, true, L>);
      launch(n_rows, k_distill_join<T>, 64);
    } else if (cut.waves == 1) {
      by_tail(n_rows, 64, k_distill<T, 1, false, false, 64>, k_distill<T, 1, true, false, 64>);
    } else {
      by_tail(n_rows, ROW_THREADS, k_distill<T, W, false, false, L>, k_distill<T, W, true, false, L>);
    }
  });
  if (hipGetLastError() != hipSuccess) return BBPE_E_HIP;
  if (d_logits && !whole) launch_back(a, dtype, n_rows, st);
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

}  // extern "C"
