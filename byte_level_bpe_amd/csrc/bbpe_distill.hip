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
constexpr uint32_t STEP_WAVES = 8;  // of a workgroup that makes loss and gradient

struct DistillArgs {
  const void *x;
  int64_t stride;
  void *dx;  // where the gradient is wanted too
  int64_t dx_stride;
  uint64_t block0;
  uint32_t vocab, k, tail, parts, part;  // parts of a row, and pieces of one
  float scale, c;
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

// The end of a row, by one wave: p holds the weights of the whole row (with a
// tail: of the tokens that are not listed).  ids: the row's list in LDS, -1
// where an entry names no token.
//
// stats: the row's maximum and the logarithm of its sum of weights; the factor
// of p_j in the gradient, of tokens that are not listed; with a tail the listed
// ones' factor, without one the logarithm of the teacher's sum.
template <typename T>
__device__ __forceinline__ float4 end_row(const DistillArgs &a, uint64_t row, const T *x, Partial p, const int32_t *ids) {
  constexpr uint32_t E = LIST_MAX / 64;
  const uint32_t lane = threadIdx.x & 63;
  const float *lp = a.lp + row * a.k;
  double teach[E];
  float own[E];
  bool first[E];  // of the entries that name this token
  double top = -INFINITY;
  float high = p.max;
  bool some = false;
#pragma unroll
  for (uint32_t i = 0; i < E; ++i) {
    teach[i] = -INFINITY;
    own[i] = -INFINITY;
    first[i] = false;
    if (64 * i >= a.k) continue;
    const uint32_t t = lane + 64 * i;
    const int32_t id = t < a.k ? ids[t] : -1;
    if (id >= 0) {
      own[i] = float(x[id]);
      teach[i] = double(lp[t]);
    }
    some |= id >= 0 && (a.tail || teach[i] != -INFINITY);
    top = fmax(top, teach[i]);
    if (a.tail) {
      high = fmaxf(high, own[i]);
      first[i] = id >= 0;
      for (uint32_t s = 0; s < t && s < a.k; ++s) first[i] &= ids[s] != id;
    }
  }
  some = __any(some);
  // the teacher
  double c = 0.0, mass = 0.0, rest = 0.0;
  if (!a.tail) c = top = wave_max(top);
#pragma unroll
  for (uint32_t i = 0; i < E; ++i)
    if (64 * i < a.k) mass += teach[i] == -INFINITY ? 0.0 : exp(teach[i] - c);
  mass = wave_sum(mass);
  if (a.tail) rest = mass < 1.0 ? 1.0 - mass : mass == mass ? 0.0 : mass;
  else c += log(mass);
  // the student
  if (a.tail) high = wave_max(high);
  const float ref = finite_max(high);
  double others = double(p.sum), listed = 0.0;
  if (a.tail) {
    if (p.max != -INFINITY) others *= exp((double(p.max) - ref) * a.scale);
#pragma unroll
    for (uint32_t i = 0; i < E; ++i)
      if (64 * i < a.k && first[i]) listed += exp((double(own[i]) - ref) * a.scale);
    listed = wave_sum(listed);
  }
  const double sum = others + listed, log_sum = log(sum);
  double loss = 0.0;
#pragma unroll
  for (uint32_t i = 0; i < E; ++i) {
    if (64 * i >= a.k || teach[i] == -INFINITY) continue;
    const double log_q = teach[i] - c, q = exp(log_q);
    const double log_p = own[i] == -INFINITY ? -INFINITY : (double(own[i]) - ref) * a.scale - log_sum;
    if (q != 0.0) loss += q * (log_q - log_p);
  }
  loss = wave_sum(loss);
  double ratio = 0.0;
  if (rest > 0.0) {
    // log p_r = -log(1 + listed / others): of the ratio, not of two logarithms
    loss += rest * (log(rest) + log1p(listed / others));
    ratio = others > 0.0 ? rest * (1.0 + listed / others) : 0.0;
  }
  const bool none = high == -INFINITY && sum == 0.0, bad = !(sum == sum) || high == INFINITY;
  const float nan = __uint_as_float(0x7FC00000u);
  float4 st = make_float4(high, float(log_sum), 0.0f, 0.0f);
  if (!some) {  // no teacher: no loss and no gradient, whatever the row holds
    loss = 0.0;
    st.x = -INFINITY;
  } else if (bad) {
    loss = nan;
    st.x = 0.0f;
    st.y = nan;
  } else if (none) {
    loss = INFINITY;
  }
  if (a.tail) {
    st.z = float(mass + rest - ratio);
    st.w = float(mass + rest);
  } else {
    st.z = 1.0f;
    st.w = float(c);
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

template <uint32_t WAVES, bool TAIL> struct DistillShared {
  Partial sums[WAVES];
  int32_t ids[LIST_MAX];  // the row's list, -1 where an entry names no token
  float q[LIST_MAX];
  uint32_t bits[TAIL ? BITS<WAVES> / 32 : 1];
  float4 stats;
};

// The list to LDS, without a barrier.
template <uint32_t WAVES>
__device__ __forceinline__ void load_list(const DistillArgs &a, uint64_t row, int32_t *ids) {
  for (uint32_t t = threadIdx.x; t < a.k; t += 64 * WAVES) {
    const int32_t id = a.ids[row * a.k + t];
    ids[t] = id >= 0 && uint32_t(id) < a.vocab ? id : -1;
  }
}

// The weights of pieces [first, last) of a row; with a tail, of tokens that are
// not listed.
template <typename T, uint32_t WAVES, bool TAIL>
__device__ __forceinline__ Partial sum_pieces(const DistillArgs &a, const Row<const T> &r, uint32_t first, uint32_t last,
                                              DistillShared<WAVES, TAIL> &sh) {
  typedef Piece<T> P;
  constexpr uint32_t THREADS = 64 * WAVES, STEP = THREADS * ROW_UNROLL;
  constexpr uint32_t STRETCH = BITS<WAVES> / P::N;  // pieces between two settings of the bits
  const uint32_t tid = threadIdx.x;
  last = min(last, r.pieces());
  Partial s{-INFINITY, 0.0f, 0.0f};
  float ref = 0.0f;
  for (uint32_t p0 = first; p0 < last; p0 += STEP) {
    if (TAIL && (p0 - first) % STRETCH == 0) {
      const uint32_t from = p0 * P::N, words = (min(last - p0, STRETCH) * P::N + 31) / 32;
      __syncthreads();
      for (uint32_t w = tid; w < words; w += THREADS) sh.bits[w] = 0;
      __syncthreads();
      for (uint32_t t = tid; t < a.k; t += THREADS) {
        const uint32_t place = sh.ids[t] >= 0 ? r.lead + uint32_t(sh.ids[t]) - from : ~0u;
        if (place < words * 32) atomicOr(&sh.bits[place / 32], 1u << place % 32);
      }
      __syncthreads();
    }
    typename P::raw raw[ROW_UNROLL];
    r.template load_step<THREADS>(raw, r.at, p0 + tid, last);
    typename P::val v[ROW_UNROLL];
    float m = -INFINITY;
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      v[u] = values<T>(raw[u]);
      if (TAIL) {
        const uint32_t place = ((p0 - first) % STRETCH + u * THREADS + tid) * P::N;  // (past `last`: of old bits, and nothing to mask)
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
      s.sum = s.max == -INFINITY ? s.sum : relative(s, m, a.c).sum;
      ref = s.max = m;
    }
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u)
#pragma unroll
      for (uint32_t e = 0; e < P::N; ++e) s.sum += __builtin_amdgcn_exp2f((v[u][e] - ref) * a.c);
  }
  return row_partial<WAVES>(s, a.c, sh.sums);  // (with a barrier, for the list too)
}

// The gradient of pieces [from, to) of a row as they are written, from its stats
// and list in LDS.  The listed tokens are written once more when the part is
// done, from what was there before (dx may be x): each by one thread, or by
// several with the same value.
template <typename T, uint32_t WAVES>
__device__ __forceinline__ void grad_pieces(const DistillArgs &a, uint64_t row, const T *x, const Row<T> &r, uint32_t from, uint32_t to, float4 st,
                                            const int32_t *ids, float *q) {
  typedef Piece<T> P;
  constexpr uint32_t THREADS = 64 * WAVES, STEP = THREADS * ROW_UNROLL, TERMS = (LIST_MAX + THREADS - 1) / THREADS;
  const uint32_t tid = threadIdx.x;
  const float g = a.grad[row] * a.scale;
  const bool zero = st.x == -INFINITY || g == 0.0f;
  const float inv = __builtin_amdgcn_exp2f(-st.y * LOG2E);
  const auto weight = [&](float v) { return __builtin_amdgcn_exp2f((v - st.x) * a.c); };
  float before[TERMS];
  bool mine[TERMS];
#pragma unroll
  for (uint32_t i = 0; i < TERMS; ++i) {
    const uint32_t t = tid + i * THREADS;
    mine[i] = false;
    if (t >= a.k) continue;
    const int32_t id = ids[t];
    q[t] = id >= 0 ? __builtin_amdgcn_exp2f((a.lp[row * a.k + t] - (a.tail ? 0.0f : st.w)) * LOG2E) : 0.0f;
    mine[i] = id >= 0 && !zero && (r.lead + uint32_t(id)) / P::N - from < to - from;
    if (mine[i]) before[i] = float(x[id]);
  }
  __syncthreads();
  const float all = g * st.z * inv;
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
        for (uint32_t e = 0; e < P::N; ++e) v[e] = weight(v[e]) * all;
      }
      r.store(p, v);
    }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < TERMS; ++i) {
    if (!mine[i]) continue;
    const int32_t id = ids[tid + i * THREADS];
    float sum = 0.0f;
    for (uint32_t t = 0; t < a.k; ++t) sum += ids[t] == id ? q[t] : 0.0f;
    r.at[r.lead + uint32_t(id)] = T(g * ((a.tail ? st.w : st.z) * inv * weight(before[i]) - sum));
  }
}

// A workgroup a row or, SPLIT, a part of one.  GRAD: the gradient too, the row
// read again while it is near.
template <typename T, uint32_t WAVES, bool TAIL, bool SPLIT, bool GRAD>
__global__ __launch_bounds__(64 * WAVES) void k_distill(DistillArgs a) {
  __shared__ DistillShared<WAVES, TAIL> sh;
  const uint64_t block = a.block0 + blockIdx.x, row = SPLIT ? block / a.parts : block;
  const uint32_t first = SPLIT ? uint32_t(block % a.parts) * a.part : 0;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  if (TAIL || !SPLIT) load_list<WAVES>(a, row, sh.ids);
  const Partial s = sum_pieces<T, WAVES, TAIL>(a, Row<const T>(x, a.vocab), first, SPLIT ? first + a.part : ~0u, sh);
  if (SPLIT) {
    if (threadIdx.x == 0) a.parted[block] = s;
    return;
  }
  if (threadIdx.x < 64) {
    const float4 st = end_row<T>(a, row, x, s, sh.ids);
    if (GRAD && threadIdx.x == 0) sh.stats = st;
  }
  if (!GRAD) return;
  __syncthreads();
  const Row<T> r(static_cast<T *>(a.dx) + int64_t(row) * a.dx_stride, a.vocab);
  grad_pieces<T, WAVES>(a, row, x, r, 0, r.pieces(), sh.stats, sh.ids, sh.q);
}

// Joins a row's parts.
template <typename T>
__global__ __launch_bounds__(64) void k_distill_join(DistillArgs a) {
  __shared__ int32_t ids[LIST_MAX];
  const uint64_t row = a.block0 + blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  load_list<1>(a, row, ids);
  Partial p{-INFINITY, 0.0f, 0.0f};
  if (threadIdx.x < a.parts) p = a.parted[row * a.parts + threadIdx.x];
  p = wave_partial(p, a.c);
  __syncthreads();
  end_row<T>(a, row, x, p, ids);
}

// The gradient by itself: a workgroup a part of a row.
template <typename T, uint32_t WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_distill_back(DistillArgs a) {
  __shared__ int32_t ids[LIST_MAX];
  __shared__ float q[LIST_MAX];
  const uint64_t block = a.block0 + blockIdx.x, row = block / a.parts;
  const Row<T> r(static_cast<T *>(a.dx) + int64_t(row) * a.dx_stride, a.vocab);
  const uint32_t from = uint32_t(block % a.parts) * a.part, to = min(r.pieces(), from + a.part);
  if (from >= to) return;  // (parts are counted for rows that begin anywhere)
  load_list<WAVES>(a, row, ids);
  // (every thread reads back the entries that it has written itself, until the barrier)
  grad_pieces<T, WAVES>(a, row, static_cast<const T *>(a.x) + int64_t(row) * a.stride, r, from, to, a.stats[row], ids, q);
}

int check(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab, const int32_t *ids, const float *lp,
          uint32_t k, int tail, float scale) {
  if (bad_logits(dtype, logits, row_stride, n_rows, vocab, false) || k == 0 || k > LIST_MAX || tail < 0 || tail > 1 ||
      k > vocab || (tail && k >= vocab) || !(scale > 0.0f) || !std::isfinite(scale))
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
  a.c = scale * LOG2E;
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
  *out_bytes = parted_bytes(cut_rows(dtype, n_rows, vocab, true, PARTS_MAX), n_rows);
  return BBPE_OK;
}

int bbpe_distill_loss_backward(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                               const int32_t *d_top_ids, const float *d_top_logprobs, uint32_t top_k, int tail, float scale,
                               const float *d_stats, const float *d_grad, void *d_logits, int64_t dl_stride, void *hip_stream) {
  const int rc = check(dtype, logits, row_stride, n_rows, vocab, d_top_ids, d_top_logprobs, top_k, tail, scale);
  if (rc) return rc;
  if (bad_logits(dtype, d_logits, dl_stride, n_rows, vocab, true) || (n_rows && (!d_stats || !d_grad)) ||
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
      (d_logits && bad_logits(dtype, d_logits, dl_stride, n_rows, vocab, true)))
    return BBPE_E_INVALID_ARG;
  if (n_rows == 0) return BBPE_OK;
  const Cut cut = cut_rows(dtype, n_rows, vocab, true, PARTS_MAX);
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
  const bool grad = d_logits != nullptr;
  with_element(dtype, [&](auto t) {
    typedef decltype(t) T;
    constexpr uint32_t W = ROW_WAVES;
    if (cut.parts > 1) {
      launch(n_rows * cut.parts, tail ? k_distill<T, W, true, true, false> : k_distill<T, W, false, true, false>, ROW_THREADS);
      launch(n_rows, k_distill_join<T>, 64);
    } else if (cut.waves == 1) {
      if (grad) launch(n_rows, tail ? k_distill<T, 1, true, false, true> : k_distill<T, 1, false, false, true>, 64);
      else launch(n_rows, tail ? k_distill<T, 1, true, false, false> : k_distill<T, 1, false, false, false>, 64);
    } else if (grad) {
      launch(n_rows, tail ? k_distill<T, STEP_WAVES, true, false, true> : k_distill<T, STEP_WAVES, false, false, true>, 64 * STEP_WAVES);
    } else {
      launch(n_rows, tail ? k_distill<T, W, true, false, false> : k_distill<T, W, false, false, false>, ROW_THREADS);
    }
  });
  if (hipGetLastError() != hipSuccess) return BBPE_E_HIP;
  if (grad && cut.parts > 1) launch_back(a, dtype, n_rows, st);
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

}  // extern "C"
