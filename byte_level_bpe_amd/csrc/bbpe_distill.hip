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

constexpr uint32_t LIST_MAX = 256;       // listed tokens at most
constexpr uint32_t BIT_WORDS = 1u << 12; // words of 32 tokens in LDS: a stretch of 131,072 at a time

struct DistillArgs {
  const void *x;
  int64_t stride;
  uint64_t row0;
  uint32_t vocab, k, tail;
  float scale, c;
  const int32_t *ids;
  const float *lp;
  float *loss, *lse;
  float4 *stats;
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
__device__ void end_row(const DistillArgs &a, uint64_t row, const T *x, Partial p, const int32_t *ids) {
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
  if (lane) return;
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
  a.loss[row] = float(loss);
  a.lse[row] = bad ? nan : none ? -INFINITY : float(double(high) * a.scale + log_sum);
  a.stats[row] = st;
}

template <typename T, bool TAIL>
__global__ __launch_bounds__(ROW_THREADS) void k_distill(DistillArgs a) {
  typedef Piece<T> P;
  typedef typename P::raw Raw;
  constexpr uint32_t STRETCH = TAIL ? BIT_WORDS * 32 / P::N / ROW_STEP : 1;  // steps between two settings of the bits
  __shared__ Partial sh[ROW_WAVES];
  __shared__ int32_t ids[LIST_MAX];
  __shared__ uint32_t bits[TAIL ? BIT_WORDS : 1];
  const uint64_t row = a.row0 + blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  const Row<const T> r(x, a.vocab);
  const uint32_t tid = threadIdx.x;
  if (tid < a.k) {
    const int32_t id = a.ids[row * a.k + tid];
    ids[tid] = id >= 0 && uint32_t(id) < a.vocab ? id : -1;
  }
  Partial s{-INFINITY, 0.0f, 0.0f};
  float ref = 0.0f;
  const uint32_t steps = (r.pieces() + ROW_STEP - 1) / ROW_STEP;
  for (uint32_t i = 0; i < steps; ++i) {
    if (TAIL && i % STRETCH == 0) {
      const uint32_t from = i * ROW_STEP * P::N;
      __syncthreads();
      for (uint32_t w = tid; w < BIT_WORDS; w += ROW_THREADS) bits[w] = 0;
      __syncthreads();
      const uint32_t place = tid < a.k && ids[tid] >= 0 ? r.lead + uint32_t(ids[tid]) - from : ~0u;
      if (place < BIT_WORDS * 32) atomicOr(&bits[place / 32], 1u << place % 32);
      __syncthreads();
    }
    typename P::val v[ROW_UNROLL];
    float m = -INFINITY;
    Raw raw[ROW_UNROLL];
    r.template load_step<ROW_THREADS>(raw, r.at, i * ROW_STEP + tid, r.pieces());
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      v[u] = values<T>(raw[u]);
      if (TAIL) {
        const uint32_t place = (i % STRETCH * ROW_STEP + u * ROW_THREADS + tid) * P::N;
        const uint32_t mask = bits[place / 32] >> place % 32 & ((1u << P::N) - 1);
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
  s = row_partial<ROW_WAVES>(s, a.c, sh);  // (with a barrier, for the list too)
  if (tid < 64) end_row<T>(a, row, x, s, ids);
}

struct DistillBackArgs {
  const void *x;
  int64_t stride;
  void *dx;
  int64_t dx_stride;
  uint64_t block0;
  uint32_t vocab, k, tail, parts, part;  // parts of a row, and pieces of one
  float scale, c;
  const int32_t *ids;
  const float *lp;
  const float4 *stats;
  const float *grad;
};

// One workgroup a part of a row.  The listed tokens are written once more when
// the part is done, from what was there before (dx may be x): each by one
// thread, or by several with the same value.
template <typename T>
__global__ __launch_bounds__(ROW_THREADS) void k_distill_back(DistillBackArgs a) {
  typedef Piece<T> P;
  __shared__ int32_t ids[LIST_MAX];
  __shared__ float q[LIST_MAX];
  const uint32_t tid = threadIdx.x;
  const uint64_t block = a.block0 + blockIdx.x, row = block / a.parts;
  const T *x = static_cast<const T *>(a.x) + int64_t(row) * a.stride;
  T *dx = static_cast<T *>(a.dx) + int64_t(row) * a.dx_stride;
  const Row<T> r(dx, a.vocab);  // pieces as they are written
  const uint32_t from = uint32_t(block % a.parts) * a.part, to = min(r.pieces(), from + a.part);
  if (from >= to) return;  // (parts are counted for rows that begin anywhere)
  const float4 st = a.stats[row];
  const float g = a.grad[row] * a.scale;
  const bool zero = st.x == -INFINITY || g == 0.0f;
  const float inv = __builtin_amdgcn_exp2f(-st.y * LOG2E);
  const auto weight = [&](float v) { return __builtin_amdgcn_exp2f((v - st.x) * a.c); };
  float before = 0.0f;
  bool mine = false;
  if (tid < a.k) {
    const int32_t id = a.ids[row * a.k + tid];
    const float lp = a.lp[row * a.k + tid];
    const bool there = id >= 0 && uint32_t(id) < a.vocab;
    ids[tid] = there ? id : -1;
    q[tid] = there ? __builtin_amdgcn_exp2f((lp - (a.tail ? 0.0f : st.w)) * LOG2E) : 0.0f;
    mine = there && !zero && (r.lead + uint32_t(id)) / P::N - from < to - from;
    if (mine) before = float(x[id]);
  }
  __syncthreads();
  const float all = g * st.z * inv;
  for (uint32_t p0 = from; p0 < to; p0 += ROW_STEP) {
    typename P::raw raw[ROW_UNROLL];
    if (!zero) r.template load_step<ROW_THREADS>(raw, x - r.lead, p0 + tid, to);
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      const uint32_t p = p0 + u * ROW_THREADS + tid;
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
  if (!mine) return;
  float sum = 0.0f;
  for (uint32_t t = 0; t < a.k; ++t) sum += ids[t] == ids[tid] ? q[t] : 0.0f;
  dx[ids[tid]] = T(g * ((a.tail ? st.w : st.z) * inv * weight(before) - sum));
}

constexpr uint64_t MAX_GROUPS = 1u << 23;  // workgroups of a launch: fewer than 2^32 threads

int check(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab, const int32_t *ids, const float *lp,
          uint32_t k, int tail, float scale) {
  if (bad_logits(dtype, logits, row_stride, n_rows, vocab, false) || k == 0 || k > LIST_MAX || tail < 0 || tail > 1 ||
      k > vocab || (tail && k >= vocab) || !(scale > 0.0f) || !std::isfinite(scale))
    return BBPE_E_INVALID_ARG;
  if ((n_rows && (!ids || !lp)) || ((address(ids) | address(lp)) & 3)) return BBPE_E_INVALID_ARG;
  return BBPE_OK;
}

}  // namespace
}  // namespace bbpe

using namespace bbpe;

extern "C" {

int bbpe_distill_loss_backward(int dtype, const void *logits, int64_t row_stride, uint64_t n_rows, uint32_t vocab,
                               const int32_t *d_top_ids, const float *d_top_logprobs, uint32_t top_k, int tail, float scale,
                               const float *d_stats, const float *d_grad, void *d_logits, int64_t dl_stride, void *hip_stream) {
  const int rc = check(dtype, logits, row_stride, n_rows, vocab, d_top_ids, d_top_logprobs, top_k, tail, scale);
  if (rc) return rc;
  if (bad_logits(dtype, d_logits, dl_stride, n_rows, vocab, true) || (n_rows && (!d_stats || !d_grad)) ||
      (address(d_stats) & 15) || (address(d_grad) & 3))
    return BBPE_E_INVALID_ARG;
  if (n_rows == 0) return BBPE_OK;
  DistillBackArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.dx = d_logits;
  a.dx_stride = dl_stride;
  a.vocab = vocab;
  a.k = top_k;
  a.tail = uint32_t(tail);
  a.scale = scale;
  a.c = scale * LOG2E;
  a.ids = d_top_ids;
  a.lp = d_top_logprobs;
  a.stats = reinterpret_cast<const float4 *>(d_stats);
  a.grad = d_grad;
  a.part = 2 * ROW_STEP;
  a.parts = (most_pieces(dtype, vocab) + a.part - 1) / a.part;
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const uint64_t blocks = n_rows * a.parts;
  for (; a.block0 < blocks; a.block0 += MAX_GROUPS)
    with_element(dtype, [&](auto t) {
      k_distill_back<decltype(t)><<<uint32_t(std::min(blocks - a.block0, MAX_GROUPS)), ROW_THREADS, 0, st>>>(a);
    });
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

int bbpe_distill_loss_workspace_bytes(int dtype, uint64_t n_rows, uint32_t vocab, uint64_t *out_bytes) {
  if (!out_bytes || bad_sizes(dtype, n_rows, vocab)) return BBPE_E_INVALID_ARG;
  *out_bytes = 0;
  return BBPE_OK;
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
  DistillArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.vocab = vocab;
  a.k = top_k;
  a.tail = uint32_t(tail);
  a.scale = scale;
  a.c = scale * LOG2E;
  a.ids = d_top_ids;
  a.lp = d_top_logprobs;
  a.loss = d_loss;
  a.lse = d_lse;
  a.stats = reinterpret_cast<float4 *>(d_stats);
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  for (; a.row0 < n_rows; a.row0 += MAX_GROUPS)
    with_element(dtype, [&](auto t) {
      const uint32_t grid = uint32_t(std::min(n_rows - a.row0, MAX_GROUPS));
      if (tail) k_distill<decltype(t), true><<<grid, ROW_THREADS, 0, st>>>(a);
      else k_distill<decltype(t), false><<<grid, ROW_THREADS, 0, st>>>(a);
    });
  if (hipGetLastError() != hipSuccess) return BBPE_E_HIP;
  return d_logits ? bbpe_distill_loss_backward(dtype, logits, row_stride, n_rows, vocab, d_top_ids, d_top_logprobs, top_k, tail,
                                               scale, d_stats, d_weights, d_logits, dl_stride, hip_stream)
                  : BBPE_OK;
}

}  // extern "C"
