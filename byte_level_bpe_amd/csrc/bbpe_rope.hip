// Per-head RMS norm of queries and keys with the position rotation, forward
// and backward.
//
// One row is a head of a token, x[0..D).  Forward: rstd = 1/sqrt(mean x^2 +
// eps), y = x * rstd * w, and each of the first R/2 pairs of y turns by
// a_j = position * inv_freq[j].  Backward, g the gradient of the turned row:
// dy = g turned back, h = dy * w, dx = rstd * (h - n * mean(h * n)) with
// n = x * rstd, and dw = sum over rows of dy * n.
//
// Bound by HBM: every row is read once and written once (backward: two reads,
// one write) and the arithmetic is some ten operations an element.  A lane
// holds 16 elements of a row as two runs of eight, chosen so that both
// elements of a pair are in one lane: no exchange but the row's sum over its
// D/16 lanes.  A workgroup takes a token, with its R/2 sines and cosines made
// once, by R/2 lanes, for all of the token's heads.
//
// Measured on an MI355X, bfloat16, 32 + 8 heads of 128: forward into a cache,
// 16,384 tokens, 93 us (403 MB, 4.3 TB/s; a copy reaches 4.8); one token a
// workgroup and many workgroups hide the loads better than fewer that load
// ahead (121 to 152 us with 512 to 1,024 workgroups).  Backward, 8,192 tokens,
// 65 us and 5 for the weights' sums (252 MB): its sums of the weights'
// gradients live in registers, which leaves room for two workgroups a compute
// unit, so it loads ahead.  8 tokens forward: 4.7 us in the kernel, 5.4 a call.
// As many elements in other heads, calls queued, forward without a cache and
// backward in TB/s: 32 + 8 of 128 4.5 and 3.6; 64 + 8 of 128, a workgroup's rows in
// two rounds, 4.6 and 3.4; 40 + 40 of 128 4.0 and 3.8; 16 + 16 of 256 5.0 and
// 4.5; 64 + 64 of 64 5.2 and 4.7.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/bbpe.h"
#include "bbpe_float.h"

namespace bbpe {
namespace {

// Workgroups of the backward pass at most: two a compute unit, as many as its
// registers leave room for (1,024: 74 us instead of 67 for 8,192 tokens of 40 heads).
constexpr uint32_t QK_GRID = 512;
constexpr uint32_t QK_MAX_BLOCK = 512;
constexpr uint32_t QK_BATCH = 4;        // tokens of a batch of the backward pass at most
constexpr uint64_t QK_MAX_TOKENS = 1u << 22;  // tokens of one forward launch

struct Rows {
  void *p;
  int64_t ts, hs;  // token and head strides in elements
  uint32_t vec;    // every row 16-byte aligned
};

struct QkArgs {
  Rows q, k, v, qo, ko;       // inputs and outputs (backward: the rows, and their gradients)
  Rows gq, gk;                // backward: gradients of the turned rows
  const void *wq, *wk;        // null: ones
  const int32_t *pos;
  const float *inv_freq;
  const int64_t *slots;       // null: no cache
  char *kc, *vc;
  int64_t page_stride, head_stride, token_stride;
  uint64_t n_pages;
  uint32_t page_shift, page;  // page_shift 32: the page size is no power of two
  uint64_t n_tok, tok0;       // forward: the launch's first token
  uint32_t hq, hk, dim, rot;
  uint32_t lanes;             // lanes of a row, a power of two >= dim / 16
  float eps;
  uint32_t batch;             // backward: tokens of a batch
  float *part;                // backward: [workgroups][2][dim] sums of the weights' gradients
};

// sin and cos of position * inv_freq.  The product and its reduction to a
// fraction of a turn are in 64 bits: at position 10^6 a 32-bit product is off
// by a sixteenth of a radian.  The fraction (|t| <= 1/2) goes on in 32.
__device__ __forceinline__ float2 turn_of(int32_t position, float inv_freq) {
  double t = double(position) * double(inv_freq) * 0.15915494309189533577;  // 1 / (2 pi)
  t -= __builtin_rint(t);
  float s, c;
  sincospif(2.0f * float(t), &s, &c);
  return make_float2(c, s);
}

// Where a lane's two runs of eight begin in the row.  Half pairs: 8c and R/2 +
// 8c turn against each other; past the rotated lanes, and for neighbouring
// pairs, the lane's 16 elements are consecutive.
template <bool INTER>
__device__ __forceinline__ void runs_of(uint32_t c, uint32_t rot, uint32_t &d0, uint32_t &d1) {
  d0 = 16 * c;
  d1 = d0 + 8;
  if (!INTER && 16 * c < rot) {
    d0 = 8 * c;
    d1 = rot / 2 + 8 * c;
  }
}

// (a, b): the lane's two runs; turned by +a_j, or back by -a_j.
template <bool INTER, bool BACK>
__device__ __forceinline__ void turn(f32x8 &a, f32x8 &b, const float2 *cs, uint32_t c) {
  if (INTER) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = cs[8 * c + j], w = cs[8 * c + 4 + j];
      const float us = BACK ? -u.y : u.y, ws = BACK ? -w.y : w.y;
      const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
      a[2 * j] = a0 * u.x - a1 * us;
      a[2 * j + 1] = a1 * u.x + a0 * us;
      b[2 * j] = b0 * w.x - b1 * ws;
      b[2 * j + 1] = b1 * w.x + b0 * ws;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 u = cs[8 * c + j];
      const float us = BACK ? -u.y : u.y, a0 = a[j], b0 = b[j];
      a[j] = a0 * u.x - b0 * us;
      b[j] = b0 * u.x + a0 * us;
    }
  }
}

// Sum over the row's lanes (a power of two of neighbours), in all of them.
__device__ __forceinline__ float row_sum(float v, uint32_t lanes) {
  for (uint32_t d = 1; d < lanes; d <<= 1) v += __shfl_xor(v, int(d), 64);
  return v;
}
__device__ __forceinline__ float sum_of(f32x8 a) {
  return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
}

template <typename T, bool INTER>
__global__ __launch_bounds__(QK_MAX_BLOCK) void k_qk_norm_rope(QkArgs a) {
  __shared__ float2 cs[128];
  const uint64_t tok = a.tok0 + blockIdx.x;
  const uint32_t c = threadIdx.x & (a.lanes - 1), group = threadIdx.x / a.lanes, groups = blockDim.x / a.lanes;
  const bool in_row = 16 * c < a.dim;
  const bool cached = a.slots != nullptr;
  const uint32_t normed = a.hq + a.hk, rows = normed + (cached ? a.hk : 0);
  uint32_t d0, d1;
  runs_of<INTER>(c, a.rot, d0, d1);
  char *kc = nullptr, *vc = nullptr;  // the token's place in the cache, null: none
  if (cached) {
    const int64_t slot = a.slots[tok];
    const uint64_t page = a.page_shift < 32 ? uint64_t(slot) >> a.page_shift : uint64_t(slot) / a.page;
    if (slot >= 0 && page < a.n_pages) {
      const int64_t at = (int64_t(page) * a.page_stride + (slot - int64_t(page) * a.page) * a.token_stride) * int64_t(sizeof(T));
      kc = a.kc + at;
      vc = a.vc + at;
    }
  }
  bool made = a.rot == 0;
  for (uint32_t r = group;; r += groups) {
    // every thread makes the first round, for the barrier after the turns
    typename Vec8<T>::type ra{}, rb{};
    const bool live = r < rows && in_row;
    const bool is_q = r < a.hq, is_v = r >= normed;
    const Rows &src = is_q ? a.q : is_v ? a.v : a.k;
    const uint32_t h = is_q ? r : is_v ? r - normed : r - a.hq;
    if (live) {
      const T *x = static_cast<const T *>(src.p) + int64_t(tok) * src.ts + int64_t(h) * src.hs;
      ra = load8_raw(x + d0, src.vec);
      rb = load8_raw(x + d1, src.vec);
    }
    if (!made) {
      for (uint32_t j = threadIdx.x; j < a.rot / 2; j += blockDim.x) cs[j] = turn_of(a.pos[tok], a.inv_freq[j]);
      __syncthreads();
      made = true;
    }
    f32x8 xa = to_float<T>(ra), xb = to_float<T>(rb);
    const float ss = row_sum(sum_of(xa * xa) + sum_of(xb * xb), a.lanes);
    if (live) {
      if (is_v) {
        if (vc) {
          T *o = reinterpret_cast<T *>(vc) + int64_t(h) * a.head_stride;
          store8_raw(o + d0, ra, true);
          store8_raw(o + d1, rb, true);
        }
      } else {
        const float rstd = 1.0f / sqrtf(ss / float(a.dim) + a.eps);
        const T *w = static_cast<const T *>(is_q ? a.wq : a.wk);
        f32x8 wa = 1.0f, wb = 1.0f;
        if (w) {
          wa = to_float<T>(load8_raw(w + d0, true));
          wb = to_float<T>(load8_raw(w + d1, true));
        }
        xa = xa * rstd * wa;
        xb = xb * rstd * wb;
        if (16 * c < a.rot) turn<INTER, false>(xa, xb, cs, c);
        const typename Vec8<T>::type oa = from_float<T>(xa), ob = from_float<T>(xb);
        const Rows &dst = is_q ? a.qo : a.ko;
        if (dst.p) {
          T *o = static_cast<T *>(dst.p) + int64_t(tok) * dst.ts + int64_t(h) * dst.hs;
          store8_raw(o + d0, oa, dst.vec);
          store8_raw(o + d1, ob, dst.vec);
        }
        if (!is_q && kc) {
          T *o = reinterpret_cast<T *>(kc) + int64_t(h) * a.head_stride;
          store8_raw(o + d0, oa, true);
          store8_raw(o + d1, ob, true);
        }
      }
    }
    if (r - group + groups >= rows) break;
  }
}

// Backward.  Workgroup b takes batches b, b + gridDim, ... of a.batch tokens,
// whose turns are made at once, a barrier apart from their use and one batch
// ahead.  A lane's columns are the same in all of its rows, so the weights'
// gradients add up in registers (queries' and keys' apart), then over the
// workgroup's groups in LDS, and over workgroups in k_qk_norm_weights: every
// order is fixed by the sizes.  ONE: a token's rows fit the workgroup, so that
// a lane keeps to one head, and its next token's rows are loaded before the
// present one's are worked on.
template <typename T, bool INTER, bool ONE>
__global__ __launch_bounds__(QK_MAX_BLOCK) void k_qk_norm_rope_back(QkArgs a) {
  typedef typename Vec8<T>::type V;
  __shared__ float2 cs[2][QK_BATCH][128];
  extern __shared__ float sums[];  // [groups][dim]
  const uint32_t c = threadIdx.x & (a.lanes - 1), group = threadIdx.x / a.lanes, groups = blockDim.x / a.lanes;
  const bool in_row = 16 * c < a.dim;
  const uint32_t rows = a.hq + a.hk;
  uint32_t d0, d1;
  runs_of<INTER>(c, a.rot, d0, d1);
  f32x8 qa = 0.0f, qb = 0.0f, ka = 0.0f, kb = 0.0f;
  struct Raw {
    V xa, xb, ga, gb;
  };
  const auto load = [&](uint64_t tok, uint32_t r) {
    Raw v{};
    if (tok < a.n_tok && r < rows && in_row) {
      const bool is_q = r < a.hq;
      const uint32_t h = is_q ? r : r - a.hq;
      const Rows &src = is_q ? a.q : a.k, &up = is_q ? a.gq : a.gk;
      const T *x = static_cast<const T *>(src.p) + int64_t(tok) * src.ts + int64_t(h) * src.hs;
      const T *g = static_cast<const T *>(up.p) + int64_t(tok) * up.ts + int64_t(h) * up.hs;
      v.xa = load8_raw(x + d0, src.vec);
      v.xb = load8_raw(x + d1, src.vec);
      v.ga = load8_raw(g + d0, up.vec);
      v.gb = load8_raw(g + d1, up.vec);
    }
    return v;
  };
  f32x8 wa = 1.0f, wb = 1.0f;
  const auto weights = [&](uint32_t r) {
    const T *w = static_cast<const T *>(r < a.hq ? a.wq : a.wk);
    wa = wb = 1.0f;
    if (w && in_row) {
      wa = to_float<T>(load8_raw(w + d0, true));
      wb = to_float<T>(load8_raw(w + d1, true));
    }
  };
  const auto work = [&](const Raw &v, uint64_t tok, uint32_t r, const float2 *turns) {
    const bool live = r < rows && in_row, is_q = r < a.hq;
    f32x8 xa = to_float<T>(v.xa), xb = to_float<T>(v.xb), ga = to_float<T>(v.ga), gb = to_float<T>(v.gb);
    if (16 * c < a.rot) turn<INTER, true>(ga, gb, turns, c);
    const f32x8 ha = ga * wa, hb = gb * wb;
    const float ss = row_sum(sum_of(xa * xa) + sum_of(xb * xb), a.lanes);
    const float rstd = 1.0f / sqrtf(ss / float(a.dim) + a.eps);
    const f32x8 na = xa * rstd, nb = xb * rstd;
    const float mean = row_sum(sum_of(ha * na) + sum_of(hb * nb), a.lanes) / float(a.dim);
    if (!live) return;
    const uint32_t h = is_q ? r : r - a.hq;
    const Rows &dst = is_q ? a.qo : a.ko;
    T *o = static_cast<T *>(dst.p) + int64_t(tok) * dst.ts + int64_t(h) * dst.hs;
    store8_raw(o + d0, from_float<T>((ha - na * mean) * rstd), dst.vec);
    store8_raw(o + d1, from_float<T>((hb - nb * mean) * rstd), dst.vec);
    if (ONE || is_q) {
      qa += ga * na;
      qb += gb * nb;
    } else {
      ka += ga * na;
      kb += gb * nb;
    }
  };
  const uint64_t batches = (a.n_tok + a.batch - 1) / a.batch;
  const auto make = [&](uint64_t b, uint32_t buf) {
    if (b >= batches) return;
    for (uint32_t j = threadIdx.x; j < a.rot / 2 * a.batch; j += blockDim.x) {
      const uint32_t t = j / (a.rot / 2), e = j - t * (a.rot / 2);
      const uint64_t tok = b * a.batch + t;
      if (tok < a.n_tok) cs[buf][t][e] = turn_of(a.pos[tok], a.inv_freq[e]);
    }
  };
  uint32_t buf = 0;
  Raw next{};
  if (ONE) {
    weights(group);
    next = load(uint64_t(blockIdx.x) * a.batch, group);
  }
  make(blockIdx.x, 0);
  for (uint64_t b = blockIdx.x; b < batches; b += gridDim.x, buf ^= 1) {
    __syncthreads();  // this batch's turns are made, and the other buffer's are no longer read
    make(b + gridDim.x, buf ^ 1);
    for (uint32_t t = 0; t < a.batch; ++t) {
      const uint64_t tok = b * a.batch + t;
      if (tok >= a.n_tok) break;
      if (ONE) {
        const Raw v = next;
        next = load(t + 1 < a.batch ? tok + 1 : (b + gridDim.x) * a.batch, group);
        work(v, tok, group, cs[buf][t]);
      } else {
        for (uint32_t r0 = 0; r0 < rows; r0 += groups) {
          weights(r0 + group);
          work(load(tok, r0 + group), tok, r0 + group, cs[buf][t]);
        }
      }
    }
  }
  if (!a.part) return;
  // ONE: groups below hq hold queries' sums, those after them keys', in one round
  for (int which = 0; which < (ONE ? 1 : 2); ++which) {
    __syncthreads();
    if (in_row) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sums[group * a.dim + d0 + j] = which ? ka[j] : qa[j];
        sums[group * a.dim + d1 + j] = which ? kb[j] : qb[j];
      }
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < (ONE ? 2 : 1) * a.dim; e += blockDim.x) {
      const uint32_t keys = ONE ? e / a.dim : uint32_t(which), d = ONE ? e - keys * a.dim : e;
      const uint32_t from = ONE && keys ? a.hq : 0, to = ONE ? (keys ? rows : a.hq) : groups;
      float s = 0.0f;
      for (uint32_t g = from; g < to; ++g) s += sums[g * a.dim + d];
      a.part[(uint64_t(blockIdx.x) * 2 + keys) * a.dim + d] = s;
    }
  }
}

// Sums the workgroups' parts: one workgroup for 16 columns of one weight, 64
// threads a column, so that 512 parts are 8 loads under way at once.
__global__ __launch_bounds__(1024) void k_qk_norm_weights(const float *part, uint32_t n, uint32_t dim, float *dwq, float *dwk) {
  __shared__ float sh[64][17];
  const uint32_t e = threadIdx.x & 15, d = blockIdx.x * 16 + e, g = threadIdx.x >> 4, which = blockIdx.y;
  float s = 0.0f;
  if (d < dim) {
    float v[QK_GRID / 64];
#pragma unroll
    for (uint32_t j = 0; j < QK_GRID / 64; ++j) v[j] = g + 64 * j < n ? part[(uint64_t(g + 64 * j) * 2 + which) * dim + d] : 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < QK_GRID / 64; ++j) s += v[j];
  }
  sh[g][e] = s;
  for (uint32_t half = 32; half; half /= 2) {
    __syncthreads();
    if (g < half) sh[g][e] += sh[g + half][e];
  }
  float *out = which ? dwk : dwq;
  if (g == 0 && d < dim && out) out[d] = sh[0][e];
}

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
uint64_t size_of(int dtype) { return dtype == BBPE_F32 ? 4 : 2; }

// 16-byte aligned rows, for vector loads and stores
Rows rows_of(const void *p, int64_t ts, int64_t hs, int dtype) {
  const int64_t e = int64_t(size_of(dtype));
  const bool vec = (addr(p) & 15) == 0 && ((ts * e) & 15) == 0 && ((hs * e) & 15) == 0;
  return Rows{const_cast<void *>(p), ts, hs, vec ? 1u : 0u};
}

bool bad_rows(const void *p, int dtype) { return (addr(p) & (size_of(dtype) - 1)) != 0; }

// What forward and backward ask of their sizes alike.
int check_sizes(int dtype, uint64_t n_tok, uint32_t hq, uint32_t hk, uint32_t dim, uint32_t rot, int inter, float eps,
                const void *wq, const void *wk, const int32_t *pos, const float *inv_freq) {
  if (dtype < BBPE_BF16 || dtype > BBPE_F32 || inter < 0 || inter > 1 || !(eps >= 0.0f)) return BBPE_E_INVALID_ARG;
  if (dim == 0 || dim > 256 || dim % 16 || rot > dim || rot % 16 || hq > 4096 || hk > 4096 || hq + hk == 0 ||
      n_tok > 0x7FFFFFFFull)
    return BBPE_E_INVALID_ARG;
  if ((addr(wq) & 15) || (addr(wk) & 15) || (rot && (!inv_freq || (addr(inv_freq) & 3))) ||
      (n_tok && rot && (!pos || (addr(pos) & 3))))
    return BBPE_E_INVALID_ARG;
  return BBPE_OK;
}

void shape(QkArgs &a, uint32_t rows, uint32_t &block) {
  a.lanes = 1;
  while (a.lanes * 16 < a.dim) a.lanes *= 2;
  // all rows of a token in one round if they fit, else in rounds of one block
  block = std::min(QK_MAX_BLOCK, (rows * a.lanes + 63) / 64 * 64);
}

// Calls f with the kernel's template arguments.
template <typename F>
void with_type(int dtype, int inter, F f) {
  if (dtype == BBPE_BF16) inter ? f((__bf16)0, std::true_type{}) : f((__bf16)0, std::false_type{});
  else if (dtype == BBPE_F16) inter ? f((_Float16)0, std::true_type{}) : f((_Float16)0, std::false_type{});
  else inter ? f(0.0f, std::true_type{}) : f(0.0f, std::false_type{});
}

}  // namespace
}  // namespace bbpe

using namespace bbpe;

extern "C" {

int bbpe_qk_norm_rope(int dtype, uint64_t n_tokens, uint32_t n_q_heads, uint32_t n_kv_heads,
                      uint32_t head_dim, uint32_t rot_dim, int interleaved, float eps,
                      const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts,
                      int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs, const void *w_q,
                      const void *w_k, const int32_t *d_positions, const float *d_inv_freq,
                      void *q_out, int64_t qo_ts, int64_t qo_hs, void *k_out, int64_t ko_ts,
                      int64_t ko_hs, const bbpe_paged_cache *cache, const int64_t *d_slots,
                      void *hip_stream) {
  const int rc = check_sizes(dtype, n_tokens, n_q_heads, n_kv_heads, head_dim, rot_dim, interleaved, eps, w_q, w_k,
                             d_positions, d_inv_freq);
  if (rc) return rc;
  if ((cache == nullptr) != (d_slots == nullptr)) return BBPE_E_INVALID_ARG;
  if (n_tokens && ((n_q_heads && (!q || !q_out)) || (n_kv_heads && (!k || (!k_out && !cache) || (cache && !v)))))
    return BBPE_E_INVALID_ARG;
  if (bad_rows(q, dtype) || bad_rows(k, dtype) || bad_rows(v, dtype) || bad_rows(q_out, dtype) || bad_rows(k_out, dtype) ||
      (addr(d_slots) & 7))
    return BBPE_E_INVALID_ARG;
  QkArgs a{};
  if (cache) {
    if (cache->dtype != dtype || dtype == BBPE_F32 || cache->head_dim != head_dim || cache->n_kv_heads != n_kv_heads ||
        cache->page_size == 0 || cache->page_size > (1u << 30) || !cache->k || !cache->v ||
        ((addr(cache->k) | addr(cache->v)) & 15) || cache->n_pages > 0x7FFFFFFFull ||
        ((cache->page_stride | cache->head_stride | cache->token_stride) & 7))
      return BBPE_E_INVALID_ARG;
    a.kc = static_cast<char *>(cache->k);
    a.vc = static_cast<char *>(cache->v);
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.token_stride = cache->token_stride;
    a.n_pages = cache->n_pages;
    a.page = cache->page_size;
    a.page_shift = (a.page & (a.page - 1)) == 0 ? uint32_t(__builtin_ctz(a.page)) : 32u;
    a.slots = d_slots;
  }
  if (n_tokens == 0) return BBPE_OK;
  a.q = rows_of(q, q_ts, q_hs, dtype);
  a.k = rows_of(k, k_ts, k_hs, dtype);
  a.v = rows_of(v, v_ts, v_hs, dtype);
  a.qo = rows_of(q_out, qo_ts, qo_hs, dtype);
  a.ko = rows_of(k_out, ko_ts, ko_hs, dtype);
  a.wq = w_q;
  a.wk = w_k;
  a.pos = d_positions;
  a.inv_freq = d_inv_freq;
  a.n_tok = n_tokens;
  a.hq = n_q_heads;
  a.hk = n_kv_heads;
  a.dim = head_dim;
  a.rot = rot_dim;
  a.eps = eps;
  uint32_t block;
  shape(a, a.hq + a.hk + (cache ? a.hk : 0), block);
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  // a launch holds fewer than 2^32 threads
  for (; a.tok0 < n_tokens; a.tok0 += QK_MAX_TOKENS)
    with_type(dtype, interleaved, [&](auto t, auto inter) {
      k_qk_norm_rope<decltype(t), decltype(inter)::value>
          <<<uint32_t(std::min(n_tokens - a.tok0, QK_MAX_TOKENS)), block, 0, st>>>(a);
    });
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

int bbpe_qk_norm_rope_backward_workspace_bytes(uint64_t n_tokens, uint32_t head_dim, uint64_t *out_bytes) {
  if (!out_bytes || head_dim > 256) return BBPE_E_INVALID_ARG;
  *out_bytes = std::min<uint64_t>(n_tokens, QK_GRID) * 2 * head_dim * sizeof(float);
  return BBPE_OK;
}

int bbpe_qk_norm_rope_backward(int dtype, uint64_t n_tokens, uint32_t n_q_heads,
                               uint32_t n_kv_heads, uint32_t head_dim, uint32_t rot_dim,
                               int interleaved, float eps, const void *g_q, int64_t gq_ts,
                               int64_t gq_hs, const void *g_k, int64_t gk_ts, int64_t gk_hs,
                               const void *q, int64_t q_ts, int64_t q_hs, const void *k,
                               int64_t k_ts, int64_t k_hs, const void *w_q, const void *w_k,
                               const int32_t *d_positions, const float *d_inv_freq, void *d_q,
                               int64_t dq_ts, int64_t dq_hs, void *d_k, int64_t dk_ts,
                               int64_t dk_hs, float *d_wq, float *d_wk, void *d_workspace,
                               uint64_t workspace_bytes, void *hip_stream) {
  const int rc = check_sizes(dtype, n_tokens, n_q_heads, n_kv_heads, head_dim, rot_dim, interleaved, eps, w_q, w_k,
                             d_positions, d_inv_freq);
  if (rc) return rc;
  if (n_tokens && ((n_q_heads && (!q || !g_q || !d_q)) || (n_kv_heads && (!k || !g_k || !d_k)))) return BBPE_E_INVALID_ARG;
  if (bad_rows(q, dtype) || bad_rows(k, dtype) || bad_rows(g_q, dtype) || bad_rows(g_k, dtype) || bad_rows(d_q, dtype) ||
      bad_rows(d_k, dtype) || (addr(d_wq) & 3) || (addr(d_wk) & 3))
    return BBPE_E_INVALID_ARG;
  // few tokens: one a workgroup; more: up to four in a row
  const uint32_t batch = uint32_t(std::min<uint64_t>(QK_BATCH, (n_tokens + QK_GRID - 1) / QK_GRID));
  const uint32_t grid = batch ? uint32_t(std::min<uint64_t>((n_tokens + batch - 1) / batch, QK_GRID)) : 0;
  const bool weights = d_wq || d_wk;
  if (weights && grid &&
      (!d_workspace || (addr(d_workspace) & 255) || workspace_bytes < uint64_t(grid) * 2 * head_dim * sizeof(float)))
    return BBPE_E_WORKSPACE;
  QkArgs a{};
  a.gq = rows_of(g_q, gq_ts, gq_hs, dtype);
  a.gk = rows_of(g_k, gk_ts, gk_hs, dtype);
  a.q = rows_of(q, q_ts, q_hs, dtype);
  a.k = rows_of(k, k_ts, k_hs, dtype);
  a.qo = rows_of(d_q, dq_ts, dq_hs, dtype);
  a.ko = rows_of(d_k, dk_ts, dk_hs, dtype);
  a.wq = w_q;
  a.wk = w_k;
  a.pos = d_positions;
  a.inv_freq = d_inv_freq;
  a.n_tok = n_tokens;
  a.hq = n_q_heads;
  a.hk = n_kv_heads;
  a.dim = head_dim;
  a.rot = rot_dim;
  a.eps = eps;
  a.part = weights ? static_cast<float *>(d_workspace) : nullptr;
  a.batch = batch;
  uint32_t block;
  shape(a, a.hq + a.hk, block);
  const bool one = (a.hq + a.hk) * a.lanes <= block;
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  if (grid)
    with_type(dtype, interleaved, [&](auto t, auto inter) {
      const size_t lds = size_t(block / a.lanes) * a.dim * sizeof(float);
      if (one) k_qk_norm_rope_back<decltype(t), decltype(inter)::value, true><<<grid, block, lds, st>>>(a);
      else k_qk_norm_rope_back<decltype(t), decltype(inter)::value, false><<<grid, block, lds, st>>>(a);
    });
  if (weights) k_qk_norm_weights<<<dim3((a.dim + 15) / 16, 2), 1024, 0, st>>>(a.part, grid, a.dim, d_wq, d_wk);
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

}  // extern "C"
