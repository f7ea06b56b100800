// Attention of new tokens (a tree of drafts, a chain, one token) over a paged
// key/value cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp2(s_ij - m_i),
//   s_ij = scale * log2(e) * q_i . k_j  over the keys j that row i sees.
//
// Rows.  The query heads that share a key/value head are rows of one product,
// M of them a row tile: the request's rows one after the other, or, in a chain,
// where a tile ends with its last token's key, a power of two of whole tokens.
//
// Split.  A unit is one row tile times KT keys.  For every key/value head the
// units of all requests, row tile after row tile, are laid in one line and cut
// into equal runs, one a workgroup: long and short requests, few and many rows
// keep the card equally busy, and no length has to be known on the host.  A
// row tile cut by a run's end leaves its parts (sums relative to their own
// maximum) in the workspace, and k_attn_join adds them in order: which parts
// there are depends on the lengths alone.
//
// Product.  Transposed, so that nothing moves between lanes: S^T = K Q^T has a
// row's scores in one column of lanes (4 lanes, 8 keys each, of every 32),
// which is just how the second product, O^T = V^T P^T, reads P.  K's fragment
// is 16 bytes of one key a lane.  V's needs eight keys of one element: a lane
// loads D/16 elements of eight keys and turns that block over in registers
// (one byte permute for two elements).  In k_attn_rows, for few rows, keys and
// values go from HBM to registers without a stop in LDS, and the waves join at
// the end of a segment; in k_attn_tiles, for many, they are shared in LDS.
//
// Rounding.  Scores, maxima, sums and parts are 32-bit.  The weights are rounded
// once to the cache's type, the second product's operand: the mean error against
// 64 bits grows by 1.1 (one token) to 1.4 times over 32 bits and one rounding at
// the end.  The sums that divide are the weights' before that, as d_lse needs
// them; dividing by the rounded weights' sums is 1 to 3% nearer and takes 8% more
// time (trees 177 -> 192 us, 100 drafts on 131,001 keys 210 -> 227, prompts 124
// -> 134), and weights in two terms would double the second product.  A weight
// rounded to zero times a visible infinity is NaN.
//
// Measured on an MI355X, bfloat16, 8 key/value heads of 128 (a copy of the card's
// memory runs at 4.8 TB/s, a large matrix product at 1,140 to 1,380 TFLOP/s):
// single tokens are bound by HBM: 128 requests of one on 64 to 32,768 keys, 480 us,
// 5.8 TB/s read.  Many rows are bound by the matrix cores and the softmax's
// arithmetic next to them: 32 trees of 64 drafts on 16,384 keys, 610 us, 900
// TFLOP/s; a prompt of 8,192 tokens, 560 us, 980 TFLOP/s; heads of 64, where a
// score costs as much softmax for half the product, 700.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/bbpe.h"
#include "bbpe_device.h"
#include "bbpe_float.h"

namespace bbpe {
namespace {

constexpr uint32_t AT_BLOCK = 256, AT_WAVES = 4;
constexpr uint32_t AT_REQ = 1024;    // requests of one launch (their units' sums lie in LDS)
constexpr uint32_t AT_TILE = 32;     // keys a wave takes at once
constexpr uint32_t AT_KT_LOG = 7;    // log2 of a unit's keys (AT_WAVES tiles)
// Units that stand for what a row tile costs k_attn_tiles besides its keys.
// None: 765 us for a prompt of 8,192 tokens, as the runs of many short row
// tiles end last; 2: 676, 4: 608, 8: 608.
constexpr uint32_t AT_HEAD = 4;
// Units of keys of the longest row tiles that are never cut, in k_attn_tiles and
// k_attn_rows (74 prompts of 95 to 120 tokens, most row tiles cut by a run's end:
// 72 us, none cut: 55).
constexpr uint32_t AT_WHOLE = 5, AT_ROWS_WHOLE = 3;
constexpr uint32_t AT_RUNS = 512;    // workgroups of a launch, over all heads

// Rows that a workgroup of k_attn_join takes.
constexpr uint32_t join_rows(uint32_t m, uint32_t dim) { return m <= 32 ? 1 : 2 * (AT_BLOCK / (dim / 4)); }

struct AttnArgs {
  const void *q;
  int64_t q_ts, q_hs;
  const char *kc, *vc;
  int64_t page_stride, head_stride, token_stride;
  uint64_t n_pages;
  uint32_t page_shift;
  const int32_t *table;
  uint64_t table_stride;
  uint32_t cap;            // keys that a table row can hold
  const int64_t *q_off;
  const int32_t *ctx;
  uint32_t n_req;
  const uint64_t *mask;    // null: a chain
  uint32_t words;
  float scale2;            // |scale| * log2(e)
  uint32_t flip;           // a negative scale: the queries' signs are flipped
  void *out;
  int64_t out_ts, out_hs;
  float *lse;
  uint64_t n_tok;
  uint32_t hq, hk, grp;
  uint32_t tok_log;        // a chain: log2 of a row tile's tokens
  uint32_t stride;         // rows of a row tile: M with masks, whole tokens in a chain
  uint32_t runs;           // workgroups of one head
  uint32_t q_vec, out_vec; // rows 16-byte aligned
  uint32_t *meta;          // [hk][runs][4]: the row tile that begins in a run and ends in a later one
  const uint32_t *after;   // a launch behind others: not 0 where an earlier one met broken offsets
  uint32_t *broken;        // a launch before others: what the next one reads there
  float *part;             // [hk][runs][2][M][D + 2]: its parts
};

// One request's lengths, as the kernels use them.
struct Lengths {
  bool ok;        // offsets that can be followed
  int64_t first;  // its first token
  uint32_t n;     // new tokens
  uint32_t ctx;   // context; past the table's row: the row's keys
  uint32_t klen;  // keys in all, within the table's row
};
__device__ __forceinline__ Lengths lengths_of(const AttnArgs &a, uint32_t r) {
  Lengths L;
  const int64_t lo = a.q_off[r], hi = a.q_off[r + 1];
  L.ok = lo >= 0 && hi >= lo && uint64_t(hi) <= a.n_tok;
  L.first = lo;
  L.n = L.ok ? uint32_t(hi - lo) : 0;
  const int32_t c = max(a.ctx[r], 0);
  L.ctx = uint32_t(c);
  L.klen = uint32_t(min(int64_t(c) + L.n, int64_t(a.cap)));
  return L;
}

// sum over j = 1..n of ceil(j / 2^q)
__device__ __forceinline__ uint64_t ceil_sum(uint64_t n, uint32_t q) {
  const uint64_t a = n >> q, b = n & ((uint64_t(1) << q) - 1);
  return ((a * (a + 1) / 2) << q) + b * (a + 1);
}

// Units of a request's first t row tiles.  Masks: every row tile spans all
// keys.  A chain: tile i ends at key ctx + (i + 1) * tokens, tokens = 2^tok_log.
template <uint32_t KT_LOG>
__device__ __forceinline__ uint64_t units_before(const AttnArgs &a, const Lengths &L, uint32_t t) {
  constexpr uint32_t KT = 1u << KT_LOG;
  // (a request whose tokens pass the table's row: as with masks)
  if (a.mask || uint64_t(L.ctx) + L.n > a.cap) return uint64_t(t) * ((L.klen + KT - 1) >> KT_LOG);
  const uint32_t whole = L.ctx >> KT_LOG, rest = L.ctx & (KT - 1);
  if (a.tok_log <= KT_LOG) {
    const uint32_t s = (rest + (1u << a.tok_log) - 1) >> a.tok_log, q = KT_LOG - a.tok_log;
    return uint64_t(t) * whole + ceil_sum(s + t, q) - ceil_sum(s, q);
  }
  const uint64_t steps = uint64_t(t) * (t + 1) / 2;
  return uint64_t(t) * (whole + (rest ? 1 : 0)) + (steps << (a.tok_log - KT_LOG));
}
__device__ __forceinline__ uint32_t row_tiles(const AttnArgs &a, uint32_t n) {
  return (n * a.grp + a.stride - 1) / a.stride;
}

// The requests in line: sums of their units up to and with each, in a wave's
// lanes, with their lengths, for up to 64 requests, else in LDS.
struct Line {
  uint64_t total, incl;
  uint64_t per;    // units of a run
  uint32_t head;   // units of every row tile that stand for what it costs besides its keys
  uint32_t whole;  // row tiles of up to so many units are not cut
  Lengths L;
};
// (a 64-bit division takes some hundred instructions)
__device__ __forceinline__ uint64_t divide_up(uint64_t total, uint32_t runs) {
  const uint64_t x = total + runs - 1;
  return x >> 32 ? x / runs : uint64_t(uint32_t(x) / runs);
}
// HEAD counts where runs are long enough to be evened out by it: where they are
// short it would be most of them.  Row tiles of up to WHOLE units besides it are
// not cut: the second start and the join cost more than that saves.
template <uint32_t HEAD, uint32_t WHOLE>
__device__ __forceinline__ void set_runs(const AttnArgs &a, Line &line, uint64_t units, uint64_t tiles) {
  line.head = HEAD && units >= uint64_t(2 * HEAD) * a.runs ? HEAD : 0;
  line.total = units + line.head * tiles;
  line.per = divide_up(line.total, a.runs);
  line.whole = WHOLE + line.head;
}
// Requests from the first broken offset on have no row tiles, in this launch and
// the ones after it: offsets that decrease would give a token to two requests.
__device__ __forceinline__ uint32_t good_requests(const AttnArgs &a, uint32_t first) {
  if (a.after && *a.after) first = 0;
  if (a.broken && (blockIdx.x | blockIdx.y | threadIdx.x) == 0) *a.broken = first < a.n_req;
  return first;
}
template <uint32_t KT_LOG, uint32_t HEAD, uint32_t WHOLE, uint32_t NT>
__device__ __forceinline__ Line line_up(const AttnArgs &a, uint64_t *incl, uint64_t *sh) {
  const auto add = [](uint64_t x, uint64_t y) { return x + y; };
  Line line;
  if (a.n_req <= 64) {
    const uint32_t lane = threadIdx.x & 63;
    line.L = lengths_of(a, min(lane, a.n_req - 1));
    const uint64_t bad = __ballot(!line.L.ok);
    const uint32_t good = good_requests(a, bad ? uint32_t(__ffsll((unsigned long long)bad)) - 1 : a.n_req);
    const uint32_t t = lane < good ? row_tiles(a, line.L.n) : 0;
    const uint64_t units = wave_incl_scan(units_before<KT_LOG>(a, line.L, t), uint64_t(0), add);
    const uint64_t tiles = HEAD ? wave_incl_scan(uint64_t(t), uint64_t(0), add) : 0;
    set_runs<HEAD, WHOLE>(a, line, lane63(units), HEAD ? lane63(tiles) : 0);
    line.incl = units + line.head * tiles;
    return line;
  }
  constexpr uint32_t PER = AT_REQ / NT;
  const uint32_t k = (a.n_req + NT - 1) / NT, r0 = threadIdx.x * k;
  uint64_t u[PER], units = 0, tiles = 0;
  uint32_t t[PER], good = a.n_req;
#pragma unroll
  for (uint32_t j = 0; j < PER; ++j) {
    u[j] = t[j] = 0;
    if (j < k && r0 + j < a.n_req) {
      const Lengths L = lengths_of(a, r0 + j);
      t[j] = row_tiles(a, L.n);
      u[j] = units_before<KT_LOG>(a, L, t[j]);
      if (!L.ok) good = min(good, r0 + j);
    }
  }
  good = wave_reduce(good, ~0u, [](uint32_t x, uint32_t y) { return min(x, y); });
  if ((threadIdx.x & 63) == 0) incl[threadIdx.x >> 6] = good;
  __syncthreads();
#pragma unroll
  for (uint32_t w = 0; w < NT / 64; ++w) good = min(good, uint32_t(incl[w]));
  good = good_requests(a, good);
#pragma unroll
  for (uint32_t j = 0; j < PER; ++j) {
    if (r0 + j >= good) u[j] = t[j] = 0;
    units += u[j];
    tiles += t[j];
  }
  uint64_t all_units, all_tiles = 0;
  uint64_t at = block_incl_scan<NT, uint64_t>(units, 0, add, sh, all_units) - units;
  if (HEAD) tiles = block_incl_scan<NT, uint64_t>(tiles, 0, add, sh, all_tiles) - tiles;
  set_runs<HEAD, WHOLE>(a, line, all_units, all_tiles);
  at += line.head * tiles;
#pragma unroll
  for (uint32_t j = 0; j < PER; ++j) {
    at += u[j] + line.head * t[j];
    if (j < k && r0 + j < a.n_req) incl[r0 + j] = at;
  }
  __syncthreads();
  return line;
}
// Runs that a row tile of n units spans which begins at unit u, in run `run`.
__device__ __forceinline__ uint32_t parts_of(uint64_t u, uint32_t n, uint64_t per, uint32_t run) {
  const uint64_t x = u + n - 1;
  return ((x | per) >> 32 ? uint32_t(x / per) : uint32_t(x) / uint32_t(per)) - run + 1;
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, uint32_t lane) { return uint32_t(__builtin_amdgcn_readlane(int(v), int(lane))); }
__device__ __forceinline__ uint64_t lane_of(uint64_t v, uint32_t lane) {
  return uint64_t(lane_of(uint32_t(v), lane)) | uint64_t(lane_of(uint32_t(v >> 32), lane)) << 32;
}

// The run's segments one after the other: which request, row tile and units.
struct Segment {
  Lengths L;
  uint32_t r, row0;        // request, the row tile's first row in it (row: token * group + head)
  uint32_t n_units, first, count;
  bool skip;               // another run's
  uint32_t klim, open;     // keys that any row of the tile sees, and those that all of them see
};
template <uint32_t KT_LOG>
__device__ __forceinline__ Segment segment_at(const AttnArgs &a, const Line &line, const uint64_t *incl, uint64_t u, uint64_t u_end) {
  Segment s;
  uint64_t before;
  if (a.n_req <= 64) {
    s.r = uint32_t(__ffsll((unsigned long long)__ballot(line.incl > u)) - 1);
    s.L.first = int64_t(lane_of(uint64_t(line.L.first), s.r));
    s.L.n = lane_of(line.L.n, s.r);
    s.L.ctx = lane_of(line.L.ctx, s.r);
    s.L.klen = lane_of(line.L.klen, s.r);
    before = s.r ? lane_of(line.incl, s.r - 1) : 0;
  } else {
    uint32_t lo = 0, hi = a.n_req - 1;
    while (lo < hi) {
      const uint32_t mid = (lo + hi) / 2;
      if (incl[mid] > u) hi = mid;
      else lo = mid + 1;
    }
    s.r = __builtin_amdgcn_readfirstlane(lo);
    s.L = lengths_of(a, s.r);
    before = s.r ? incl[s.r - 1] : 0;
  }
  const uint64_t local = u - before;
  uint32_t t = 0, t_hi = row_tiles(a, s.L.n) - 1;
  while (t < t_hi) {  // the last tile that begins at or before `local`
    const uint32_t mid = (t + t_hi + 1) / 2;
    if (units_before<KT_LOG>(a, s.L, mid) + line.head * uint64_t(mid) <= local) t = mid;
    else t_hi = mid - 1;
  }
  const uint64_t keys_u = units_before<KT_LOG>(a, s.L, t);
  s.n_units = uint32_t(units_before<KT_LOG>(a, s.L, t + 1) - keys_u) + line.head;
  s.first = uint32_t(local - keys_u - line.head * uint64_t(t));
  // one that is not cut is the run's in which it begins
  s.skip = s.n_units <= line.whole && s.first;
  s.count = s.n_units <= line.whole ? s.n_units - s.first : uint32_t(min(uint64_t(s.n_units - s.first), u_end - u));
  s.row0 = t * a.stride;
  s.klim = a.mask ? s.L.klen : uint32_t(min(uint64_t(s.L.klen), uint64_t(s.L.ctx) + (uint64_t(t + 1) << a.tok_log)));
  // (a chain's rows all see the keys up to the tile's first token's)
  s.open = a.mask ? min(s.L.ctx, s.klim) : uint32_t(min(uint64_t(s.klim), uint64_t(s.L.ctx) + (uint64_t(t) << a.tok_log) + 1));
  return s;
}

// Row `row` of a segment's row tile: its token in the request and its head in the group.
struct Row {
  uint32_t token, h;
  bool live;  // one of the tile's rows; else the tile's rows' last token stands in
};
__device__ __forceinline__ Row row_of(const AttnArgs &a, const Segment &s, uint32_t row) {
  const uint32_t at = s.row0 + row, token = at / a.grp;
  return Row{min(token, s.L.n - 1), at - token * a.grp, row < a.stride && token < s.L.n};
  // (a row that is not live has a token and a head all the same: its products are not used)
}

template <typename T> struct Mma;
template <> struct Mma<__bf16> {
  static __device__ __forceinline__ f32x4 mul(bf16x8 x, bf16x8 y, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
  }
  static constexpr uint32_t EXP = 0x7F80;  // exponent of infinities and NaN
  // log2 of the weight of the maximum's key.  float16 has 24 powers of two below
  // 1 and the least of them without bits to spare: with weights up to 2^7 a
  // weight keeps its 11 bits down to 2^-21 of the largest, and is lost below
  // 2^-32 (e^-22), where from 1 on those would be 2^-14 and 2^-25.
  static constexpr float LIFT = 0.0f;
  // Sums of 16 weights of a lane past which k_attn_tiles brings the maximum up to
  // date; no weight of float16 overflows below.
  static constexpr float GROWN = 16384.0f;
};
template <> struct Mma<_Float16> {
  static __device__ __forceinline__ f32x4 mul(f16x8 x, f16x8 y, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
  }
  static constexpr uint32_t EXP = 0x7C00;
  static constexpr float LIFT = 7.0f, GROWN = 32768.0f;
};
// What a row's weights are relative to, as an exponent of two, from its maximum.
template <typename T>
__device__ __forceinline__ float base_of(const AttnArgs &a, float m) {
  return __builtin_fmaf(m, a.scale2, -Mma<T>::LIFT);
}

__device__ __forceinline__ float sum8(f32x8 a) {
  return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
}

// The larger of two, as the middle of them and an infinity that the compiler
// does not know for one: from fmaxf() it makes a maximum behind two more
// instructions, which quiet a NaN in either.  (A NaN among the scores makes its
// weight NaN, and with it the row, whatever the maximum is.)
__device__ __forceinline__ float max2(float x, float y) {
  float inf = INFINITY;
  asm("" : "+s"(inf));
  return __builtin_amdgcn_fmed3f(x, y, inf);
}
// The larger, and the sum, of the four lanes 16 apart, in all four.
__device__ __forceinline__ float max_quarters(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = max2(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max2(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float sum_quarters(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The low min(n, 8) bits (none for n <= 0).
__device__ __forceinline__ uint32_t low_bits(int64_t n) {
  return n <= 0 ? 0u : n >= 8 ? 0xFFu : (1u << uint32_t(n)) - 1u;
}

// Which of the eight keys from kb a row sees: below klim, and of the new ones
// (from ctx on) those of its mask, or up to itself.
__device__ __forceinline__ uint32_t seen8(const AttnArgs &a, const Lengths &L, uint32_t klim, uint32_t kb, uint32_t token) {
  const uint32_t within = low_bits(int64_t(klim) - kb);
  if (!a.mask) return within & low_bits(int64_t(L.ctx) + token + 1 - kb);
  const uint32_t old = low_bits(int64_t(L.ctx) - kb);
  if (old == 0xFFu) return within;
  const int64_t j0 = int64_t(kb) - L.ctx;
  const uint64_t *row = a.mask + (uint64_t(L.first) + token) * a.words;
  uint64_t w = 0;
  if (j0 < 0) {
    w = a.words ? row[0] << uint32_t(-j0) : 0;
  } else {
    const uint32_t at = uint32_t(j0 >> 6), sh = uint32_t(j0 & 63);
    if (at < a.words) w = row[at] >> sh;
    if (sh > 56 && at + 1 < a.words) w |= row[at + 1] << (64 - sh);
  }
  return within & (old | (uint32_t(w) & 0xFFu & ~old));
}

// N elements of one output row from d on, from the sums o relative to 2^top and
// the softmax sum.  A row that saw nothing: zeros, -inf.
template <typename T, uint32_t N>
__device__ __forceinline__ void finish(const AttnArgs &a, int64_t token, uint32_t h, uint32_t d, const float *o, float top,
                                       float sum, bool with_lse) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  T *p = static_cast<T *>(a.out) + token * a.out_ts + int64_t(h) * a.out_hs + d;
  typedef T TN __attribute__((ext_vector_type(N)));
  TN x;
#pragma unroll
  for (uint32_t j = 0; j < N; ++j) x[j] = T(sum == 0.0f ? 0.0f : o[j] * inv);
  if (a.out_vec) {
    *reinterpret_cast<TN *>(p) = x;
  } else {
#pragma unroll
    for (uint32_t j = 0; j < N; ++j) p[j] = x[j];
  }
  if (with_lse && a.lse)
    a.lse[token * a.hq + h] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
}

// Two transposing reads: four elements of the row that this lane and the three
// beside it name become four rows' elements at this lane's place among 16.
template <typename T>
__device__ __forceinline__ u32x4 turned(const T *p0, const T *p1) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 *lds;
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p0)), y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p1));
  const uint2 u = __builtin_bit_cast(uint2, x), v = __builtin_bit_cast(uint2, y);
  return u32x4{u.x, u.y, v.x, v.y};
}

// Values that masked places may hold.  0 * inf is NaN, so infinities and NaN
// leave the products of tiles with masked places (they become zeros), and
// add_apart() adds them, at the end of a segment, to the rows that see them.
template <typename T>
__device__ __forceinline__ uint32_t set_apart(uint32_t &f) {  // not 0: there were some
  const uint32_t bad = ((f & 0x7FFF7FFFu) + (0x8000u - Mma<T>::EXP) * 0x10001u) & 0x80008000u;
  f &= ~((bad >> 15) * 0xFFFFu);
  return bad;
}

// place(v, seen) for each key of a tile: its values' row, and which of the
// lane's rows (token[0..MT)) see it.
template <typename T, uint32_t MT, typename F>
__device__ void add_apart(const AttnArgs &a, const Segment &s, const char *vc, uint32_t from, uint32_t to, const uint32_t *token,
                          F place) {
  for (uint32_t key = from; key < to; ++key) {
    const uint32_t page = uint32_t(a.table[uint64_t(s.r) * a.table_stride + (key >> a.page_shift)]);
    if (page >= a.n_pages) continue;
    const T *v = reinterpret_cast<const T *>(vc) + int64_t(page) * a.page_stride + int64_t(key & ((1u << a.page_shift) - 1)) * a.token_stride;
    uint32_t seen = 0;
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) seen |= (seen8(a, s.L, s.klim, key, token[i]) & 1) << i;
    place(v, seen);
  }
}
template <typename T>
__device__ __forceinline__ float apart(T v) {  // an infinity or NaN, or 0
  const float x = float(v);
  return (__builtin_bit_cast(uint16_t, v) & Mma<T>::EXP) == Mma<T>::EXP ? x : 0.0f;
}

template <typename T, uint32_t D, uint32_t MT>
__global__ __launch_bounds__(AT_BLOCK, (D * MT <= 128 ? 3 : D * MT <= 256 ? 2 : 1)) void k_attn_rows(AttnArgs a) {
  typedef typename Vec8<T>::type T8;
  constexpr uint32_t NS = D / 32;          // steps of the first product
  constexpr uint32_t VD = D / 16;          // a lane's elements of one value row
  constexpr uint32_t M = 16 * MT;
  constexpr uint32_t JC = VD < 8 ? VD : 8; // elements joined at once
  constexpr uint32_t PAD = 16 * JC + 4;
  __shared__ uint64_t s_incl[AT_REQ];
  __shared__ uint64_t s_scan[2 * AT_BLOCK / 64 + 1];
  __shared__ float s_o[AT_WAVES][16][PAD];
  __shared__ float s_m[AT_WAVES][M], s_l[AT_WAVES][M];

  const uint32_t head = blockIdx.x, run = blockIdx.y;
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, g = lane >> 4;
  const Line line = line_up<AT_KT_LOG, 0, AT_ROWS_WHOLE, AT_BLOCK>(a, s_incl, s_scan);
  const uint64_t total = line.total;
  const uint64_t per = line.per;
  const uint64_t u_end = min(total, (uint64_t(run) + 1) * per);
  uint64_t u = uint64_t(run) * per;
  uint32_t *meta = a.meta + (uint64_t(head) * a.runs + run) * 4;
  bool left_open = false;  // a row tile begins here and ends in a later run

  const char *kc = a.kc + int64_t(head) * a.head_stride * int64_t(sizeof(T));
  const char *vc = a.vc + int64_t(head) * a.head_stride * int64_t(sizeof(T));

  while (u < u_end) {
    const Segment sg = segment_at<AT_KT_LOG>(a, line, s_incl, u, u_end);
    if (sg.skip) {
      u += sg.count;
      continue;
    }
    const Lengths &L = sg.L;
    const uint32_t r = sg.r, n_units = sg.n_units, first = sg.first, count = sg.count;
    const uint32_t klim = sg.klim, open = sg.open;
    const int32_t *pages = a.table + uint64_t(r) * a.table_stride;

    // queries: row 16 * i + n16 of the tile
    T8 q[MT][NS];
    uint32_t token[MT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
      const Row w = row_of(a, sg, 16 * i + n16);
      token[i] = w.token;
      const T *p = static_cast<const T *>(a.q) + (L.first + w.token) * a.q_ts + int64_t(head * a.grp + w.h) * a.q_hs;
#pragma unroll
      for (uint32_t s = 0; s < NS; ++s) {
        q[i][s] = __builtin_bit_cast(T8, __builtin_bit_cast(u32x4, load8_raw(p + s * 32 + g * 8, a.q_vec)) ^ a.flip);
      }
    }
    f32x4 acc[MT][VD];
    float m[MT], l[MT];
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (uint32_t j = 0; j < VD; ++j) acc[i][j] = f32x4{};
    }

    uint32_t odd_from = ~0u;  // this wave's first unit with infinities or NaN beside masked places
    for (uint32_t unit = first; unit < first + count; ++unit) {
      const uint32_t key0 = (unit << AT_KT_LOG) + wave * AT_TILE;
      if (key0 >= klim) break;
      // the pages of this lane's eight values (keys kb..) and of its two keys (8 * (n16 / 4) + n16 % 4, and + 4)
      const uint32_t kb = key0 + 8 * g, kk = key0 + 8 * (n16 >> 2);
      const int32_t pv = pages[min(kb, klim - 1) >> a.page_shift];
      const int32_t pk = pages[min(kk, klim - 1) >> a.page_shift];
      const uint32_t in_page = (1u << a.page_shift) - 1;
      const bool v_ok = uint32_t(pv) < a.n_pages, k_ok = uint32_t(pk) < a.n_pages;
      const char *kp = kc + (int64_t(k_ok ? pk : 0) * a.page_stride + int64_t((kk & in_page) + (n16 & 3)) * a.token_stride) * int64_t(sizeof(T)) + g * 16;
      const char *vp = vc + (int64_t(v_ok ? pv : 0) * a.page_stride + int64_t(kb & in_page) * a.token_stride) * int64_t(sizeof(T)) + n16 * (VD * sizeof(T));
      T8 ka[NS], kb8[NS];
#pragma unroll
      for (uint32_t s = 0; s < NS; ++s) {
        ka[s] = *reinterpret_cast<const T8 *>(kp + s * 64);
        kb8[s] = *reinterpret_cast<const T8 *>(kp + 4 * a.token_stride * int64_t(sizeof(T)) + s * 64);
      }
      uint32_t v[8][VD / 2];
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        const char *p = vp + int64_t(e) * a.token_stride * int64_t(sizeof(T));
        if constexpr (VD == 4) {
          const uint2 x = *reinterpret_cast<const uint2 *>(p);
          v[e][0] = x.x;
          v[e][1] = x.y;
        } else {
#pragma unroll
          for (uint32_t c = 0; c < VD / 8; ++c) {
            const u32x4 x = *reinterpret_cast<const u32x4 *>(p + 16 * c);
#pragma unroll
            for (uint32_t w = 0; w < 4; ++w) v[e][4 * c + w] = x[w];
          }
        }
      }
      // tiles in which some row does not see some key
      const bool part = key0 + AT_TILE > open || __any(!v_ok);
      if (part) {
        uint32_t bad = 0;
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
#pragma unroll
          for (uint32_t w = 0; w < VD / 2; ++w) bad |= set_apart<T>(v[e][w]);
        if (__any(bad != 0)) odd_from = min(odd_from, unit);
      }
      T8 pf[MT];
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i) {
        f32x4 sa{}, sb{};
#pragma unroll
        for (uint32_t s = 0; s < NS; ++s) {
          sa = Mma<T>::mul(ka[s], q[i][s], sa);
          sb = Mma<T>::mul(kb8[s], q[i][s], sb);
        }
        float x[8] = {sa[0], sa[1], sa[2], sa[3], sb[0], sb[1], sb[2], sb[3]};
        if (part) {
          const uint32_t seen = v_ok ? seen8(a, L, klim, kb, token[i]) : 0;
#pragma unroll
          for (uint32_t e = 0; e < 8; ++e) x[e] = (seen >> e & 1) ? x[e] : -INFINITY;
        }
        const float top = max_quarters(max2(max2(max2(x[0], x[1]), max2(x[2], x[3])), max2(max2(x[4], x[5]), max2(x[6], x[7]))));
        if (__any(top > m[i])) {
          const float m_new = max2(m[i], top);
          const float f = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[i] - m_new) * a.scale2);
          m[i] = m_new;
          l[i] *= f;
#pragma unroll
          for (uint32_t j = 0; j < VD; ++j) acc[i][j] *= f;
        }
        const float base = m[i] == -INFINITY ? 0.0f : base_of<T>(a, m[i]);
        f32x8 p;
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], a.scale2, -base));
        l[i] += sum8(p);
        // (rounded: the matrix product's operand)
        pf[i] = from_float<T>(p);
      }
      // values turned over, two elements of eight keys at a time
#pragma unroll
      for (uint32_t w = 0; w < VD / 2; ++w) {
        u32x4 f0, f1;
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          f0[e] = __builtin_amdgcn_perm(v[2 * e + 1][w], v[2 * e][w], 0x05040100);
          f1[e] = __builtin_amdgcn_perm(v[2 * e + 1][w], v[2 * e][w], 0x07060302);
        }
#pragma unroll
        for (uint32_t half = 0; half < 2; ++half) {
          const u32x4 f = half ? f1 : f0;
#pragma unroll
          for (uint32_t i = 0; i < MT; ++i)
            acc[i][2 * w + half] = Mma<T>::mul(__builtin_bit_cast(T8, f), pf[i], acc[i][2 * w + half]);
        }
      }
    }

    for (uint32_t unit = odd_from; unit < first + count; ++unit) {
      const uint32_t key0 = (unit << AT_KT_LOG) + wave * AT_TILE;
      if (key0 >= klim) break;
      if (!__any(!(uint32_t(pages[min(key0 + 8 * g, klim - 1) >> a.page_shift]) < a.n_pages)) && key0 + AT_TILE <= open) continue;
      add_apart<T, MT>(a, sg, vc, key0, min(key0 + AT_TILE, klim), token, [&](const T *v, uint32_t seen) {
#pragma unroll
        for (uint32_t j = 0; j < VD; ++j)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            const float x = apart(v[(4 * g + e) * VD + j]);
#pragma unroll
            for (uint32_t i = 0; i < MT; ++i) acc[i][j][e] += (seen >> i & 1) ? x : 0.0f;
          }
      });
    }

    // the waves' sums join: [wave][row][element]
    const bool whole = first == 0 && count == n_units;
    float *part = a.part + ((uint64_t(head) * a.runs + run) * 2 + (first == 0 ? 1 : 0)) * (M * (D + 2));
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
      l[i] = sum_quarters(l[i]);
      if (g == 0) {
        s_m[wave][16 * i + n16] = base_of<T>(a, m[i]);
        s_l[wave][16 * i + n16] = l[i];
      }
    }
    const uint32_t jr = threadIdx.x >> 4, jd = threadIdx.x & 15;  // a thread's row and run of elements in the join
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
#pragma unroll
      for (uint32_t j0 = 0; j0 < VD; j0 += JC) {
        __syncthreads();
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
#pragma unroll
          for (uint32_t j = 0; j < JC; ++j) s_o[wave][n16][(4 * g + e) * JC + j] = acc[i][j0 + j][e];
        __syncthreads();
        const uint32_t row = 16 * i + jr;
        float top = s_m[0][row];
#pragma unroll
        for (uint32_t w = 1; w < AT_WAVES; ++w) top = fmaxf(top, s_m[w][row]);
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f, o[JC];
#pragma unroll
        for (uint32_t j = 0; j < JC; ++j) o[j] = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < AT_WAVES; ++w) {
          const float f = __builtin_amdgcn_exp2f(s_m[w][row] - base);
          sum += s_l[w][row] * f;
#pragma unroll
          for (uint32_t j = 0; j < JC; ++j) o[j] += s_o[w][jr][jd * JC + j] * f;
        }
        const uint32_t d = jd * VD + j0;
        const Row w = row_of(a, sg, row);
        if (!w.live) continue;
        if (whole) {
          finish<T, JC>(a, L.first + w.token, head * a.grp + w.h, d, o, top, sum, d == 0);
        } else {
#pragma unroll
          for (uint32_t j = 0; j < JC; ++j) part[row * D + d + j] = o[j];
          if (d == 0) {
            part[M * D + row] = top;
            part[M * D + M + row] = sum;
          }
        }
      }
    }
    __syncthreads();  // s_m, s_l and s_o are free again
    if (first == 0 && !whole) {
      left_open = true;
      if (threadIdx.x == 0) {
        meta[0] = parts_of(u, n_units, per, run);
        meta[1] = uint32_t(L.first);
        meta[2] = L.n;
        meta[3] = sg.row0;
      }
    }
    u += count;
  }
  if (!left_open && threadIdx.x == 0) meta[0] = 0;
}

// Row tiles of 16 * MT rows for each of W waves.  With this many rows the
// products, not the cache, take the time, and what counts is how often K and V
// pass from memory to the registers: the waves of a workgroup share tiles of KT
// keys in LDS, two of them, one read while the next is on its way (from global
// memory to LDS without registers between; the two are variables of their own,
// so that the compiler sees that reads of one need not wait for the other).  The products are k_attn_rows'; V's fragment comes turned over from
// LDS by the transposing reads.  16-byte chunks of a row are stored at (chunk
// XOR a function of the row), so that 16 rows at one chunk, and 16 rows by four
// lanes, fall on different banks.
template <uint32_t D>
__device__ __forceinline__ uint32_t k_chunk(uint32_t row, uint32_t c) {
  return D == 64 ? c ^ (row >> 1 & 7) : c ^ (row & 15);
}
template <uint32_t D>
__device__ __forceinline__ uint32_t v_chunk(uint32_t row, uint32_t c) {
  return D == 64 ? c ^ ((row >> 1 & 3) << 1) : c ^ ((row & 7) << 1);
}

// Which of the 64 keys from key0 on a row sees (seen8's rules).
__device__ __forceinline__ uint64_t low_bits64(int64_t n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t(0) : (uint64_t(1) << uint32_t(n)) - 1;
}
__device__ __forceinline__ uint64_t seen64(const AttnArgs &a, const Lengths &L, uint32_t klim, uint32_t key0, uint32_t token) {
  const uint64_t within = low_bits64(int64_t(klim) - key0);
  if (!a.mask) return within & low_bits64(int64_t(L.ctx) + token + 1 - key0);
  const uint64_t old = low_bits64(int64_t(L.ctx) - key0);
  const int64_t j0 = int64_t(key0) - L.ctx;
  if (j0 <= -64) return within;
  const uint64_t *row = a.mask + (uint64_t(L.first) + token) * a.words;
  uint64_t w = 0;
  if (j0 < 0) {
    w = row[0] << uint32_t(-j0);
  } else {
    const uint32_t at = uint32_t(j0 >> 6), sh = uint32_t(j0 & 63);
    if (at < a.words) w = row[at] >> sh;
    if (sh && at + 1 < a.words) w |= row[at + 1] << (64 - sh);
  }
  return within & (old | w);  // (w has no bits below the context's end)
}

// Waits for this wave's loads (s_waitcnt vmcnt(0), the other counters free).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

template <typename T, uint32_t D, uint32_t W, uint32_t MT, uint32_t KT_LOG>
__global__ __launch_bounds__(64 * W, 2) void k_attn_tiles(AttnArgs a) {
  typedef typename Vec8<T>::type T8;
  constexpr uint32_t KT = 1u << KT_LOG;      // keys of a tile
  constexpr uint32_t NS = D / 32, ND = D / 16;
  constexpr uint32_t CH = D / 8;             // 16-byte chunks of a row
  constexpr uint32_t RPI = 64 / CH;          // rows of one load to LDS (1 KiB)
  constexpr uint32_t ROWS = KT / W;          // rows that a wave fetches, in groups of 8 (of one page each)
  constexpr uint32_t GROUPS = ROWS / 8, LPG = 8 / RPI;
  constexpr uint32_t LOADS = 2 * GROUPS * LPG;  // a wave's loads for one tile
  constexpr uint32_t M = 16 * MT * W;
  static_assert(ROWS % 8 == 0 && KT >= 32 && KT <= 64, "");
  __shared__ __attribute__((aligned(1024))) T s_k0[KT * D], s_v0[KT * D], s_k1[KT * D], s_v1[KT * D];
  __shared__ uint64_t s_incl[AT_REQ];
  __shared__ uint64_t s_scan[2 * W + 1];
  __shared__ __attribute__((aligned(8))) uint8_t s_hidden[4][8];  // a tile's groups of eight keys whose page is not in the cache
  __shared__ uint32_t s_odd;               // the segment has infinities or NaN in tiles with masked places

  const uint32_t head = blockIdx.x, run = blockIdx.y;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n16 = lane & 15, g = lane >> 4;
  const Line line = line_up<KT_LOG, AT_HEAD, AT_WHOLE, 64 * W>(a, s_incl, s_scan);
  const uint64_t total = line.total;
  const uint64_t per = line.per;
  const uint64_t u_end = min(total, (uint64_t(run) + 1) * per);
  uint64_t u = uint64_t(run) * per;
  uint32_t *meta = a.meta + (uint64_t(head) * a.runs + run) * 4;
  bool left_open = false;
  const char *kc = a.kc + int64_t(head) * a.head_stride * int64_t(sizeof(T));
  const char *vc = a.vc + int64_t(head) * a.head_stride * int64_t(sizeof(T));
  const uint32_t in_page = (1u << a.page_shift) - 1;
  if (threadIdx.x < 32) (&s_hidden[0][0])[threadIdx.x] = 0;  // (a tile of 32 keys has four groups)
  // a lane's sources in its loads to LDS, from a group of eight rows' first on:
  // row i * RPI + lane / CH of the group, and the chunk whose place is lane % CH
  uint32_t k_from[GROUPS][LPG], v_from[LPG];
#pragma unroll
  for (uint32_t i = 0; i < LPG; ++i) {
    const uint32_t row = i * RPI + lane / CH;
    v_from[i] = row * uint32_t(a.token_stride) * uint32_t(sizeof(T)) + 16 * v_chunk<D>(row, lane % CH);
#pragma unroll
    for (uint32_t gi = 0; gi < GROUPS; ++gi)
      k_from[gi][i] = row * uint32_t(a.token_stride) * uint32_t(sizeof(T)) + 16 * k_chunk<D>(8 * (wave * GROUPS + gi) + row, lane % CH);
  }
  // its places in the fragments' reads of a tile: K's row 16 k + n16, V's rows
  // 32 k + 4 g + n16 / 4 and + 16 (four lanes read 32 bytes of a row), both with
  // chunks that repeat within the row steps
  constexpr uint32_t VA = ND < 8 ? ND : 8;
  uint32_t k_at[NS], v_at[VA];
#pragma unroll
  for (uint32_t e = 0; e < NS; ++e) k_at[e] = n16 * D + 8 * k_chunk<D>(n16, 4 * e + g);
#pragma unroll
  for (uint32_t j = 0; j < VA; ++j) {
    const uint32_t row = 4 * g + (n16 >> 2);
    v_at[j] = row * D + 8 * v_chunk<D>(row, 2 * j + (n16 >> 1 & 1)) + 4 * (n16 & 1);
  }

  while (u < u_end) {
    const Segment sg = segment_at<KT_LOG>(a, line, s_incl, u, u_end);
    if (sg.skip) {
      u += sg.count;
      continue;
    }
    const Lengths &L = sg.L;
    // the table's row, read by scalar loads, whose counter the loads to LDS do not share
    const __attribute__((address_space(4))) int32_t *pages =
        (const __attribute__((address_space(4))) int32_t *)(a.table + uint64_t(sg.r) * a.table_stride);
    // tiles of keys [unit0, unit_end): the segment's units without the row tile's first line.head
    const uint32_t unit0 = max(sg.first, line.head) - line.head;
    const uint32_t unit_end = min(max(sg.first + sg.count, line.head) - line.head, (sg.klim + KT - 1) >> KT_LOG);

    uint32_t page[GROUPS];  // of this wave's groups in the next tile to fetch
    const auto look = [&](uint32_t unit) {
#pragma unroll
      for (uint32_t gi = 0; gi < GROUPS; ++gi)
        page[gi] = uint32_t(pages[min((unit << KT_LOG) + 8 * (wave * GROUPS + gi), sg.klim - 1) >> a.page_shift]);
    };
    // this wave's rows of a tile, on their way to LDS: load n of LOADS, K's first.
    // (A page outside the cache reads page 0 and is masked.)
    int64_t from_at[GROUPS];
    const auto aim = [&](uint32_t unit) {
#pragma unroll
      for (uint32_t gi = 0; gi < GROUPS; ++gi) {
        const uint32_t group = wave * GROUPS + gi, key = (unit << KT_LOG) + 8 * group;
        const bool ok = page[gi] < a.n_pages;
        from_at[gi] = (int64_t(ok ? page[gi] : 0) * a.page_stride + int64_t(key & in_page) * a.token_stride) * int64_t(sizeof(T));
        if (lane == 0) s_hidden[unit & 3][group] = !ok;
      }
    };
    const auto fetch = [&](uint32_t n, T *k_to, T *v_to) {
      typedef const __attribute__((address_space(1))) void *from;
      typedef __attribute__((address_space(3))) void *to;
      const uint32_t gi = n % (LOADS / 2) / LPG, i = n % LPG, row = 8 * (wave * GROUPS + gi) + i * RPI;
      if (n < LOADS / 2) __builtin_amdgcn_global_load_lds((from)(kc + from_at[gi] + k_from[gi][i]), (to)(k_to + row * D), 16, 0, 0);
      else __builtin_amdgcn_global_load_lds((from)(vc + from_at[gi] + v_from[i]), (to)(v_to + row * D), 16, 0, 0);
    };
    if (threadIdx.x == 0) s_odd = 0;
    __syncthreads();
    if (unit0 < unit_end) {
      look(unit0);
      aim(unit0);
#pragma unroll
      for (uint32_t n = 0; n < LOADS; ++n) fetch(n, s_k0, s_v0);
      look(min(unit0 + 1, unit_end - 1));
      aim(min(unit0 + 1, unit_end - 1));
    }

    T8 q[MT][NS];
    uint32_t token[MT];
    bool any = false;  // a row of this wave's is one of the tile's
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
      const Row w = row_of(a, sg, 16 * (wave * MT + i) + n16);
      any |= w.live;
      token[i] = w.token;
      const T *p = static_cast<const T *>(a.q) + (L.first + w.token) * a.q_ts + int64_t(head * a.grp + w.h) * a.q_hs;
#pragma unroll
      for (uint32_t s = 0; s < NS; ++s) {
        q[i][s] = __builtin_bit_cast(T8, __builtin_bit_cast(u32x4, load8_raw(p + s * 32 + g * 8, a.q_vec)) ^ a.flip);
      }
    }
    any = __any(any);
    f32x4 acc[MT][ND];
    float m[MT], l[MT];
    bool fresh = true;
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (uint32_t j = 0; j < ND; ++j) acc[i][j] = f32x4{};
    }

    // this wave's rows of V, once they are there: in a tile where some row does
    // not see some key all of them, in others those of a group that is hidden
    const auto clean = [&](T *v, bool all, uint64_t hidden) {
      uint32_t bad = 0;
#pragma unroll
      for (uint32_t i = 0; i < ROWS / RPI; ++i) {
        if (!all && !(hidden >> (8 * (wave * GROUPS + i / LPG)) & 1)) continue;
        u32x4 *p = reinterpret_cast<u32x4 *>(v + wave * ROWS * D) + 64 * i + lane;
        u32x4 f = *p;
        uint32_t here = 0;
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          uint32_t w = f[e];
          here |= set_apart<T>(w);
          f[e] = w;
        }
        if (here) *p = f;
        bad |= here;
      }
      if (all && __any(bad != 0)) s_odd = 1;  // (every wave that finds some writes the same)
    };

    const auto step = [&](uint32_t unit, const T *s_k, T *s_v, T *k_free, T *v_free) {
      wait_loads();  // this wave's rows of the tile are there
      const bool ends = ((unit + 1) << KT_LOG) > sg.open;  // some row does not see some key
      uint64_t hidden = *reinterpret_cast<const uint64_t *>(s_hidden[unit & 3]);  // (this wave's groups: its own writes)
      if (ends || hidden) clean(s_v, ends, hidden);
      __syncthreads();  // everybody's are, and everybody is done with the tile before
      // The next tile's loads, aimed in the step before: what the waves do here
      // they all do at once, with the matrix cores at rest.  (Past the segment's
      // last tile they fetch that one again: no branch cuts the products apart.)
#pragma unroll
      for (uint32_t n = 0; n < LOADS; ++n) fetch(n, k_free, v_free);
      const uint32_t after = min(unit + 2, unit_end - 1);
      if (!any) {
        look(after);
        aim(after);
        return;
      }
      hidden = *reinterpret_cast<const uint64_t *>(s_hidden[unit & 3]);
      const uint32_t key0 = unit << KT_LOG;
      // Fragments are read a group ahead of the products that use them; left to
      // itself the compiler puts each read right before its use.
      T8 kf[2][NS];
      const auto read_k = [&](uint32_t k) {
#pragma unroll
        for (uint32_t e = 0; e < NS; ++e) kf[k & 1][e] = *reinterpret_cast<const T8 *>(s_k + k_at[e] + 16 * k * D);
      };
      constexpr uint32_t VG = ND < 4 ? ND : 4, VN = ND / VG * (KT / 32);  // V's fragments of a group; groups
      T8 vf[2][VG];
      const auto read_v = [&](uint32_t n) {
#pragma unroll
        for (uint32_t e = 0; e < VG; ++e) {
          const uint32_t j = n * VG % ND + e, k = n * VG / ND;
          const T *p = s_v + v_at[j % 8] + 128 * (j / 8) + 32 * k * D;
          vf[n & 1][e] = __builtin_bit_cast(T8, turned(p, p + 16 * D));
        }
      };
      f32x4 s[MT][KT / 16];
      float add[MT];
      // Weights are relative to m, which need not be the running maximum: it is
      // brought up to it while a row has seen no key (`fresh`), and when weights
      // grow past GROWN; then the tile is done again.  Nearly every tile gets
      // by without its maximum.
      for (bool exact = fresh;; exact = true) {
        read_k(0);
#pragma unroll
        for (uint32_t k = 0; k < KT / 16; ++k) {
          if (k + 1 < KT / 16) read_k(k + 1);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (uint32_t i = 0; i < MT; ++i) s[i][k] = f32x4{};
#pragma unroll
          for (uint32_t e = 0; e < NS; ++e)
#pragma unroll
            for (uint32_t i = 0; i < MT; ++i) s[i][k] = Mma<T>::mul(kf[k & 1][e], q[i][e], s[i][k]);
          __builtin_amdgcn_sched_barrier(0);
        }
        look(after);
        read_v(0);
        __builtin_amdgcn_sched_barrier(0);
        if (ends || hidden) {
          uint64_t shown = ~uint64_t(0);
          for (uint32_t e = 0; e < KT / 8; ++e)
            if (hidden >> (8 * e) & 1) shown &= ~(uint64_t(0xFF) << (8 * e));
#pragma unroll
          for (uint32_t i = 0; i < MT; ++i) {
            const uint64_t seen = (seen64(a, L, sg.klim, key0, token[i]) & shown) >> (4 * g);  // a lane's keys are 16 k + 4 g ..+3
#pragma unroll
            for (uint32_t k = 0; k < KT / 16; ++k)
#pragma unroll
              for (uint32_t e = 0; e < 4; ++e) s[i][k][e] = (seen >> (16 * k + e) & 1) ? s[i][k][e] : -INFINITY;
          }
        }
        if (exact) {
          bool none = false;
#pragma unroll
          for (uint32_t i = 0; i < MT; ++i) {
            float top = m[i];
#pragma unroll
            for (uint32_t k = 0; k < KT / 16; ++k) top = max2(top, max2(max2(s[i][k][0], s[i][k][1]), max2(s[i][k][2], s[i][k][3])));
            top = max_quarters(top);
            const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[i] - top) * a.scale2);
            m[i] = top;
            none |= top == -INFINITY;
            l[i] *= f;
#pragma unroll
            for (uint32_t j = 0; j < ND; ++j) acc[i][j] *= f;
          }
          fresh = __any(none);
        }
        bool grown = false;
#pragma unroll
        for (uint32_t i = 0; i < MT; ++i) {
          const float base = m[i] == -INFINITY ? 0.0f : base_of<T>(a, m[i]);
          add[i] = 0.0f;
#pragma unroll
          for (uint32_t k = 0; k < KT / 16; ++k) {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) s[i][k][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][k][e], a.scale2, -base));
            add[i] += (s[i][k][0] + s[i][k][1]) + (s[i][k][2] + s[i][k][3]);
          }
          grown |= add[i] > Mma<T>::GROWN;
        }
        if (exact || !__any(grown)) break;
      }
      aim(after);
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i) l[i] += add[i];
      T8 pf[MT][KT / 32];
#pragma unroll
      for (uint32_t k = 0; k < KT / 32; ++k)
#pragma unroll
        for (uint32_t i = 0; i < MT; ++i) {
          // (rounded: the matrix product's operand)
          const f32x4 x = s[i][2 * k], y = s[i][2 * k + 1];
          pf[i][k] = from_float<T>(f32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
        }
#pragma unroll
      for (uint32_t n = 0; n < VN; ++n) {
        if (n + 1 < VN) read_v(n + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (uint32_t e = 0; e < VG; ++e)
#pragma unroll
          for (uint32_t i = 0; i < MT; ++i) {
            const uint32_t j = n * VG % ND + e;
            acc[i][j] = Mma<T>::mul(vf[n & 1][e], pf[i][n * VG / ND], acc[i][j]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (uint32_t unit = unit0; unit < unit_end; unit += 2) {
      step(unit, s_k0, s_v0, s_k1, s_v1);
      if (unit + 1 < unit_end) step(unit + 1, s_k1, s_v1, s_k0, s_v0);
    }
    wait_loads();     // nothing is on its way to LDS any more,
    __syncthreads();  // s_odd is settled, and every stage is free for the next segment
    if (s_odd && any)
      for (uint32_t unit = max(unit0, sg.open >> KT_LOG); unit < unit_end; ++unit)
        add_apart<T, MT>(a, sg, vc, unit << KT_LOG, min((unit + 1) << KT_LOG, sg.klim), token, [&](const T *v, uint32_t seen) {
#pragma unroll
          for (uint32_t j = 0; j < ND; ++j)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const float x = apart(v[16 * j + 4 * g + e]);
#pragma unroll
              for (uint32_t i = 0; i < MT; ++i) acc[i][j][e] += (seen >> i & 1) ? x : 0.0f;
            }
        });
    __syncthreads();  // s_odd has been read

    const bool whole = sg.first == 0 && sg.count == sg.n_units;
    float *part = a.part + ((uint64_t(head) * a.runs + run) * 2 + (sg.first == 0 ? 1 : 0)) * (M * (D + 2));
#pragma unroll
    for (uint32_t i = 0; i < MT; ++i) {
      const float sum = sum_quarters(l[i]), top = base_of<T>(a, m[i]);
      const uint32_t row = 16 * (wave * MT + i) + n16;
      const Row w = row_of(a, sg, row);
      if (!w.live) continue;
      if (whole) {
#pragma unroll
        for (uint32_t j = 0; j < ND; ++j) {
          const float o[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
          finish<T, 4>(a, L.first + w.token, head * a.grp + w.h, 16 * j + 4 * g, o, top, sum, j == 0 && g == 0);
        }
      } else {
#pragma unroll
        for (uint32_t j = 0; j < ND; ++j) *reinterpret_cast<f32x4 *>(part + row * D + 16 * j + 4 * g) = acc[i][j];
        if (g == 0) {
          part[M * D + row] = top;
          part[M * D + M + row] = sum;
        }
      }
    }
    if (sg.first == 0 && !whole) {
      left_open = true;
      if (threadIdx.x == 0) {
        meta[0] = parts_of(u, sg.n_units, per, run);
        meta[1] = uint32_t(L.first);
        meta[2] = L.n;
        meta[3] = sg.row0;
      }
    }
    u += sg.count;
  }
  if (!left_open && threadIdx.x == 0) meta[0] = 0;
}

// Adds up the parts of the row tiles that were cut, of the one that begins in
// run blockIdx.y.  D / 4 threads have a row, four elements each.  Small tiles
// are cut into many parts and are few: a workgroup takes one row, and its
// threads' groups every SLOTS-th part; large ones come in two parts or three:
// a group takes two rows, whose loads are under way together.
template <typename T, uint32_t D, uint32_t M>
__global__ __launch_bounds__(AT_BLOCK) void k_attn_join(AttnArgs a) {
  constexpr uint32_t TPR = D / 4, SLOTS = AT_BLOCK / TPR, R = join_rows(M, D) == 1 ? 1 : 2;
  constexpr uint32_t U = 4;  // parts whose loads are under way together
  constexpr uint64_t SIZE = M * (D + 2);
  __shared__ f32x4 s_o[R == 1 ? AT_BLOCK : 1];
  __shared__ float s_top[SLOTS], s_sum[SLOTS];
  const uint32_t head = blockIdx.x, run = blockIdx.y, slot = threadIdx.x / TPR, c = threadIdx.x % TPR;
  const uint4 meta = *reinterpret_cast<const uint4 *>(a.meta + (uint64_t(head) * a.runs + run) * 4);
  const uint32_t n = meta.x;
  if (n == 0) return;
  Segment sg;
  sg.L.first = meta.y;
  sg.L.n = meta.z;
  sg.row0 = meta.w;
  // the first part is this run's second place, the others the first places of the runs after it
  const float *base = a.part + (uint64_t(head) * a.runs + run) * 2 * SIZE;
  const auto at = [&](uint32_t p) { return base + (p == 0 ? SIZE : uint64_t(p) * 2 * SIZE); };
  uint32_t row[R];
  Row w[R];
  float top[R], sum[R];
  f32x4 o[R];
#pragma unroll
  for (uint32_t i = 0; i < R; ++i) {
    row[i] = R == 1 ? blockIdx.z : (blockIdx.z * R + i) * SLOTS + slot;
    w[i] = row_of(a, sg, row[i]);
    top[i] = -INFINITY;
    sum[i] = 0.0f;
    o[i] = f32x4{};
  }
  if (R == 1 && !w[0].live) return;
  for (uint32_t p0 = R == 1 ? slot : 0; p0 < n; p0 += R == 1 ? U * SLOTS : U) {
    f32x4 x[R][U];
    float m[R][U], l[R][U];
#pragma unroll
    for (uint32_t i = 0; i < R; ++i)
#pragma unroll
      for (uint32_t e = 0; e < U; ++e) {
        const uint32_t p = p0 + e * (R == 1 ? SLOTS : 1);
        m[i][e] = -INFINITY;
        l[i][e] = 0.0f;
        x[i][e] = f32x4{};
        if (p < n && w[i].live) {
          const float *src = at(p);
          x[i][e] = *reinterpret_cast<const f32x4 *>(src + row[i] * D + 4 * c);
          m[i][e] = src[M * D + row[i]];
          l[i][e] = src[M * D + M + row[i]];
        }
      }
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) {
      float next = top[i];
#pragma unroll
      for (uint32_t e = 0; e < U; ++e) next = fmaxf(next, m[i][e]);
      const float from = next == -INFINITY ? 0.0f : next;
      const float f = __builtin_amdgcn_exp2f(top[i] - from);
      sum[i] *= f;
      o[i] *= f;
#pragma unroll
      for (uint32_t e = 0; e < U; ++e) {
        const float g = __builtin_amdgcn_exp2f(m[i][e] - from);
        sum[i] += l[i][e] * g;
        o[i] += x[i][e] * g;
      }
      top[i] = next;
    }
  }
  if constexpr (R == 1) {
    s_o[threadIdx.x] = o[0];
    if (c == 0) {
      s_top[slot] = top[0];
      s_sum[slot] = sum[0];
    }
    __syncthreads();
    if (slot) return;
    const uint32_t used = min(n, SLOTS);
    for (uint32_t e = 1; e < used; ++e) top[0] = fmaxf(top[0], s_top[e]);
    const float from = top[0] == -INFINITY ? 0.0f : top[0];
    sum[0] = 0.0f;
    o[0] = f32x4{};
    for (uint32_t e = 0; e < used; ++e) {
      const float g = __builtin_amdgcn_exp2f(s_top[e] - from);
      sum[0] += s_sum[e] * g;
      o[0] += s_o[e * TPR + c] * g;
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < R; ++i) {
    if (!w[i].live) continue;
    const float v[4] = {o[i][0], o[i][1], o[i][2], o[i][3]};
    finish<T, 4>(a, sg.L.first + w[i].token, head * a.grp + w[i].h, 4 * c, v, top[i], sum[i], c == 0);
  }
}

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

// Rows of a row tile: 16 or 32 (k_attn_rows), 64, 128 or 256 (k_attn_tiles), by
// the rows that a request has for one key/value head on average.  us a call with
// each, at 32 requests of 8,192 keys and 8 heads (4 of 256 elements):
//   rows   heads of 64                 heads of 128                 heads of 256
//     16   108, 114, 102, 104, 130     215, 213, 197, 198, 190      235, 242, 200, 203
//     32   132, 120, 104, 107, 130     232, 220, 203, 203, 190      291, 252, 205, 210
//     64   253, 157, 111, 114, 137     452, 225, 211, 215, 192      462, 320, 222, 221
//     96   375, 307, 145, 119, 141     676, 593, 241, 226, 205      786, 624, 244, 232
//    256   997, 589, 306, 212, 195     1788, 868, 511, 333, 294     1877, 922, 449, 363
// Where row tiles are few they are cut into many parts, and the small tiles'
// parts are joined sooner: one request of 4 rows and 4,000 keys takes 12, 17, 26,
// 29, 21, and of 131,072 keys for a single head 38, 40, 114, 119, 86; 8 requests
// of 1,000 keys take 16, 20, 15, 19, 20.
// Where a call is short a tile's start and end are most of its time, and rows that
// a request does not fill are waste: tiles of 64 up to so many rows times keys of
// a table row, over all requests and heads.  What a table row can hold is all
// that the host knows of the keys.  us with tiles of 64 and of the size below,
// trees by 4 query heads on contexts of a quarter to all of the row's keys (8
// heads of 64 and 128, 4 of 256; of 64 with rows <= 128: 128, else 256):
//   requests x rows, keys   heads of 64        heads of 128       heads of 256
//     8 x 256, 1,000        22, 26             32, 37             39, 40
//     8 x 256, 4,000        36, 35             52, 49             57, 54
//     32 x 96, 500          23, 25             31, 34             36, 43
//     32 x 96, 4,000        51, 46             93, 84             102, 84
//     32 x 256, 1,000       46, 53             65, 71             73, 76
//     32 x 256, 4,000       100, 91            190, 128           204, 148
//     128 x 96, 1,000       73, 70             110, 111           118, 116
//     128 x 96, 4,000       201, 157           414, 282           409, 284
//     128 x 256, 250        89, 77             118, 104           111, 99
//     128 x 256, 4,000      420, 304           918, 430           907, 579
// The limits lie a little past where the two meet (at 2^26, and 2^25), since
// contexts far shorter than the row gain more than full rows lose: 59 trees of 4
// to 22 tokens on up to 192 keys take 19 and 34.  Heads of 256 on rows of 161 to
// 320 keys are cut and joined only where tiles of 64 rows have units of 32 keys: 32
// x 96 rows on 250 keys 30 and 23.
uint32_t tile_rows(uint64_t n_tok, uint32_t n_req, uint32_t hk, uint32_t grp, uint32_t dim, uint64_t keys) {
  const uint64_t rows = std::max<uint64_t>(grp, n_tok * grp / std::max(1u, n_req));
  if (rows <= 32 && uint64_t(n_req) * hk <= 64) return rows <= 16 ? 16 : 32;
  const uint64_t all = std::max<uint64_t>(1, n_tok * grp * hk);
  const bool brief = rows <= 256 && grp <= 64 && keys <= 4096 && keys <= (dim == 256 ? 1u << 26 : 1u << 27) / all &&
                     !(dim == 256 && keys > AT_WHOLE * 32 && keys <= AT_WHOLE * 64);
  if (rows <= 16 || brief) return 64;
  if (dim == 128) return 256;
  if (rows <= 64) return 64;
  return rows <= 128 || dim == 256 ? 128 : 256;
}

struct Plan {
  uint32_t rows, runs;
  uint64_t meta_bytes, bytes;
};
Plan plan_of(uint64_t n_tok, uint32_t n_req, uint32_t hq, uint32_t hk, uint32_t dim, uint64_t keys) {
  Plan p;
  p.rows = tile_rows(n_tok, n_req, hk, hq / hk, dim, keys);
  p.runs = std::max(1u, (p.rows > 128 || (dim == 256 && p.rows == 128) ? AT_RUNS / 2 : AT_RUNS) / hk);
  p.meta_bytes = (uint64_t(hk) * p.runs * 16 + 8 + 255) / 256 * 256;  // (and two words between launches)
  p.bytes = p.meta_bytes + uint64_t(hk) * p.runs * 2 * p.rows * (dim + 2) * sizeof(float);
  return p;
}

bool good_cache(const bbpe_paged_cache *c) {
  return c && (c->dtype == BBPE_BF16 || c->dtype == BBPE_F16) && (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256) &&
         c->n_kv_heads >= 1 && c->n_kv_heads <= 4096 && c->page_size >= 8 && c->page_size <= 65536 &&
         (c->page_size & (c->page_size - 1)) == 0 && c->n_pages >= 1 && c->n_pages <= 0x7FFFFFFFull && c->k && c->v &&
         ((addr(c->k) | addr(c->v)) & 15) == 0 && ((c->page_stride | c->head_stride | c->token_stride) & 7) == 0 &&
         c->token_stride >= 0 && c->token_stride < (1 << 27);
}
bool good_heads(uint32_t hq, const bbpe_paged_cache *c) {
  return hq >= 1 && hq % c->n_kv_heads == 0 && hq / c->n_kv_heads <= 128;
}

template <typename T, uint32_t D, uint32_t M>
void launch(const AttnArgs &a, hipStream_t st) {
  const dim3 grid(a.hk, a.runs);
  if constexpr (M <= 32) k_attn_rows<T, D, M / 16><<<grid, AT_BLOCK, 0, st>>>(a);
  else if constexpr (D == 256 && M == 128) k_attn_tiles<T, D, 8, 1, 6><<<grid, 2 * AT_BLOCK, 0, st>>>(a);
  else if constexpr (M <= 128) k_attn_tiles<T, D, 4, M / 64, (D == 256 ? 5 : 6)><<<grid, AT_BLOCK, 0, st>>>(a);
  else k_attn_tiles<T, D, 8, M / 128, 6><<<grid, 2 * AT_BLOCK, 0, st>>>(a);
  // Nothing to join where no row tile can be long enough to be cut (a chain's
  // last one counts keys up to its end, past the request's).
  constexpr uint32_t whole = M <= 32 ? AT_ROWS_WHOLE << AT_KT_LOG : AT_WHOLE << (D == 256 && M == 64 ? 5 : 6);
  if (uint64_t(a.cap) + (a.mask ? 0 : 1u << a.tok_log) <= whole) return;
  k_attn_join<T, D, M><<<dim3(a.hk, a.runs, M / join_rows(M, D)), AT_BLOCK, 0, st>>>(a);
}
template <typename T, uint32_t D>
void launch_rows(const AttnArgs &a, uint32_t rows, hipStream_t st) {
  if (rows == 16) return launch<T, D, 16>(a, st);
  if (rows == 32) return launch<T, D, 32>(a, st);
  if (rows == 64) return launch<T, D, 64>(a, st);
  if constexpr (D != 128)
    if (rows == 128) return launch<T, D, 128>(a, st);
  if constexpr (D != 256) launch<T, D, 256>(a, st);
}
template <typename T>
void launch_dim(const AttnArgs &a, uint32_t dim, uint32_t rows, hipStream_t st) {
  dim == 64 ? launch_rows<T, 64>(a, rows, st) : dim == 128 ? launch_rows<T, 128>(a, rows, st) : launch_rows<T, 256>(a, rows, st);
}

}  // namespace
}  // namespace bbpe

using namespace bbpe;

extern "C" {

int bbpe_tree_attention_workspace_bytes(uint64_t n_tokens, uint32_t n_req, uint32_t n_q_heads,
                                        const bbpe_paged_cache *cache, uint64_t *out_bytes) {
  if (!out_bytes || !good_cache(cache) || !good_heads(n_q_heads, cache)) return BBPE_E_INVALID_ARG;
  // for tables of any width
  *out_bytes = std::max(plan_of(n_tokens, n_req, n_q_heads, cache->n_kv_heads, cache->head_dim, 0).bytes,
                        plan_of(n_tokens, n_req, n_q_heads, cache->n_kv_heads, cache->head_dim, ~uint64_t(0)).bytes);
  return BBPE_OK;
}

int bbpe_tree_attention(const void *q, int64_t q_ts, int64_t q_hs, uint64_t n_tokens,
                        uint32_t n_q_heads, const bbpe_paged_cache *cache, const int32_t *d_table,
                        uint64_t table_stride, uint32_t table_width, const int64_t *d_q_off,
                        const int32_t *d_ctx_len, uint32_t n_req, const uint64_t *d_tree_mask,
                        uint32_t mask_words, float scale, void *out, int64_t out_ts,
                        int64_t out_hs, float *d_lse, void *d_workspace, uint64_t workspace_bytes,
                        void *hip_stream) {
  if (!good_cache(cache) || !good_heads(n_q_heads, cache)) return BBPE_E_INVALID_ARG;
  if (n_tokens > 0x7FFFFFFFull || n_tokens * (n_q_heads / cache->n_kv_heads) > 0x7FFFFFFFull || !std::isfinite(scale) || (n_req > 1 && table_stride < table_width) ||
      uint64_t(table_width) * cache->page_size > 0x7FFFFFFFull)
    return BBPE_E_INVALID_ARG;
  if (n_tokens == 0 || n_req == 0) return BBPE_OK;
  if (!q || !out || !d_table || table_width == 0 || !d_q_off || !d_ctx_len || (d_tree_mask && mask_words == 0))
    return BBPE_E_INVALID_ARG;
  if ((addr(q) & 1) || (addr(out) & 1) || (addr(d_table) & 3) || (addr(d_q_off) & 7) || (addr(d_ctx_len) & 3) ||
      (addr(d_tree_mask) & 7) || (addr(d_lse) & 3))
    return BBPE_E_INVALID_ARG;
  const Plan p = plan_of(n_tokens, n_req, n_q_heads, cache->n_kv_heads, cache->head_dim, uint64_t(table_width) * cache->page_size);
  if (!d_workspace || (addr(d_workspace) & 255) || workspace_bytes < p.bytes) return BBPE_E_WORKSPACE;
  AttnArgs a{};
  a.q = q;
  a.q_ts = q_ts;
  a.q_hs = q_hs;
  a.kc = static_cast<const char *>(cache->k);
  a.vc = static_cast<const char *>(cache->v);
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.n_pages = cache->n_pages;
  a.page_shift = uint32_t(__builtin_ctz(cache->page_size));
  a.table_stride = table_stride;
  a.cap = table_width * cache->page_size;
  a.mask = d_tree_mask;
  a.words = mask_words;
  // 2^-120 for a scale of zero: every weight comes out one, and a masked score stays -inf
  a.scale2 = scale == 0.0f ? 0x1p-120f : std::fabs(scale) * 1.44269504088896340736f;
  a.flip = scale < 0.0f ? 0x80008000u : 0u;
  a.out = out;
  a.out_ts = out_ts;
  a.out_hs = out_hs;
  a.lse = d_lse;
  a.n_tok = n_tokens;
  a.hq = n_q_heads;
  a.hk = cache->n_kv_heads;
  a.grp = a.hq / a.hk;
  a.tok_log = uint32_t(31 - __builtin_clz(p.rows / a.grp));
  a.stride = d_tree_mask ? p.rows : a.grp << a.tok_log;
  a.runs = p.runs;
  a.q_vec = ((addr(q) | uint64_t(q_ts * 2) | uint64_t(q_hs * 2)) & 15) == 0;
  a.out_vec = ((addr(out) | uint64_t(out_ts * 2) | uint64_t(out_hs * 2)) & 15) == 0;
  a.meta = static_cast<uint32_t *>(d_workspace);
  a.part = reinterpret_cast<float *>(static_cast<char *>(d_workspace) + p.meta_bytes);
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  for (uint32_t r0 = 0; r0 < n_req; r0 += AT_REQ) {
    a.table = d_table + r0 * table_stride;
    a.q_off = d_q_off + r0;
    a.ctx = d_ctx_len + r0;
    a.n_req = std::min(AT_REQ, n_req - r0);
    uint32_t *const flags = a.meta + uint64_t(a.hk) * a.runs * 4;
    a.after = r0 ? flags + (r0 / AT_REQ & 1) : nullptr;
    a.broken = n_req - r0 > AT_REQ ? flags + (r0 / AT_REQ + 1 & 1) : nullptr;
    if (cache->dtype == BBPE_BF16) launch_dim<__bf16>(a, cache->head_dim, p.rows, st);
    else launch_dim<_Float16>(a, cache->head_dim, p.rows, st);
  }
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

}  // extern "C"
