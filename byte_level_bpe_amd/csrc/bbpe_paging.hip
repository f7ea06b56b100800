// Block tables and slot maps built on the device from request lengths: the
// pages that a serving step's new tokens need are handed out from a free list,
// and every token gets its cache slot and its position.
//
// Request r with c = ctx[r] cached and n = q_off[r+1] - q_off[r] new tokens
// holds ceil(c/P) pages and needs ceil((c+n)/P) - ceil(c/P) more; its first is
// entry (sum of the needs before r) of the free list.  Token i of it sits at
// place p = c + i, so in entry p / P of the row, at p % P of that page.
//
// The work is stores (16 bytes a token, 4 a table entry) behind one scan over
// the requests.  Up to PG_FOLD requests every workgroup makes that scan for
// itself and one launch does everything; beyond, a one-workgroup scan goes
// first.  Measured on an MI355X, captured in a graph: 5.4 us for 8 requests of
// one token (queued from Python 6.2), nearly all of it the launch and the chain of
// three dependent loads; 18.2 us for 4,096 requests and 2.9 million tokens (46 MB,
// which a fill alone writes in 9 us), of which the scan, by instructions that
// every workgroup runs, takes 6; with the scan as a launch of its own 29.6.  8,192
// requests of 350 tokens 40 us, 65,536 of 44 173: there the one workgroup's scan
// is most of it (65,536 of one token 150).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/bbpe.h"
#include "bbpe_device.h"

namespace bbpe {
namespace {

// Threads of a workgroup: many for many requests (a wave scans 64 at a time:
// four rounds for 4,096 with 1,024 threads, 18.6 us for 700 tokens each, eight
// with 512, 26 us), few for few (8 requests of 358,400 tokens: 15 us with 256,
// 17 with 512, 18 with 1,024).
constexpr uint32_t PG_FEW = 256, PG_MANY = 1024, PG_FEW_REQ = 512;
// Requests that every workgroup scans for itself.
constexpr uint32_t PG_FOLD = 4096;
constexpr uint32_t PG_TOKENS = 4;                    // a thread's tokens in one round
constexpr uint32_t PG_PIECE = 2048;                  // table entries of one wave's piece
constexpr uint32_t PG_FAILED = 0xFFFFFFFFu;          // start of a request that failed
constexpr uint32_t PG_THREADS = 512 * 1024;          // threads of a launch at most (two large workgroups a compute unit)

struct TableArgs {
  const int64_t *q_off;
  const int32_t *ctx;
  const int32_t *free_pages;
  int32_t *table;
  const int32_t *depth;
  int64_t *slots;
  int32_t *pos, *req, *seq;
  int64_t *status;
  uint32_t *start;      // [n_req] more than PG_FOLD requests: first free-list entry, or PG_FAILED
  uint32_t *n_good;     // [1] requests before the first broken offset
  uint64_t table_stride, n_free, n_tok;
  uint32_t n_req, width, page, page_shift;  // page_shift: 32 if the page size is no power of two
  uint32_t vec_tok, vec_table;              // outputs 16-byte aligned: vector stores
};

__device__ __forceinline__ uint32_t page_of(const TableArgs &a, uint32_t p) {
  return a.page_shift < 32 ? p >> a.page_shift : p / a.page;
}
// ceil(x / P) for x up to 2^31
__device__ __forceinline__ uint32_t pages_for(const TableArgs &a, uint32_t x) {
  return x ? page_of(a, x - 1) + 1 : 0;
}

// offsets that cannot be followed
__device__ __forceinline__ bool off_broken(const TableArgs &a, int64_t lo, int64_t hi) {
  return uint64_t(lo) > uint64_t(hi) || uint64_t(hi) > a.n_tok;  // (a negative one is a large one)
}

struct Request {
  int64_t lo, hi;
  int32_t ctx;
};
__device__ __forceinline__ Request read_request(const TableArgs &a, uint32_t r) {
  return Request{a.q_off[r], a.q_off[r + 1], a.ctx[r]};
}

// Pages that request q needs, and its code before the free list is looked at.
__device__ __forceinline__ uint32_t need_of(const TableArgs &a, const Request &q, bool broken, int &code) {
  code = BBPE_OK;
  if (broken || q.ctx < 0 || q.hi - q.lo + q.ctx > 0x7FFFFFFFll) {
    code = BBPE_E_INVALID_ARG;
    return 0;
  }
  const uint32_t n = uint32_t(q.hi - q.lo), old = pages_for(a, uint32_t(q.ctx));
  const uint32_t end = pages_for(a, uint32_t(q.ctx) + n);
  if (end > a.width) {
    code = BBPE_E_CAPACITY;
    return 0;
  }
  return n ? end - old : 0;
}

// What a run of requests adds to the status record.
struct Tally {
  uint32_t first;  // first failed request (~0: none)
  int code;
  uint32_t pages, tokens;  // (pages handed out once, from fewer than 2^31; tokens up to n_tok)
};
__device__ __forceinline__ void settle(const TableArgs &a, const Request &q, uint32_t r, uint32_t need, int code,
                                       uint64_t start, bool write, uint32_t &kept, Tally &t) {
  if (code == BBPE_OK && need && start + need > a.n_free) code = BBPE_E_CAPACITY;
  kept = code == BBPE_OK ? uint32_t(start < PG_FAILED ? start : PG_FAILED - 1) : PG_FAILED;
  if (code == BBPE_OK) {
    t.pages += need;
    t.tokens += uint32_t(q.hi - q.lo);
  } else if (r < t.first) {
    t.first = r;
    t.code = code;
  }
  if (write) a.seq[r] = code == BBPE_OK ? int32_t(q.ctx + (q.hi - q.lo)) : max(q.ctx, 0);
}

// Minimum over the block (sh: one word a wave).
__device__ __forceinline__ uint32_t block_min(uint32_t v, uint32_t *sh, uint32_t waves) {
  for (int d = 32; d; d >>= 1) v = min(v, uint32_t(__shfl_xor(int(v), d, 64)));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t m = sh[0];
  for (uint32_t w = 1; w < waves; ++w) m = min(m, sh[w]);
  return m;
}
__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t *sh, uint32_t waves) {
  for (int d = 32; d; d >>= 1) v += uint64_t(__shfl_xor((unsigned long long)v, d, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t m = 0;
  for (uint32_t w = 0; w < waves; ++w) m += sh[w];
  return m;
}

__device__ __forceinline__ void write_status(const TableArgs &a, Tally t, uint32_t *sh32, uint64_t *sh64, uint32_t waves) {
  const uint32_t first = block_min(t.first, sh32, waves);
  const uint64_t pages = block_sum(t.pages, sh64, waves), tokens = block_sum(t.tokens, sh64, waves);
  if (threadIdx.x == 0) {
    a.status[2] = int64_t(pages);
    a.status[3] = int64_t(tokens);
    if (first == 0xFFFFFFFFu) {
      a.status[0] = BBPE_OK;
      a.status[1] = -1;
    }
  }
  if (first != 0xFFFFFFFFu && t.first == first) {
    a.status[0] = t.code;
    a.status[1] = int64_t(first);
  }
}

// The scan for more than PG_FOLD requests: one workgroup, 1,024 requests a round.
__global__ __launch_bounds__(1024) void k_page_scan(TableArgs a) {
  constexpr uint32_t NT = 1024;
  __shared__ uint64_t sh[2 * NT / 64 + 1];
  __shared__ uint32_t shm[NT / 64];
  uint64_t base = 0;
  uint32_t good = a.n_req;
  Tally t{0xFFFFFFFFu, BBPE_OK, 0, 0};
  for (uint32_t r0 = 0; r0 < a.n_req; r0 += NT) {
    const uint32_t r = r0 + threadIdx.x;
    Request q{0, 0, 0};
    if (r < a.n_req) q = read_request(a, r);
    const bool mine = r < a.n_req && off_broken(a, q.lo, q.hi);
    good = min(good, block_min(mine ? r : 0xFFFFFFFFu, shm, NT / 64));
    int code = BBPE_OK;
    const uint32_t need = r < a.n_req ? need_of(a, q, r >= good, code) : 0;
    uint64_t total;
    const uint64_t incl = block_incl_scan<NT, uint64_t>(need, 0, [](uint64_t x, uint64_t y) { return x + y; }, sh, total);
    if (r < a.n_req) {
      uint32_t kept;
      settle(a, q, r, need, code, base + incl - need, true, kept, t);
      a.start[r] = kept;
    }
    base += total;
  }
  write_status(a, t, shm, sh, NT / 64);
  if (threadIdx.x == 0) *a.n_good = good;
}

template <bool FOLDED, uint32_t PG_BLOCK>
__global__ __launch_bounds__(PG_BLOCK) void k_page_tables(TableArgs a) {
  constexpr uint32_t PG_TILE = PG_BLOCK * PG_TOKENS;  // a workgroup's tokens in one round
  constexpr uint32_t REQS = PG_BLOCK == PG_FEW ? PG_FEW_REQ : PG_FOLD;
  __shared__ uint64_t s_tally[PG_BLOCK / 64][3];
  __shared__ uint32_t shm[2 * (PG_BLOCK / 64)];  // the waves' first broken requests, then their sums
  __shared__ uint32_t s_off[FOLDED ? REQS + 1 : 1], s_start[FOLDED ? REQS : 1];
  __shared__ int32_t s_ctx[FOLDED ? REQS : 1];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr uint32_t WAVES = PG_BLOCK / 64;
  uint32_t good;
  if (FOLDED) {
    // A wave scans 64 k requests one after the other, 64 at a time; rolled, since
    // fetching straight-line code takes a small call longer than running it.
    // Every workgroup does it, so instructions count: sums are 32 bits wide and
    // stay at 2^32 - 1, past any free list, where they would pass it.
    const uint32_t k = (a.n_req + PG_BLOCK - 1) / PG_BLOCK;
    const auto add = [](uint32_t u, uint32_t v) { return __builtin_elementwise_add_sat(u, v); };
    uint32_t first = a.n_req, sum = 0;
    Request next{0, 0, 0};
    if (wave * k * 64 + lane < a.n_req) next = read_request(a, wave * k * 64 + lane);
#pragma unroll 1
    for (uint32_t j = 0; j < k; ++j) {
      const uint32_t r = (wave * k + j) * 64 + lane;
      const Request q = next;
      if (j + 1 < k && r + 64 < a.n_req) next = read_request(a, r + 64);
      uint32_t need = 0;
      int code = BBPE_E_INVALID_ARG;
      if (r < a.n_req) {
        const bool broken = off_broken(a, q.lo, q.hi);
        if (broken) first = min(first, r);
        need = need_of(a, q, broken, code);
        s_off[r] = uint32_t(q.lo);  // (read up to the first broken request's: within n_tok, so within 32 bits)
        if (r + 1 == a.n_req) s_off[r + 1] = uint32_t(q.hi);
        s_ctx[r] = q.ctx;
      }
      const uint32_t incl = add(sum, wave_incl_scan(need, 0u, add));
      if (r < a.n_req) s_start[r] = code == BBPE_OK ? min(incl - need, PG_FAILED - 1) : PG_FAILED;
      sum = lane63(incl);
    }
    first = wave_reduce(first, 0xFFFFFFFFu, [](uint32_t u, uint32_t v) { return min(u, v); });
    if (lane == 63) {
      shm[wave] = first;
      shm[WAVES + wave] = sum;
    }
    __syncthreads();
    uint32_t base = 0, total = 0;
    good = a.n_req;
#pragma unroll
    for (uint32_t w = 0; w < WAVES; ++w) {
      good = min(good, shm[w]);
      if (w == wave) base = total;
      total = add(total, shm[WAVES + w]);
    }
    if (blockIdx.x != 0 && total <= a.n_free) {
      // the list is long enough for all: only what follows a broken offset still fails
#pragma unroll 1
      for (uint32_t j = 0; j < k; ++j) {
        const uint32_t r = (wave * k + j) * 64 + lane;
        if (r >= a.n_req) break;
        const uint32_t at = s_start[r];
        s_start[r] = at == PG_FAILED || r >= good ? PG_FAILED : base + at;
      }
    } else {
      // (requests from the first broken offset on fail: the others' sums do not depend on them)
      Tally t{0xFFFFFFFFu, BBPE_OK, 0, 0};
#pragma unroll 1
      for (uint32_t j = 0; j < k; ++j) {
        const uint32_t r = (wave * k + j) * 64 + lane;
        if (r >= a.n_req) break;
        Request q{0, 0, s_ctx[r]};
        if (r < good) {
          q.lo = s_off[r];
          q.hi = s_off[r + 1];
        }
        int code;
        const uint32_t need = need_of(a, q, r >= good, code);
        settle(a, q, r, need, code, uint64_t(base) + s_start[r], blockIdx.x == 0, s_start[r], t);
      }
      if (blockIdx.x == 0) {
        // the first failed request with its code in one word, and the sums
        const uint64_t key = wave_reduce(uint64_t(t.first) << 8 | uint8_t(-t.code), ~uint64_t(0), [](uint64_t u, uint64_t v) { return u < v ? u : v; });
        const uint32_t pages = wave_sum(t.pages), tokens = wave_sum(t.tokens);
        if (lane == 0) {
          s_tally[wave][0] = key;
          s_tally[wave][1] = pages;
          s_tally[wave][2] = tokens;
        }
      }
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      uint64_t key = ~uint64_t(0), pages = 0, tokens = 0;
      for (uint32_t w = 0; w < WAVES; ++w) {
        key = key < s_tally[w][0] ? key : s_tally[w][0];
        pages += s_tally[w][1];
        tokens += s_tally[w][2];
      }
      const bool fine = uint32_t(key >> 8) == 0xFFFFFFFFu;
      a.status[0] = fine ? BBPE_OK : -int64_t(key & 0xFF);
      a.status[1] = fine ? -1 : int64_t(uint32_t(key >> 8));
      a.status[2] = int64_t(pages);
      a.status[3] = int64_t(tokens);
    }
  } else {
    good = *a.n_good;
  }
  const auto off = [&](uint32_t r) -> uint32_t { return FOLDED ? s_off[r] : uint32_t(a.q_off[r]); };
  const auto start_of = [&](uint32_t r) -> uint32_t { return FOLDED ? s_start[r] : a.start[r]; };
  const auto ctx_of = [&](uint32_t r) -> int32_t { return FOLDED ? s_ctx[r] : a.ctx[r]; };
  // The last request that begins at or before token i, the same i for the whole
  // wave (~0: before the first; good: past them all): 64 offsets at a time.
  const auto find = [&](uint32_t i) -> uint32_t {
    if (good == 0 || off(good) <= i) return good;
    uint32_t lo = 0, span = 1;
    while (span * 64 < good) span *= 64;
    for (; span; span /= 64) {
      const uint32_t r = lo + lane * span;
      const uint32_t c = uint32_t(__popcll(__ballot(r < good && off(r) <= i)));
      if (c == 0) return 0xFFFFFFFFu;  // (at the first level only)
      lo += (c - 1) * span;
    }
    return lo;
  };

  const uint32_t tiles = uint32_t((a.n_tok + PG_TILE - 1) / PG_TILE);
  const uint32_t per_row = (a.width + PG_PIECE - 1) / PG_PIECE;
  const uint64_t pieces = uint64_t(a.n_req) * per_row;
  const uint64_t items = tiles + (pieces + PG_BLOCK / 64 - 1) / (PG_BLOCK / 64);
  for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
    if (item < tiles) {
      const uint64_t i0 = item * PG_TILE + threadIdx.x * PG_TOKENS;
      if (item * PG_TILE + wave * 64 * PG_TOKENS >= a.n_tok) continue;  // the wave's first token
      // between the requests of the wave's first and last token
      const uint32_t w0 = uint32_t(item * PG_TILE + wave * 64 * PG_TOKENS);
      uint32_t r = find(w0), last = find(uint32_t(min(uint64_t(w0) + 64 * PG_TOKENS, a.n_tok) - 1));
      if (good && r != last) {
        uint32_t lo = r + 1, hi = min(last, good) + 1;  // off(lo - 1) <= i0 < off(hi), where those are
        while (lo < hi) {
          const uint32_t mid = (lo + hi) / 2;
          if (off(mid) <= i0) lo = mid + 1;
          else hi = mid;
        }
        r = lo - 1;
      }
      int64_t slot[PG_TOKENS];
      int32_t pos[PG_TOKENS], req[PG_TOKENS];
      uint32_t last_b = 0xFFFFFFFFu, last_r = 0xFFFFFFFFu;
      int32_t page = -1;
#pragma unroll
      for (uint32_t j = 0; j < PG_TOKENS; ++j) {
        const uint64_t i = i0 + j;
        slot[j] = -1;
        pos[j] = 0;
        req[j] = -1;
        if (i >= a.n_tok || good == 0) continue;
        while (r + 1 <= good && off(r + 1) <= i) ++r;  // r == ~0u wraps to request 0
        if (r >= good) continue;
        const uint32_t s = start_of(r);
        if (s == PG_FAILED) continue;
        const uint32_t c = uint32_t(ctx_of(r)), p = c + uint32_t(i - off(r)), b = page_of(a, p);
        if (b != last_b || r != last_r) {
          const uint32_t old = pages_for(a, c);
          page = b < old ? a.table[r * a.table_stride + b] : a.free_pages[s + (b - old)];
          last_b = b;
          last_r = r;
        }
        slot[j] = page < 0 ? -1 : int64_t(page) * a.page + (p - b * a.page);
        pos[j] = int32_t(a.depth ? c + uint32_t(a.depth[i]) : p);
        req[j] = int32_t(r);
      }
      if (a.vec_tok && i0 + PG_TOKENS <= a.n_tok) {
        reinterpret_cast<int4 *>(a.pos)[i0 / 4] = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (a.req) reinterpret_cast<int4 *>(a.req)[i0 / 4] = make_int4(req[0], req[1], req[2], req[3]);
        reinterpret_cast<longlong2 *>(a.slots)[i0 / 2] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2 *>(a.slots)[i0 / 2 + 1] = make_longlong2(slot[2], slot[3]);
      } else {
#pragma unroll
        for (uint32_t j = 0; j < PG_TOKENS; ++j)
          if (i0 + j < a.n_tok) {
            a.slots[i0 + j] = slot[j];
            a.pos[i0 + j] = pos[j];
            if (a.req) a.req[i0 + j] = req[j];
          }
      }
    } else {
      const uint64_t piece = (item - tiles) * (PG_BLOCK / 64) + (threadIdx.x >> 6);
      if (piece >= pieces) continue;
      const uint32_t r = uint32_t(piece / per_row);
      const uint32_t from = uint32_t(piece - uint64_t(r) * per_row) * PG_PIECE, to = min(a.width, from + PG_PIECE);
      const uint32_t s = start_of(r);
      const int32_t c = max(ctx_of(r), 0);
      const uint32_t old = min(pages_for(a, uint32_t(c)), a.width);
      uint32_t end = old;  // a failed request, or one without new tokens, takes none
      if (s != PG_FAILED && off(r + 1) != off(r)) end = pages_for(a, uint32_t(c) + (off(r + 1) - off(r)));
      int32_t *row = a.table + r * a.table_stride;
      const auto entry = [&](uint32_t b) -> int32_t { return b < end ? a.free_pages[s + (b - old)] : -1; };
      if (a.vec_table) {
        for (uint32_t b = max(from, old & ~3u) + lane * 4; b < to; b += 256) {
          if (b >= old && b + 4 <= to) {
            *reinterpret_cast<int4 *>(row + b) = make_int4(entry(b), entry(b + 1), entry(b + 2), entry(b + 3));
          } else {
            for (uint32_t e = max(b, old); e < min(b + 4, to); ++e) row[e] = entry(e);
          }
        }
      } else {
        for (uint32_t b = max(from, old) + lane; b < to; b += 64) row[b] = entry(b);
      }
    }
  }
}

}  // namespace
}  // namespace bbpe

using namespace bbpe;

extern "C" {

int bbpe_block_tables_workspace_bytes(uint32_t n_req, uint64_t *out_bytes) {
  if (!out_bytes) return BBPE_E_INVALID_ARG;
  *out_bytes = n_req > PG_FOLD ? 256 + 4 * uint64_t(n_req) : 0;
  return BBPE_OK;
}

int bbpe_block_tables(const int64_t *d_q_off, const int32_t *d_ctx_len, uint32_t n_req,
                      const int32_t *d_free_pages, uint64_t n_free, int32_t *d_table,
                      uint64_t table_stride, uint32_t table_width, uint32_t page_size,
                      uint64_t n_tokens, const int32_t *d_depth, int64_t *d_slots,
                      int32_t *d_positions, int32_t *d_requests, int32_t *d_seq_len,
                      int64_t *d_status, void *d_workspace, uint64_t workspace_bytes,
                      void *hip_stream) {
  const auto addr = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
  if (!d_q_off || !d_status || (n_req && (!d_ctx_len || !d_seq_len)) || (n_free && !d_free_pages) ||
      (n_req && table_width && !d_table) || (n_tokens && (!d_slots || !d_positions)))
    return BBPE_E_INVALID_ARG;
  if (page_size == 0 || page_size > (1u << 30) || table_width > 0x7FFFFFFFu || n_req > (1u << 24) ||
      n_free > 0x7FFFFFFFull || n_tokens > 0x7FFFFFFFull || (n_req > 1 && table_stride < table_width))
    return BBPE_E_INVALID_ARG;
  if ((addr(d_q_off) & 7) || (addr(d_slots) & 7) || (addr(d_status) & 7) || (addr(d_ctx_len) & 3) ||
      (addr(d_free_pages) & 3) || (addr(d_table) & 3) || (addr(d_depth) & 3) || (addr(d_positions) & 3) ||
      (addr(d_requests) & 3) || (addr(d_seq_len) & 3))
    return BBPE_E_INVALID_ARG;
  const bool folded = n_req <= PG_FOLD;
  if (!folded && (!d_workspace || (addr(d_workspace) & 255) || workspace_bytes < 256 + 4 * uint64_t(n_req)))
    return BBPE_E_WORKSPACE;
  TableArgs a{};
  a.q_off = d_q_off;
  a.ctx = d_ctx_len;
  a.free_pages = d_free_pages;
  a.table = d_table;
  a.depth = d_depth;
  a.slots = d_slots;
  a.pos = d_positions;
  a.req = d_requests;
  a.seq = d_seq_len;
  a.status = d_status;
  a.table_stride = table_stride;
  a.n_free = n_free;
  a.n_tok = n_tokens;
  a.n_req = n_req;
  a.width = table_width;
  a.page = page_size;
  a.page_shift = (page_size & (page_size - 1)) == 0 ? uint32_t(__builtin_ctz(page_size)) : 32u;
  a.vec_tok = ((addr(d_slots) | addr(d_positions) | addr(d_requests)) & 15) == 0;
  a.vec_table = (addr(d_table) & 15) == 0 && (table_stride & 3) == 0;
  const uint64_t pieces = uint64_t(n_req) * ((table_width + PG_PIECE - 1) / PG_PIECE);
  const auto grid = [&](uint32_t block) {
    const uint64_t items = (n_tokens + block * PG_TOKENS - 1) / (block * PG_TOKENS) + (pieces + block / 64 - 1) / (block / 64);
    return dim3(uint32_t(std::max<uint64_t>(1, std::min<uint64_t>(PG_THREADS / block, items))));
  };
  const hipStream_t st = static_cast<hipStream_t>(hip_stream);
  if (n_req <= PG_FEW_REQ) {
    k_page_tables<true, PG_FEW><<<grid(PG_FEW), PG_FEW, 0, st>>>(a);
  } else if (folded) {
    k_page_tables<true, PG_MANY><<<grid(PG_MANY), PG_MANY, 0, st>>>(a);
  } else {
    a.n_good = static_cast<uint32_t *>(d_workspace);
    a.start = a.n_good + 64;
    k_page_scan<<<1, 1024, 0, st>>>(a);
    k_page_tables<false, PG_MANY><<<grid(PG_MANY), PG_MANY, 0, st>>>(a);
  }
  return hipGetLastError() == hipSuccess ? BBPE_OK : BBPE_E_HIP;
}

}  // extern "C"
