// Rows of logits: reading them in pieces of 16 bytes, and sums over them, for
// the operators between a model's logits and ids.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/bbpe.h"

namespace bbpe {

constexpr uint32_t ROW_THREADS = 256;  // of a workgroup, where it is not a template's
constexpr uint32_t ROW_WAVES = ROW_THREADS / 64;
constexpr uint32_t ROW_UNROLL = 4;     // pieces of a thread's step
constexpr uint32_t ROW_STEP = ROW_THREADS * ROW_UNROLL;  // pieces of a workgroup's step
constexpr double LN2 = 0.69314718055994530942;
constexpr float LOWEST = -3.4028234663852886e38f;

template <typename T> struct Piece {
  static constexpr uint32_t N = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef uint32_t raw __attribute__((ext_vector_type(4)));  // its bits: elements by themselves would be loaded one after another
  typedef T mem __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));  // at any element
  typedef float val __attribute__((ext_vector_type(16 / sizeof(T))));
};

// A row in pieces of 16 aligned bytes, wherever it begins: vocabularies of odd
// sizes are common, and loads across cache lines took an eighth more time.
// Places count from the first piece's first element: [lead, end) are the row's.
template <typename C> struct Row {
  typedef typename std::remove_const<C>::type T;
  static constexpr uint32_t N = Piece<T>::N;
  C *at;  // place 0
  uint32_t lead, end;

  __device__ __forceinline__ Row(C *x, uint32_t vocab) {
    lead = uint32_t(reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T);
    at = x - lead;
    end = lead + vocab;
  }
  // The same pieces in another matrix, where they may begin at any element.
  template <typename D> __device__ __forceinline__ Row<D> over(D *y) const {
    Row<D> o(y, 0);
    o.at = y - lead;
    o.lead = lead;
    o.end = end;
    return o;
  }
  __device__ __forceinline__ uint32_t pieces() const { return (end + N - 1) / N; }
  __device__ __forceinline__ bool whole(uint32_t p) const { return p * N >= lead && p * N + N <= end; }
  // Piece p, from `from` (place 0 of a row that may lie otherwise in memory);
  // minus infinity where it is not the row's.
  __device__ __forceinline__ typename Piece<T>::raw load(const T *from, uint32_t p) const {
    typename Piece<T>::vec t;
    if (whole(p)) {
      t = *reinterpret_cast<const typename Piece<T>::mem *>(from + p * N);
      return __builtin_bit_cast(typename Piece<T>::raw, t);
    }
#pragma unroll
    for (uint32_t e = 0; e < N; ++e) t[e] = p * N + e >= lead && p * N + e < end ? from[p * N + e] : T(-INFINITY);
    return __builtin_bit_cast(typename Piece<T>::raw, t);
  }
  __device__ __forceinline__ typename Piece<T>::raw load(uint32_t p) const { return load(at, p); }
  // A step's pieces p, p + STRIDE, ..., below `last`.
  template <uint32_t STRIDE>
  __device__ __forceinline__ void load_step(typename Piece<T>::raw (&v)[ROW_UNROLL], const T *from, uint32_t p, uint32_t last) const {
#pragma unroll
    for (uint32_t u = 0; u < ROW_UNROLL; ++u) {
      if (p + u * STRIDE < last) {
        v[u] = load(from, p + u * STRIDE);
      } else {
        const typename Piece<T>::vec t = T(-INFINITY);
        v[u] = __builtin_bit_cast(typename Piece<T>::raw, t);
      }
    }
  }
  __device__ __forceinline__ void store(uint32_t p, typename Piece<T>::val f) const {
    const typename Piece<T>::vec v = __builtin_convertvector(f, typename Piece<T>::vec);  // to nearest even
    if (whole(p)) {
      *reinterpret_cast<typename Piece<T>::mem *>(at + p * N) = v;
    } else {
#pragma unroll
      for (uint32_t e = 0; e < N; ++e)
        if (p * N + e >= lead && p * N + e < end) at[p * N + e] = v[e];
    }
  }
};

// The sum of a piece's N numbers, in pairs.
template <uint32_t N, typename V> __device__ __forceinline__ float piece_sum(V v) {
#pragma unroll
  for (uint32_t half = N / 2; half; half /= 2)
#pragma unroll
    for (uint32_t e = 0; e < half; ++e) v[e] += v[e + half];
  return v[0];
}

template <typename T>
__device__ __forceinline__ typename Piece<T>::val values(typename Piece<T>::raw v) {
  return __builtin_convertvector(__builtin_bit_cast(typename Piece<T>::vec, v), typename Piece<T>::val);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// scale * log2(e) as two floats, the first rounded down: with one, weights of
// elements ten units below the largest would be off by a millionth, all the same way.
struct Exponent {
  float c, low;  // low > 0, so that minus infinity stays that
};
inline Exponent exponent_of(float scale) {
  const double e = double(scale) * 1.4426950408889634074;
  Exponent x{float(e), 0.0f};
  if (double(x.c) > e) x.c = nextafterf(x.c, 0.0f);
  x.low = fmaxf(float(e - double(x.c)), 1.17549435e-38f);
  return x;
}
// exp(scale * d), d up to 0.  Off by half a step of the exponent besides the
// exponential's own: 3 half steps of the weight 8 units down, 10 of one 30 down.
__device__ __forceinline__ float weight_of(float d, Exponent x) { return __builtin_amdgcn_exp2f(__builtin_fmaf(d, x.low, d * x.c)); }
// The same without that, its whole part taken off first: for the factors of whole
// sums, which put all of a sum off the same way.  (For elements, whose roundings
// cancel, it would cost: the loss of 2,048 rows of 200,005 in bfloat16 160 -> 184 us, in
// float32 287 -> 298.)
__device__ __forceinline__ float fine_weight(float d, Exponent x) {
  const float n = fmaxf(rintf(d * x.c), -150.0f);
  return ldexpf(__builtin_amdgcn_exp2f(__builtin_fmaf(d, x.low, __builtin_fmaf(d, x.c, -n))), int(n));
}

// Part of a row's softmax: the largest element so far, and relative to it the
// sum of weights exp(scale * (x - max)) and of weights times (x - max).  No
// element yet, or only minus infinity: max is that, the sums are 0.  A NaN or
// plus infinity anywhere makes the sum of weights NaN.  Threads add a
// piece's weights in 32 bits, in pairs, and the pieces in 64: sums of 100,000 in 32
// bits, or 32 small weights added to a 1 one after another, are off by as much as a
// loss near 0 is worth.
struct Partial {
  double sum;
  float max, mean;
};
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }
// p relative to `max`, which is p.max or above, by the factor f = weight of the distance
__device__ __forceinline__ Partial scaled(Partial p, float max, float d, float f) {
  return Partial{p.sum * double(f), max, f == 0.0f ? 0.0f : f * (p.mean + float(p.sum) * d)};  // (0 times minus infinity is to be 0)
}
__device__ __forceinline__ Partial relative(Partial p, float max, Exponent x) {
  const float d = p.max - finite_max(max);  // -inf where p has nothing
  return scaled(p, max, d, fine_weight(d, x));
}
// The wave's, and the workgroup's of WAVES waves (sh: room for them), in every thread.
__device__ __forceinline__ Partial wave_partial(Partial p, Exponent x) {
  p = relative(p, wave_max(p.max), x);
  p.sum = wave_sum(p.sum);
  p.mean = wave_sum(p.mean);
  return p;
}
template <uint32_t WAVES>
__device__ __forceinline__ Partial row_partial(Partial p, Exponent x, Partial *sh) {
  p = wave_partial(p, x);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = p;
  __syncthreads();
  float m = sh[0].max;
#pragma unroll
  for (uint32_t w = 1; w < WAVES; ++w) m = fmaxf(m, sh[w].max);
  Partial all{0.0, m, 0.0f};
#pragma unroll
  for (uint32_t w = 0; w < WAVES; ++w) {
    const Partial q = relative(sh[w], m, x);
    all.sum += q.sum;
    all.mean += q.mean;
  }
  return all;
}

// Calls f with a value of the element type.
template <typename F>
void with_element(int dtype, F f) {
  if (dtype == BBPE_BF16) f((__bf16)0);
  else if (dtype == BBPE_F16) f((_Float16)0);
  else f(0.0f);
}

// Pieces of a row that begins anywhere.
inline uint32_t most_pieces(int dtype, uint32_t vocab) {
  const uint32_t n = dtype == BBPE_F32 ? 4 : 8;
  return (vocab + 2 * (n - 1)) / n;
}

constexpr uint32_t PARTS_MAX = 64;         // parts of a row at most: a wave joins them
constexpr uint64_t MAX_GROUPS = 1u << 21;  // workgroups (of up to 1,024) a launch: fewer than 2^32 threads

// How rows are cut: waves a workgroup, parts a row and pieces of a part.
//
// Short rows go to a wave each (where `small` allows it), which has no barrier to wait
// at.  Up to 512 pieces always: from 1,024 rows on it is faster (2,048 rows of 2,048 in
// bfloat16: log probabilities 6.8 us, by workgroups of four waves 10.6, with 20
// alternatives 12.8 and 25.4; 8,192 rows 12.6 and 29.7, 26.6 and 76.3), and for fewer
// rows it is no slower with alternatives (1 row of 1,280: 8.5 us and 9.2; 512 rows: 10.2
// and 12.1) and the same without (5.4 and 5.4, 6.7 and 6.7), but for distillation of few
// rows near 512 pieces (1 row of 4,000: 5.6 and 5.0).  Up to 1,024 pieces where there are
// more than 1,024 rows: with alternatives workgroups win until there (rows of 5,003: 512
// rows 13.4 us and by waves 14.3, 1,000 15.7 and 15.3, 1,200 17.2 and 16.1, 1,536 24.9 and
// 16.6; of 8,184: 1,000 16.7 and 16.8, 1,536 25.0 and 18.4), and without until 1,536 or
// 2,048 (of 5,003: 1,200 8.8 and 9.4, 2,048 11.3 and 10.3; of 8,184: 1,200 9.2 and 10.7,
// 2,048 12.2 and 12.1, 8,192 38.5 and 31.1).
//
// Longer rows go to a workgroup each.  Up to 512 of them would not fill 256 CUs, and
// go to several, about 1,024 in all and no more than a row has steps, which a second
// kernel joins (1 row of 100,256: 8.8 us and, by one workgroup, 16; 400 rows: 25 us,
// with 800 workgroups 26.7, with 2,048 26.7); from 513 rows on the second kernel
// costs more (1,000 rows: by one each 43 us, by two 49, with 20 alternatives 51
// and 63).  Parts are equal, in 64 pieces, not whole steps: a last step may be nearly
// empty (128 rows of 200,005 in float32: 8 parts of six steps and 128 pieces).
struct Cut {
  uint32_t waves, parts, part;
};
inline Cut cut_rows(int dtype, uint64_t n_rows, uint32_t vocab, bool small, uint32_t most_parts) {
  const uint32_t per = dtype == BBPE_F32 ? 4 : 8, pieces = most_pieces(dtype, vocab);
  const bool few = n_rows <= 512, step = (vocab + per - 1) / per <= ROW_STEP;  // (a row within one, but for where it begins)
  Cut c{small && (pieces <= 512 || (step && n_rows > 1024)) ? 1u : ROW_WAVES, 1, 0};
  if (c.waves > 1 && n_rows && few && !step) {
    const uint64_t want = (1024 + n_rows - 1) / n_rows;
    uint64_t most = (pieces + ROW_STEP - 1) / ROW_STEP;
    most = most < PARTS_MAX ? most : PARTS_MAX;
    most = most < most_parts ? most : most_parts;
    c.parts = uint32_t(want < most ? want : most);
  }
  c.part = ((pieces + c.parts - 1) / c.parts + 63) / 64 * 64;
  c.parts = (pieces + c.part - 1) / c.part;  // (of parts rounded up, fewer may do)
  return c;
}

inline uintptr_t address(const void *p) { return reinterpret_cast<uintptr_t>(p); }

inline bool bad_sizes(int dtype, uint64_t rows, uint32_t vocab) {
  return dtype < BBPE_BF16 || dtype > BBPE_F32 || vocab == 0 || vocab > (1u << 30) || rows > 0x7FFFFFFFull;
}
// Scales whose two parts are ordinary floats.
inline bool bad_scale(float scale) { return !(scale >= 1e-30f && scale <= 1e30f); }
// What the operators ask of a matrix of logits alike.  `grad`: one of gradients,
// whose rows must not share memory.
inline bool bad_logits(int dtype, const void *x, int64_t stride, uint64_t rows, uint32_t vocab, bool grad) {
  if (bad_sizes(dtype, rows, vocab) || (rows && (!x || (address(x) & (dtype == BBPE_F32 ? 3 : 1))))) return true;
  return grad && rows > 1 && (stride < 0 ? -stride : stride) < int64_t(vocab);
}
// Whether a gradient's rows lie in the logits' other than each in its own place:
// workgroups would read what others have written.
inline bool crossing(int dtype, const void *x, int64_t x_stride, const void *dx, int64_t dx_stride, uint64_t rows, uint32_t vocab) {
  typedef __int128 wide;  // (strides are any numbers)
  const wide size = dtype == BBPE_F32 ? 4 : 2, row = vocab * size, xs = x_stride * size, ds = dx_stride * size, last = wide(rows) - 1;
  const wide d = wide(address(dx)) - wide(address(x));
  if (rows == 0 || (d == 0 && (rows == 1 || xs == ds))) return false;
  const wide x_from = xs < 0 ? last * xs : 0, x_to = (xs < 0 ? 0 : last * xs) + row;
  const wide d_from = d + (ds < 0 ? last * ds : 0), d_to = d + (ds < 0 ? 0 : last * ds) + row;
  if (x_to <= d_from || d_to <= x_from) return false;
  if (rows == 1 || xs != ds) return true;
  // rows that take turns with the other matrix's (a gradient's are a row apart at least)
  const wide s = xs < 0 ? -xs : xs, r = (d % s + s) % s;
  return r < row || r > s - row;
}

}  // namespace bbpe
