// The short way from Python to the operators of serving.py and scoring.py: plain calls (all
// tensors as documented, on the current device and stream) are checked, their
// outputs allocated and the library called here, in one step of a microsecond
// or two where ctypes and tensor methods take fifteen.  Whatever is not plain
// -- a stream, gradients to be recorded, tangents, a mistake -- returns NotImplemented,
// and the Python code, which says what is wrong, takes it from the start.
#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>

#include "../../include/bbpe.h"

namespace {

// The library's functions, from the handle that the package has opened.
decltype(&bbpe_block_tables) f_tables;
decltype(&bbpe_qk_norm_rope) f_norm;
decltype(&bbpe_qk_norm_rope_backward_workspace_bytes) f_back_bytes;
decltype(&bbpe_qk_norm_rope_backward) f_back;
decltype(&bbpe_tree_attention_workspace_bytes) f_attn_bytes;
decltype(&bbpe_tree_attention) f_attn;
decltype(&bbpe_token_logprobs_workspace_bytes) f_scores_bytes;
decltype(&bbpe_token_logprobs) f_scores;
decltype(&bbpe_token_logprobs_backward) f_scores_back;
decltype(&bbpe_distill_loss_workspace_bytes) f_distill_bytes;
decltype(&bbpe_distill_loss) f_distill;
decltype(&bbpe_distill_loss_backward) f_distill_back;

using at::Tensor;

struct Call {
  bool plain = true;
  int dev = -1;
  // a call whose inputs require grad is not plain, nor one whose inputs carry
  // tangents (torch has one level of them)
  bool recorded = c10::GradMode::is_enabled();
  const bool forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();

  // a tensor on the call's device; null where None is allowed and given
  const Tensor *tensor(PyObject *o, bool may_be_none = false) {
    if (o == Py_None) {
      if (!may_be_none) plain = false;
      return nullptr;
    }
    if (!THPVariable_Check(o)) {
      plain = false;
      return nullptr;
    }
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || (recorded && t.requires_grad()) || (forward && t._fw_grad(0).defined())) plain = false;
    else if (dev < 0) dev = t.get_device();
    else if (t.get_device() != dev) plain = false;
    return &t;
  }
  // contiguous, of this type and this many elements in one dimension (-1: any)
  void *flat(const Tensor *t, at::ScalarType type, int64_t n) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->dim() != 1 || (n >= 0 && t->size(0) != n) || !t->is_contiguous()) plain = false;
    return t->data_ptr();
  }
  // [n, heads, dim], the last dimension contiguous
  void *rows(const Tensor *t, at::ScalarType type, int64_t n, int64_t heads, int64_t dim) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->dim() != 3 || t->size(0) != n || t->size(1) != heads || t->size(2) != dim ||
        (dim > 1 && t->stride(2) != 1))
      plain = false;
    return t->data_ptr();
  }
  int64_t ts(const Tensor *t) const { return t && t->dim() == 3 ? t->stride(0) : 0; }
  int64_t hs(const Tensor *t) const { return t && t->dim() == 3 ? t->stride(1) : 0; }
  // contiguous, of this type and [n, m]
  void *dense(const Tensor *t, at::ScalarType type, int64_t n, int64_t m) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->dim() != 2 || t->size(0) != n || t->size(1) != m || !t->is_contiguous()) plain = false;
    return t->data_ptr();
  }
  void *table(const Tensor *t, int64_t n) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kInt || t->dim() != 2 || t->size(0) != n || (t->size(1) > 1 && t->stride(1) != 1)) plain = false;
    return t->data_ptr();
  }
  // everything is as it has to be, and on the current device: the stream to use
  bool ready(void *&stream) {
    if (!plain || dev < 0) return false;
    const c10::hip::HIPStream s = c10::hip::getCurrentHIPStream();
    if (s.device_index() != dev) return false;
    stream = s.stream();
    return true;
  }
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, dev)));
  }
};

// A one-dimensional tensor of n elements, `at` bytes into the buffer's storage.
Tensor part_of(const Tensor &buffer, int64_t at, int64_t n, at::ScalarType type) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at / int64_t(c10::elementSize(type)));
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// A call's outputs of four-byte elements, [n, width] or [n] (width -1), each in
// storage of its own: programs collect one and drop the others.  All that fit into the
// allocator's smallest block, which one by itself would take too, are in one (scores of
// 8 rows with 5 alternatives: 5.5 us of the host's time; of 64, apart, 7.1).
struct Output {
  at::ScalarType type;
  int64_t width;
};
template <size_t N>
std::array<Tensor, N> outputs(const Call &c, int64_t n, const Output (&want)[N]) {
  constexpr int64_t BLOCK = 512;
  std::array<Tensor, N> out;
  int64_t at[N + 1] = {0};
  for (size_t i = 0; i < N; ++i) at[i + 1] = at[i] + up16(4 * n * (want[i].width < 0 ? 1 : want[i].width));
  const bool together = at[N] <= BLOCK;
  const Tensor first = c.empty({together ? at[N] : at[1]}, at::kByte);
  c10::Allocator *const allocator = first.storage().allocator();
  for (size_t i = 0; i < N; ++i) {
    c10::Storage storage = first.storage();
    if (!together && i) {
      const size_t bytes = size_t(at[i + 1] - at[i]);
      storage = c10::Storage(c10::Storage::use_byte_size_t(), bytes, allocator->allocate(bytes), allocator, true);
    }
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(std::move(storage), first.key_set(), c10::scalarTypeToTypeMeta(want[i].type));
    if (together) t.unsafeGetTensorImpl()->set_storage_offset(at[i] / 4);
    if (want[i].width < 0) t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    else t.unsafeGetTensorImpl()->set_sizes_contiguous({n, want[i].width});
    out[i] = std::move(t);
  }
  return out;
}

int dtype_of(at::ScalarType t) { return t == at::kBFloat16 ? BBPE_BF16 : t == at::kHalf ? BBPE_F16 : t == at::kFloat ? BBPE_F32 : -1; }

PyObject *not_plain() { Py_RETURN_NOTIMPLEMENTED; }

// q_off, ctx_len, free_pages, table, page_size, n_tokens, depth -> (slots, positions, requests, seq_len, status)
PyObject *block_tables(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 7) return not_plain();
  Call c;
  const Tensor *q_off = c.tensor(a[0]), *ctx = c.tensor(a[1]), *free_pages = c.tensor(a[2]), *table = c.tensor(a[3]), *depth = c.tensor(a[6], true);
  const long long page = PyLong_AsLongLong(a[4]), n_tok = PyLong_AsLongLong(a[5]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_plain();
  }
  if (!c.plain || ctx->dim() != 1 || ctx->size(0) > 4096 || page <= 0 || page > (1 << 30) || n_tok < 0 || n_tok > 0x7FFFFFFF) return not_plain();
  const int64_t n = ctx->size(0);
  const void *p_off = c.flat(q_off, at::kLong, n + 1), *p_ctx = c.flat(ctx, at::kInt, n), *p_free = c.flat(free_pages, at::kInt, -1);
  const void *p_depth = c.flat(depth, at::kInt, n_tok);
  void *p_table = c.table(table, n), *stream;
  if (!c.ready(stream)) return not_plain();
  // the tokens' outputs, which live and die together, in one allocation; the
  // requests' in another: a program keeps seq_len as its next context lengths
  const int64_t at_pos = up16(8 * n_tok), at_req = at_pos + up16(4 * n_tok), at_seq = 32;
  const Tensor tokens = c.empty({at_req + 4 * n_tok}, at::kByte), requests = c.empty({at_seq + 4 * n}, at::kByte);
  Tensor slots = part_of(tokens, 0, n_tok, at::kLong), pos = part_of(tokens, at_pos, n_tok, at::kInt), req = part_of(tokens, at_req, n_tok, at::kInt),
         status = part_of(requests, 0, 4, at::kLong), seq = part_of(requests, at_seq, n, at::kInt);
  const int rc = f_tables(static_cast<const int64_t *>(p_off), static_cast<const int32_t *>(p_ctx), uint32_t(n),
                          static_cast<const int32_t *>(p_free), uint64_t(free_pages->size(0)), static_cast<int32_t *>(p_table),
                          uint64_t(table->stride(0)), uint32_t(table->size(1)), uint32_t(page), uint64_t(n_tok),
                          static_cast<const int32_t *>(p_depth), static_cast<int64_t *>(slots.data_ptr()),
                          static_cast<int32_t *>(pos.data_ptr()), static_cast<int32_t *>(req.data_ptr()),
                          static_cast<int32_t *>(seq.data_ptr()), static_cast<int64_t *>(status.data_ptr()), nullptr, 0, stream);
  if (rc) return not_plain();
  PyObject *out = PyTuple_New(5);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(slots)));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(pos)));
  PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(std::move(req)));
  PyTuple_SET_ITEM(out, 3, THPVariable_Wrap(std::move(seq)));
  PyTuple_SET_ITEM(out, 4, THPVariable_Wrap(std::move(status)));
  return out;
  END_HANDLE_TH_ERRORS
}

// What the norm's two directions take alike.
struct Norm {
  const Tensor *q, *k, *wq, *wk, *pos, *freq;
  at::ScalarType type;
  int64_t n, hq, hk, dim;
  void *p_q, *p_k, *p_wq, *p_wk, *p_pos, *p_freq;
  int inter;
  float eps;

  bool read(Call &c, PyObject *const *a, PyObject *o_eps, PyObject *o_inter) {
    q = c.tensor(a[0]);
    k = c.tensor(a[1]);
    wq = c.tensor(a[2], true);
    wk = c.tensor(a[3], true);
    pos = c.tensor(a[4]);
    freq = c.tensor(a[5]);
    if (!c.plain || q->dim() != 3 || k->dim() != 3) return false;
    type = q->scalar_type();
    if (dtype_of(type) < 0) return false;
    n = q->size(0);
    hq = q->size(1);
    hk = k->size(1);
    dim = q->size(2);
    p_q = c.rows(q, type, n, hq, dim);
    p_k = c.rows(k, type, n, hk, dim);
    p_wq = c.flat(wq, type, dim);
    p_wk = c.flat(wk, type, dim);
    p_pos = c.flat(pos, at::kInt, n);
    p_freq = c.flat(freq, at::kFloat, -1);
    eps = float(PyFloat_AsDouble(o_eps));
    inter = PyObject_IsTrue(o_inter);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    return c.plain;
  }
};

const bbpe_paged_cache *cache_of(PyObject *o) { return static_cast<const bbpe_paged_cache *>(PyLong_AsVoidPtr(o)); }

// q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, v, slots, cache.k, cache struct -> (q_out, k_out)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 12) return not_plain();
  Call c;
  Norm m;
  if (!m.read(c, a, a[6], a[7])) return not_plain();
  const Tensor *v = c.tensor(a[8], true), *slots = c.tensor(a[9], true), *ck = c.tensor(a[10], true);
  if (!c.plain || (v == nullptr) != (ck == nullptr) || (slots == nullptr) != (ck == nullptr)) return not_plain();
  const bbpe_paged_cache *cache = nullptr;
  if (ck) {
    cache = cache_of(a[11]);
    if (!cache || ck->scalar_type() != m.type) {
      PyErr_Clear();
      return not_plain();
    }
  }
  const void *p_v = c.rows(v, m.type, m.n, m.hk, m.dim), *p_slots = c.flat(slots, at::kLong, m.n);
  void *stream;
  if (!c.ready(stream)) return not_plain();
  Tensor q_out = c.empty({m.n, m.hq, m.dim}, m.type), k_out;
  if (!ck) k_out = c.empty({m.n, m.hk, m.dim}, m.type);
  const int rc = f_norm(dtype_of(m.type), uint64_t(m.n), uint32_t(m.hq), uint32_t(m.hk), uint32_t(m.dim), uint32_t(2 * m.freq->size(0)), m.inter, m.eps,
                        m.p_q, c.ts(m.q), c.hs(m.q), m.p_k, c.ts(m.k), c.hs(m.k), p_v, c.ts(v), c.hs(v), m.p_wq, m.p_wk,
                        static_cast<const int32_t *>(m.p_pos), static_cast<const float *>(m.p_freq), q_out.data_ptr(), m.hq * m.dim, m.dim,
                        ck ? nullptr : k_out.data_ptr(), m.hk * m.dim, m.dim, cache, static_cast<const int64_t *>(p_slots), stream);
  if (rc) return not_plain();
  PyObject *out = PyTuple_New(2);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(q_out)));
  if (ck) Py_INCREF(Py_None);
  PyTuple_SET_ITEM(out, 1, ck ? Py_None : THPVariable_Wrap(std::move(k_out)));
  return out;
  END_HANDLE_TH_ERRORS
}

// q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, grad_q, grad_k -> (dq, dk, dq_weight, dk_weight)
PyObject *qk_norm_rope_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 10) return not_plain();
  Call c;
  c.recorded = false;  // (a gradient's inputs may require grad; it is not differentiated again)
  Norm m;
  if (!m.read(c, a, a[6], a[7])) return not_plain();
  const Tensor *gq = c.tensor(a[8]), *gk = c.tensor(a[9]);
  if (!c.plain) return not_plain();
  const void *p_gq = c.rows(gq, m.type, m.n, m.hq, m.dim), *p_gk = c.rows(gk, m.type, m.n, m.hk, m.dim);
  void *stream;
  uint64_t bytes = 0;
  if (!c.ready(stream) || f_back_bytes(uint64_t(m.n), uint32_t(m.dim), &bytes)) return not_plain();
  Tensor dq = c.empty({m.n, m.hq, m.dim}, m.type), dk = c.empty({m.n, m.hk, m.dim}, m.type), dwq, dwk;
  if (m.wq || m.wk) {
    const Tensor both = c.empty({8 * m.dim}, at::kByte);
    if (m.wq) dwq = part_of(both, 0, m.dim, at::kFloat);
    if (m.wk) dwk = part_of(both, 4 * m.dim, m.dim, at::kFloat);
  }
  const Tensor ws = c.empty({int64_t(bytes)}, at::kByte);
  const int rc = f_back(dtype_of(m.type), uint64_t(m.n), uint32_t(m.hq), uint32_t(m.hk), uint32_t(m.dim), uint32_t(2 * m.freq->size(0)), m.inter, m.eps,
                        p_gq, c.ts(gq), c.hs(gq), p_gk, c.ts(gk), c.hs(gk), m.p_q, c.ts(m.q), c.hs(m.q), m.p_k, c.ts(m.k), c.hs(m.k), m.p_wq, m.p_wk,
                        static_cast<const int32_t *>(m.p_pos), static_cast<const float *>(m.p_freq), dq.data_ptr(), m.hq * m.dim, m.dim, dk.data_ptr(),
                        m.hk * m.dim, m.dim, m.wq ? static_cast<float *>(dwq.data_ptr()) : nullptr,
                        m.wk ? static_cast<float *>(dwk.data_ptr()) : nullptr, ws.data_ptr(), bytes, stream);
  if (rc) return not_plain();
  PyObject *out = PyTuple_New(4);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(dq)));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(dk)));
  for (int i = 0; i < 2; ++i) {
    Tensor &w = i ? dwk : dwq;
    const bool some = i ? m.wk != nullptr : m.wq != nullptr;
    if (!some) Py_INCREF(Py_None);
    PyTuple_SET_ITEM(out, 2 + i, some ? THPVariable_Wrap(std::move(w)) : Py_None);
  }
  return out;
  END_HANDLE_TH_ERRORS
}

// q, cache.k, cache struct, table, q_off, ctx_len, tree_mask, scale, lse wanted -> (out, lse or None)
PyObject *tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 9) return not_plain();
  Call c;
  const Tensor *q = c.tensor(a[0]), *ck = c.tensor(a[1]), *table = c.tensor(a[3]), *q_off = c.tensor(a[4]), *ctx = c.tensor(a[5]),
               *mask = c.tensor(a[6], true);
  const bbpe_paged_cache *cache = cache_of(a[2]);
  const float scale = float(PyFloat_AsDouble(a[7]));
  const int with_lse = PyObject_IsTrue(a[8]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_plain();
  }
  if (!c.plain || !cache || q->dim() != 3 || q->scalar_type() != ck->scalar_type() || q->size(2) != int64_t(cache->head_dim) || ctx->dim() != 1)
    return not_plain();
  const at::ScalarType type = q->scalar_type();
  const int64_t n = q->size(0), hq = q->size(1), dim = q->size(2), reqs = ctx->size(0);
  const void *p_q = c.rows(q, type, n, hq, dim), *p_off = c.flat(q_off, at::kLong, reqs + 1), *p_ctx = c.flat(ctx, at::kInt, reqs);
  const void *p_table = c.table(table, reqs), *p_mask = nullptr;
  if (mask) {
    if (mask->scalar_type() != at::kLong || mask->dim() != 2 || mask->size(0) != n || !mask->is_contiguous()) return not_plain();
    p_mask = mask->data_ptr();
  }
  void *stream;
  uint64_t bytes = 0;
  if (!c.ready(stream) || f_attn_bytes(uint64_t(n), uint32_t(reqs), uint32_t(hq), cache, &bytes)) return not_plain();
  Tensor out = c.empty({n, hq, dim}, type), lse;
  if (with_lse) lse = c.empty({n, hq}, at::kFloat);
  const Tensor ws = c.empty({int64_t(bytes)}, at::kByte);
  const int rc = f_attn(p_q, c.ts(q), c.hs(q), uint64_t(n), uint32_t(hq), cache, static_cast<const int32_t *>(p_table), uint64_t(table->stride(0)),
                        uint32_t(table->size(1)), static_cast<const int64_t *>(p_off), static_cast<const int32_t *>(p_ctx), uint32_t(reqs),
                        static_cast<const uint64_t *>(p_mask), mask ? uint32_t(mask->size(1)) : 0, scale, out.data_ptr(), hq * dim, dim,
                        with_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, ws.data_ptr(), bytes, stream);
  if (rc) return not_plain();
  PyObject *o = PyTuple_New(2);
  if (!o) return nullptr;
  PyTuple_SET_ITEM(o, 0, THPVariable_Wrap(std::move(out)));
  if (!with_lse) Py_INCREF(Py_None);
  PyTuple_SET_ITEM(o, 1, with_lse ? THPVariable_Wrap(std::move(lse)) : Py_None);
  return o;
  END_HANDLE_TH_ERRORS
}

// Rows of logits, or of their gradients.
struct Logits {
  const Tensor *t;
  at::ScalarType type;
  int64_t n, vocab;
  void *p;

  bool read(Call &c, PyObject *o) {
    t = c.tensor(o);
    if (!c.plain || t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1) || t->size(1) > 0x7FFFFFFF) return false;
    type = t->scalar_type();
    n = t->size(0);
    vocab = t->size(1);
    p = t->data_ptr();
    return dtype_of(type) >= 0;
  }
  bool like(Call &c, PyObject *o, const Logits &x) {
    return read(c, o) && type == x.type && n == x.n && vocab == x.vocab && (n <= 1 || t->stride(0) >= vocab);
  }
};

template <size_t N>
PyObject *tuple_of(const std::array<Tensor, N> &ts) {
  PyObject *out = PyTuple_New(Py_ssize_t(N));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor &t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}

float *floats(void *p) { return static_cast<float *>(p); }
int32_t *ints(void *p) { return static_cast<int32_t *>(p); }

// logits, ids, top_k, scale -> (logprobs, entropy, lse, ranks, top_ids, top_logprobs, stats)
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 4) return not_plain();
  Call c;
  Logits x;
  if (!x.read(c, a[0])) return not_plain();
  const Tensor *ids = c.tensor(a[1]);
  const int64_t k = PyLong_AsLongLong(a[2]), n = x.n;
  const float scale = float(PyFloat_AsDouble(a[3]));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_plain();
  }
  if (!c.plain || k < 0 || k > 256 || k > x.vocab) return not_plain();
  void *p_ids = c.flat(ids, at::kInt, n), *stream;
  if (!c.ready(stream)) return not_plain();
  uint64_t bytes = 0;
  if (f_scores_bytes(dtype_of(x.type), uint64_t(n), uint32_t(x.vocab), uint32_t(k), &bytes)) return not_plain();
  Tensor ws;
  if (bytes) ws = c.empty({int64_t(bytes)}, at::kByte);
  const auto out = outputs<7>(c, n, {{at::kFloat, -1}, {at::kFloat, -1}, {at::kFloat, -1}, {at::kInt, -1}, {at::kInt, k}, {at::kFloat, k}, {at::kFloat, 2}});
  const int rc = f_scores(dtype_of(x.type), x.p, x.t->stride(0), uint64_t(n), uint32_t(x.vocab), ints(p_ids), uint32_t(k), scale,
                          floats(out[0].data_ptr()), floats(out[1].data_ptr()), floats(out[2].data_ptr()), ints(out[3].data_ptr()), ints(out[4].data_ptr()),
                          floats(out[5].data_ptr()), floats(out[6].data_ptr()), bytes ? ws.data_ptr() : nullptr, bytes, stream);
  if (rc) return not_plain();
  return tuple_of(out);
  END_HANDLE_TH_ERRORS
}

// logits, ids, entropy, top_ids, stats, grad_logprobs, grad_entropy, grad_lse, grad_top, scale -> dlogits
PyObject *token_logprobs_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 10) return not_plain();
  Call c;
  c.recorded = false;  // (a gradient's inputs may require grad; it is not differentiated again)
  Logits x;
  if (!x.read(c, a[0])) return not_plain();
  const Tensor *ids = c.tensor(a[1]), *entropy = c.tensor(a[2]), *top_ids = c.tensor(a[3]), *stats = c.tensor(a[4]);
  const Tensor *g[4];
  for (int i = 0; i < 4; ++i) g[i] = c.tensor(a[5 + i], true);
  const float scale = float(PyFloat_AsDouble(a[9]));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_plain();
  }
  if (!c.plain || top_ids->dim() != 2) return not_plain();
  const int64_t n = x.n, k = top_ids->size(1);
  void *p_ids = c.flat(ids, at::kInt, n), *p_entropy = c.flat(entropy, at::kFloat, n), *p_top = c.dense(top_ids, at::kInt, n, k),
       *p_stats = c.dense(stats, at::kFloat, n, 2), *p_g[4], *stream;
  for (int i = 0; i < 3; ++i) p_g[i] = c.flat(g[i], at::kFloat, n);
  p_g[3] = c.dense(g[3], at::kFloat, n, k);
  if (!c.ready(stream)) return not_plain();
  Tensor dx = c.empty({n, x.vocab}, x.type);
  const int rc = f_scores_back(dtype_of(x.type), x.p, x.t->stride(0), uint64_t(n), uint32_t(x.vocab), ints(p_ids), uint32_t(k), scale, floats(p_entropy),
                               ints(p_top), floats(p_stats), floats(p_g[0]), floats(p_g[1]), floats(p_g[2]), floats(p_g[3]), dx.data_ptr(), x.vocab, stream);
  if (rc) return not_plain();
  return THPVariable_Wrap(std::move(dx));
  END_HANDLE_TH_ERRORS
}

// The lists of a distillation: [n, k] ids and log probabilities.
struct Lists {
  int64_t k;
  void *p_ids, *p_lp;

  bool read(Call &c, PyObject *ids, PyObject *lp, int64_t n) {
    const Tensor *t = c.tensor(ids), *l = c.tensor(lp);
    if (!c.plain || t->dim() != 2) return false;
    k = t->size(1);
    p_ids = c.dense(t, at::kInt, n, k);
    p_lp = c.dense(l, at::kFloat, n, k);
    return c.plain && k <= 256;
  }
};

// logits, top_ids, top_logprobs, tail, scale, weights, dlogits -> (loss, lse, stats)
PyObject *distill_loss(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 7) return not_plain();
  Call c;
  Logits x, d;
  Lists l;
  if (!x.read(c, a[0]) || !l.read(c, a[1], a[2], x.n)) return not_plain();
  const int tail = PyObject_IsTrue(a[3]);
  const float scale = float(PyFloat_AsDouble(a[4]));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_plain();
  }
  const Tensor *weights = c.tensor(a[5], true);
  if (!c.plain || (weights && !d.like(c, a[6], x))) return not_plain();
  const int64_t n = x.n;
  void *p_w = c.flat(weights, at::kFloat, n), *stream;
  uint64_t bytes = 0;
  if (!c.ready(stream) || f_distill_bytes(dtype_of(x.type), uint64_t(n), uint32_t(x.vocab), &bytes)) return not_plain();
  Tensor ws;
  if (bytes) ws = c.empty({int64_t(bytes)}, at::kByte);
  const auto out = outputs<3>(c, n, {{at::kFloat, -1}, {at::kFloat, -1}, {at::kFloat, 4}});
  const int rc = f_distill(dtype_of(x.type), x.p, x.t->stride(0), uint64_t(n), uint32_t(x.vocab), ints(l.p_ids), floats(l.p_lp), uint32_t(l.k), tail, scale,
                           floats(out[0].data_ptr()), floats(out[1].data_ptr()), floats(out[2].data_ptr()), floats(p_w), weights ? d.p : nullptr,
                           weights ? d.t->stride(0) : 0, bytes ? ws.data_ptr() : nullptr, bytes, stream);
  if (rc) return not_plain();
  // (as torch's own writes into a given tensor do: who has saved it for a backward pass learns of it)
  if (weights && !d.t->is_inference()) d.t->unsafeGetTensorImpl()->bump_version();
  return tuple_of(out);
  END_HANDLE_TH_ERRORS
}

// grad_loss, logits, top_ids, top_logprobs, stats, tail, scale -> dlogits
PyObject *distill_loss_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 7) return not_plain();
  Call c;
  c.recorded = false;  // (a gradient's inputs may require grad; it is not differentiated again)
  Logits x;
  Lists l;
  if (!x.read(c, a[1]) || !l.read(c, a[2], a[3], x.n)) return not_plain();
  const Tensor *grad = c.tensor(a[0]), *stats = c.tensor(a[4]);
  const int tail = PyObject_IsTrue(a[5]);
  const float scale = float(PyFloat_AsDouble(a[6]));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_plain();
  }
  if (!c.plain) return not_plain();
  const int64_t n = x.n;
  void *p_grad = c.flat(grad, at::kFloat, n), *p_stats = c.dense(stats, at::kFloat, n, 4), *stream;
  if (!c.ready(stream)) return not_plain();
  Tensor dx = c.empty({n, x.vocab}, x.type);
  const int rc = f_distill_back(dtype_of(x.type), x.p, x.t->stride(0), uint64_t(n), uint32_t(x.vocab), ints(l.p_ids), floats(l.p_lp), uint32_t(l.k), tail,
                                scale, floats(p_stats), floats(p_grad), dx.data_ptr(), x.vocab, stream);
  if (rc) return not_plain();
  return THPVariable_Wrap(std::move(dx));
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the twelve functions above, in their order)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  constexpr int N = 12;
  if (n_args != N) {
    PyErr_SetString(PyExc_TypeError, "bind: twelve addresses");
    return nullptr;
  }
  void *p[N];
  for (int i = 0; i < N; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  f_tables = reinterpret_cast<decltype(f_tables)>(p[0]);
  f_norm = reinterpret_cast<decltype(f_norm)>(p[1]);
  f_back_bytes = reinterpret_cast<decltype(f_back_bytes)>(p[2]);
  f_back = reinterpret_cast<decltype(f_back)>(p[3]);
  f_attn_bytes = reinterpret_cast<decltype(f_attn_bytes)>(p[4]);
  f_attn = reinterpret_cast<decltype(f_attn)>(p[5]);
  f_scores_bytes = reinterpret_cast<decltype(f_scores_bytes)>(p[6]);
  f_scores = reinterpret_cast<decltype(f_scores)>(p[7]);
  f_scores_back = reinterpret_cast<decltype(f_scores_back)>(p[8]);
  f_distill_bytes = reinterpret_cast<decltype(f_distill_bytes)>(p[9]);
  f_distill = reinterpret_cast<decltype(f_distill)>(p[10]);
  f_distill_back = reinterpret_cast<decltype(f_distill_back)>(p[11]);
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),
                         METHOD(block_tables),
                         METHOD(qk_norm_rope),
                         METHOD(qk_norm_rope_backward),
                         METHOD(tree_attention),
                         METHOD(token_logprobs),
                         METHOD(token_logprobs_backward),
                         METHOD(distill_loss),
                         METHOD(distill_loss_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
