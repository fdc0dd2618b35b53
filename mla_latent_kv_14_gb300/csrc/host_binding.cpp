// host_binding.cpp -- the Python side of the calls around the decode (appends,
// rotation, norms, index rows, index score, selection, rows read back, the
// attention of prompts): checks of the tensors, their
// device and stream, allocation of outputs, and the call of the C entry point.
//
// These calls take one to a few microseconds on the GPU at a decode step's
// sizes. Written in Python over ctypes, their checks took 8 to 17 us a call on
// the host; as an extension module they take about the launch itself.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <optional>

#include "../../include/mla.h"

namespace {

PyObject* g_error = nullptr;  // MLAError(status, where)

struct Raised {};  // a Python error is set

[[noreturn]] void raise(int status, const char* text) {
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", status, text) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, text);
  }
  throw Raised();
}

// the interpreter's lock given up for a scope
class Unlocked {
  PyThreadState* state_ = PyEval_SaveThread();

 public:
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state_); }
};

// One call: its name, for messages, and the device that its tensors are on.
struct Call {
  const char* where;
  int dev = -1;

  [[noreturn]] void refuse(const char* format, ...) const {
    char text[256];
    const int n = snprintf(text, sizeof text, "%s: ", where);
    va_list a;
    va_start(a, format);
    vsnprintf(text + n, sizeof text - n, format, a);
    va_end(a);
    raise(MLA_ERR_INVALID_ARG, text);
  }
  const at::Tensor& tensor(PyObject* o, const char* name) const {
    if (!THPVariable_Check(o)) refuse("%s: a tensor", name);
    return THPVariable_Unpack(o);
  }
  int64_t integer(PyObject* o, const char* name, int64_t low = INT32_MIN, int64_t high = INT32_MAX) const {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (v < low || v > high) refuse("%s out of range", name);
    return v;
  }
  // the first tensor settles the device, the others have to share it
  void on_device(const at::Tensor& t) {
    const int d = t.is_cuda() ? t.get_device() : -1;
    if (d < 0 || (dev >= 0 && d != dev)) refuse("tensors of one cuda device");
    dev = d;
  }
  void* status(PyObject* o) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, "status");
    on_device(t);
    if (t.nbytes() < 4) refuse("status: a 4-byte word");
    return t.data_ptr();
  }
  // The launch runs without the interpreter's lock: one into a full queue waits for the GPU, and the other Python
  // threads must not wait with it. `f` touches no Python object; the caller's arguments outlive the call.
  template <typename F>
  void run(F&& f) const {
    int st;
    {
      const Unlocked unlocked;
      const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
      st = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream()));
    }
    if (st != MLA_OK) raise(st, where);
  }
};

bool is_shape(const at::Tensor& t, std::initializer_list<int64_t> s) { return t.sizes() == c10::IntArrayRef(s); }
int dtype_code(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? MLA_DTYPE_BF16 : t.scalar_type() == at::kHalf ? MLA_DTYPE_FP16 : -1;
}
bool is_e4m3(const at::Tensor& t) { return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte; }
// the stride of a dim; of one with at most one entry, which is never stepped
// over, the dense one (any number may stand there)
int64_t stride_of(const at::Tensor& t, int64_t dim, int64_t dense) { return t.size(dim) > 1 ? t.stride(dim) : dense; }

const int32_t* int32_vector(Call& c, PyObject* o, const char* name, int64_t n) {
  const at::Tensor& t = c.tensor(o, name);
  if (t.scalar_type() != at::kInt || !is_shape(t, {n}) || !t.is_contiguous()) c.refuse("%s: int32 [%lld]", name, (long long)n);
  c.on_device(t);
  return static_cast<const int32_t*>(t.data_ptr());
}

struct Rope {
  const int32_t* positions;
  const float* table;
  int64_t rows;
  int style;
  Rope(Call& c, PyObject* pos, PyObject* tab, PyObject* sty, int64_t tokens) {
    positions = int32_vector(c, pos, "positions", tokens);
    const at::Tensor& t = c.tensor(tab, "rope_table");
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(1) != 64 || !t.is_contiguous())
      c.refuse("rope_table: fp32 [positions, 64]");
    c.on_device(t);
    table = static_cast<const float*>(t.data_ptr());
    rows = t.size(0);
    style = (int)c.integer(sty, "rope_style");
  }
};

// A row-paged cache [num_blocks, page_block, ..., row] in one piece.
struct Cache {
  void* data;
  int64_t blocks;
  int page;
  Cache(Call& c, PyObject* o, const char* name, int64_t row, at::ScalarType type) {
    const at::Tensor& t = c.tensor(o, name);
    if (t.scalar_type() != type || t.dim() < 3 || t.size(-1) != row || !t.is_contiguous() ||
        t.numel() != t.size(0) * t.size(1) * row || t.size(1) > INT32_MAX)
      c.refuse("%s: contiguous [num_blocks, page_block, 1, %lld] of %s", name, (long long)row, c10::toString(type));
    c.on_device(t);
    data = t.data_ptr();
    blocks = t.size(0);
    page = (int)t.size(1);
  }
  // the index cache of a format (16-bit: of `type`)
  Cache(Call& c, PyObject* o, int64_t format, at::ScalarType type) {
    if (format == MLA_INDEX_16BIT) {
      *this = Cache(c, o, "index_cache", MLA_INDEX_DIM, type);
      return;
    }
    if (format != MLA_INDEX_FP8) c.refuse("unknown index_format");
    const at::Tensor& t = c.tensor(o, "index_cache");
    if (t.scalar_type() != at::kByte || t.dim() != 2 || t.size(1) != MLA_INDEX_FP8_PAGE_BYTES || !t.is_contiguous())
      c.refuse("index_cache: contiguous uint8 [num_blocks, %d] (FP8)", MLA_INDEX_FP8_PAGE_BYTES);
    c.on_device(t);
    data = t.data_ptr();
    blocks = t.size(0);
    page = 64;
  }
};

// block_table [batch, max_blocks] and cache_seqlens [batch]
struct Paged {
  const int32_t *table, *seqlens;
  int max_blocks;
  Paged(Call& c, PyObject* bt, PyObject* sl, int64_t batch) {
    const at::Tensor& t = c.tensor(bt, "block_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != batch || !t.is_contiguous() || t.size(1) > INT32_MAX)
      c.refuse("block_table: int32 [%lld, max_blocks]", (long long)batch);
    c.on_device(t);
    table = static_cast<const int32_t*>(t.data_ptr());
    max_blocks = (int)t.size(1);
    seqlens = int32_vector(c, sl, "cache_seqlens", batch);
  }
};

// rows of scores [B, s_q, width], equally spaced (a column range of a wider buffer is fine)
int64_t score_stride(const Call& c, const at::Tensor& t, int64_t width) {
  if (t.is_contiguous()) return width;
  const int64_t batch = t.size(0), s_q = t.size(1);
  const int64_t stride = s_q > 1 ? t.stride(1) : batch > 1 ? t.stride(0) : width;
  if ((width > 1 && t.stride(2) != 1) || (batch > 1 && s_q > 1 && t.stride(0) != s_q * stride))
    c.refuse("rows of scores dense and equally spaced");
  return stride;
}

// a new tensor, straight from the allocator (0.2 us less than a dispatched empty, where a call with two outputs takes
// the host 3.9 us)
at::Tensor fresh(c10::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// an output: the caller's (None: a new one), of a type and shape
at::Tensor output(Call& c, PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
                  const at::Tensor& like) {
  if (o == Py_None) return fresh(c10::IntArrayRef(shape), type, like);
  const at::Tensor& t = c.tensor(o, name);
  if (t.scalar_type() != type || !is_shape(t, shape) || !t.is_contiguous())
    c.refuse("%s: contiguous %s of the result's shape", name, c10::toString(type));
  c.on_device(t);
  return t;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// (c_kv, k_rope, kvcache, slots, positions, rope_table, kv_format, rope_style, status)
PyObject* append_kv(Call& c, PyObject* const* a) {
  const int64_t format = c.integer(a[6], "kv_format");
  static constexpr int64_t rows[4] = {MLA_HEAD_DIM_K, MLA_FP8_ROW_BYTES, MLA_FP8_528_ROW_BYTES, MLA_FP4_288_ROW_BYTES};
  if (format < 0 || format > 3) c.refuse("unknown kv_format %lld", (long long)format);
  const at::Tensor &kv = c.tensor(a[0], "c_kv"), &kr = c.tensor(a[1], "k_rope");
  const int64_t latent = format >= MLA_KV_FP8_528 ? 448 : 512, n = kv.dim() ? kv.size(0) : 0;
  const int code = dtype_code(kv);
  if (code < 0 || !is_shape(kv, {n, latent}) || !is_shape(kr, {n, 64}) || kr.scalar_type() != kv.scalar_type() ||
      kv.stride(1) != 1 || kr.stride(1) != 1)
    c.refuse("c_kv [n, %lld] and k_rope [n, 64], bf16 or fp16", (long long)latent);
  c.on_device(kv);
  c.on_device(kr);
  const Cache cache(c, a[2], "kvcache", rows[format], format ? at::kByte : kv.scalar_type());
  const int32_t* slots = int32_vector(c, a[3], "slots", n);
  const Rope r(c, a[4], a[5], a[7], n);
  auto* st = static_cast<uint32_t*>(c.status(a[8]));
  c.run([&](void* stream) {
    return mla_append_kv(kv.data_ptr(), stride_of(kv, 0, latent), kr.data_ptr(), stride_of(kr, 0, 64), code, slots,
                         r.positions, r.table, r.rows, r.style, n, cache.data, cache.blocks, cache.page, (int)format,
                         st, stream);
  });
  Py_INCREF(a[2]);
  return a[2];
}

// (x, positions, rope_table, out, rope_style, status)
PyObject* rotate_q(Call& c, PyObject* const* a) {
  const at::Tensor& x = c.tensor(a[0], "x");
  const int code = dtype_code(x);
  if (code < 0 || x.dim() != 3 || x.size(2) != 64 || x.stride(2) != 1)
    c.refuse("x [tokens, heads, 64], bf16 or fp16");
  const int64_t tokens = x.size(0), heads = x.size(1);
  if (heads > INT32_MAX) c.refuse("heads out of range");
  c.on_device(x);
  const at::Tensor out = a[3] == Py_None ? fresh(x.sizes(), x.scalar_type(), x) : c.tensor(a[3], "out");
  if (out.sizes() != x.sizes() || out.scalar_type() != x.scalar_type() || out.stride(2) != 1) c.refuse("out like x");
  c.on_device(out);
  const Rope r(c, a[1], a[2], a[4], tokens);
  auto* st = static_cast<uint32_t*>(c.status(a[5]));
  c.run([&](void* stream) {
    return mla_rotate_q(x.data_ptr(), stride_of(x, 0, 64 * heads), stride_of(x, 1, 64), out.data_ptr(),
                        stride_of(out, 0, 64 * heads), stride_of(out, 1, 64), code, r.positions, r.table, r.rows,
                        r.style, tokens, (int)heads, st, stream);
  });
  if (a[3] == Py_None) return THPVariable_Wrap(out);
  Py_INCREF(a[3]);
  return a[3];
}

// (k, index_cache, slots, positions, rope_table, index_format, rope_style, status)
PyObject* append_index_k(Call& c, PyObject* const* a) {
  const at::Tensor& k = c.tensor(a[0], "k");
  const int64_t format = c.integer(a[5], "index_format"), n = k.dim() ? k.size(0) : 0;
  const int code = dtype_code(k);
  if (code < 0 || !is_shape(k, {n, MLA_INDEX_DIM}) || k.stride(1) != 1) c.refuse("k [n, 128], bf16 or fp16");
  c.on_device(k);
  const Cache cache(c, a[1], format, k.scalar_type());
  const int32_t* slots = int32_vector(c, a[2], "slots", n);
  const Rope r(c, a[3], a[4], a[6], n);
  auto* st = static_cast<uint32_t*>(c.status(a[7]));
  c.run([&](void* stream) {
    return mla_append_index_k(k.data_ptr(), stride_of(k, 0, MLA_INDEX_DIM), code, slots, r.positions, r.table, r.rows,
                              r.style, n, cache.data, cache.blocks, cache.page, (int)format, st, stream);
  });
  Py_INCREF(a[1]);
  return a[1];
}

// (q, weights, positions, rope_table, rope_style, q_out, weights_out, status)
PyObject* quantize_index_q(Call& c, PyObject* const* a) {
  const at::Tensor &q = c.tensor(a[0], "q"), &w = c.tensor(a[1], "weights");
  const int code = dtype_code(q);
  if (code < 0 || q.dim() != 3 || q.size(2) != MLA_INDEX_DIM || q.stride(2) != 1)
    c.refuse("q [tokens, heads, 128], bf16 or fp16");
  const int64_t tokens = q.size(0), heads = q.size(1);
  if (heads > INT32_MAX) c.refuse("heads out of range");
  if (w.scalar_type() != at::kFloat || !is_shape(w, {tokens, heads}) || !w.is_contiguous())
    c.refuse("weights: contiguous fp32 [tokens, heads]");
  c.on_device(q);
  c.on_device(w);
  const bool bytes = a[5] != Py_None && THPVariable_Check(a[5]) && THPVariable_Unpack(a[5]).scalar_type() == at::kByte;
  const at::Tensor q_out = output(c, a[5], "q_out", bytes ? at::kByte : at::kFloat8_e4m3fn, {tokens, heads, MLA_INDEX_DIM}, q);
  const at::Tensor w_out = output(c, a[6], "weights_out", at::kFloat, {tokens, heads}, w);
  const Rope r(c, a[2], a[3], a[4], tokens);
  auto* st = static_cast<uint32_t*>(c.status(a[7]));
  c.run([&](void* stream) {
    return mla_quantize_index_q(q.data_ptr(), stride_of(q, 0, MLA_INDEX_DIM * heads), stride_of(q, 1, MLA_INDEX_DIM),
                                code, static_cast<const float*>(w.data_ptr()), r.positions, r.table, r.rows, r.style,
                                tokens, (int)heads, static_cast<uint8_t*>(q_out.data_ptr()),
                                static_cast<float*>(w_out.data_ptr()), st, stream);
  });
  return pair(q_out, w_out);
}

// (q, weights, index_cache, block_table, cache_seqlens, width, causal, block, index_format, scores, status)
PyObject* index_score(Call& c, PyObject* const* a) {
  const at::Tensor &q = c.tensor(a[0], "q"), &w = c.tensor(a[1], "weights");
  const int64_t format = c.integer(a[8], "index_format"), block = c.integer(a[7], "block");
  if (q.dim() != 4 || q.size(3) != MLA_INDEX_DIM || !q.is_contiguous()) c.refuse("q: contiguous [B, s_q, heads, 128]");
  const int64_t batch = q.size(0), s_q = q.size(1), heads = q.size(2);
  if (batch > INT32_MAX || s_q > INT32_MAX || heads > INT32_MAX) c.refuse("q's sizes out of range");
  const int code = format == MLA_INDEX_FP8 ? (is_e4m3(q) ? 0 : -1) : dtype_code(q);
  if (code < 0) c.refuse("q's type: that of the index cache, e4m3 with an FP8 one");
  if (w.scalar_type() != at::kFloat || !is_shape(w, {batch, s_q, heads}) || !w.is_contiguous())
    c.refuse("weights: contiguous fp32 [B, s_q, heads]");
  c.on_device(q);
  c.on_device(w);
  const Cache cache(c, a[2], format, q.scalar_type());
  const Paged paged(c, a[3], a[4], batch);
  if (block != 1 && block != 64) c.refuse("block 1 or 64");
  const int causal = PyObject_IsTrue(a[6]);
  if (causal < 0) throw Raised();
  const bool given = a[9] != Py_None;
  int64_t width = (int64_t)paged.max_blocks * (64 / block);
  if (a[5] != Py_None) width = c.integer(a[5], "width", 1);
  else if (given && c.tensor(a[9], "scores").dim()) width = c.tensor(a[9], "scores").size(-1);
  if (width < 1 || width > INT32_MAX) c.refuse("width out of range");
  const at::Tensor scores = given ? c.tensor(a[9], "scores") : fresh({batch, s_q, width}, at::kFloat, w);
  int64_t stride = width;
  if (given) {
    if (scores.scalar_type() != at::kFloat || !is_shape(scores, {batch, s_q, width}))
      c.refuse("scores: fp32 [B, s_q, width]");
    c.on_device(scores);
    stride = score_stride(c, scores, width);
  }
  auto* st = static_cast<uint32_t*>(c.status(a[10]));
  c.run([&](void* stream) {
    return mla_index_score(q.data_ptr(), code, static_cast<const float*>(w.data_ptr()), cache.data, (int)format,
                           cache.blocks, cache.page, paged.table, paged.max_blocks, paged.seqlens, (int)batch, (int)s_q,
                           (int)heads, causal, (int)block, static_cast<float*>(scores.data_ptr()), stride, (int)width, st,
                           stream);
  });
  if (!given) return THPVariable_Wrap(scores);
  Py_INCREF(a[9]);
  return a[9];
}

// (scores, cache_seqlens, topk, block_table, num_blocks, causal, block, indices, lens, status)
PyObject* select_topk(Call& c, PyObject* const* a) {
  const at::Tensor& s = c.tensor(a[0], "scores");
  if (s.dim() != 3 || s.scalar_type() != at::kFloat) c.refuse("scores: fp32 [B, s_q, width]");
  const int64_t batch = s.size(0), s_q = s.size(1), width = s.size(2);
  if (batch > INT32_MAX || s_q > INT32_MAX || width > INT32_MAX) c.refuse("scores' sizes out of range");
  c.on_device(s);
  const int64_t stride = score_stride(c, s, width), topk = c.integer(a[2], "topk", 1);
  const Paged paged(c, a[3], a[1], batch);
  const int64_t blocks = c.integer(a[4], "num_blocks", 1), block = c.integer(a[6], "block");
  const int causal = PyObject_IsTrue(a[5]);
  if (causal < 0) throw Raised();
  const at::Tensor indices = output(c, a[7], "indices", at::kInt, {batch, s_q, topk}, s);
  const at::Tensor lens = output(c, a[8], "lens", at::kInt, {batch, s_q}, s);
  auto* st = static_cast<uint32_t*>(c.status(a[9]));
  c.run([&](void* stream) {
    return mla_select_topk(static_cast<const float*>(s.data_ptr()), stride, (int)width, paged.seqlens, (int)batch,
                           (int)s_q, causal, (int)block, (int)topk, paged.table, paged.max_blocks, blocks, 64,
                           static_cast<int32_t*>(indices.data_ptr()), static_cast<int32_t*>(lens.data_ptr()), st, stream);
  });
  return pair(indices, lens);
}

// a number that fits fp32
float real(const Call& c, PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  const float f = static_cast<float>(v);
  if (!std::isfinite(f)) c.refuse("%s: a finite number", name);
  return f;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
// the weights of a norm: [dim] like x, or None
const void* gain(Call& c, PyObject* o, int64_t dim, const at::Tensor& x) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = c.tensor(o, "weight");
  if (t.scalar_type() != x.scalar_type() || !is_shape(t, {dim}) || !t.is_contiguous())
    c.refuse("weight: contiguous [%lld] of the rows' type", (long long)dim);
  c.on_device(t);
  return t.data_ptr();
}
// rows of heads that the caller gives for an output
void check_rows(Call& c, const at::Tensor& t, const char* name, int64_t tokens, int64_t heads, int64_t dim, const at::Tensor& like) {
  if (!is_shape(t, {tokens, heads, dim}) || t.scalar_type() != like.scalar_type() || (dim > 1 && t.stride(2) != 1))
    c.refuse("%s: [tokens, heads, %lld] of the input's type, dense rows", name, (long long)dim);
  c.on_device(t);
}

// (x, positions, rope_table, weight, eps, rope_at, out, rope_out, rope_style, status)
PyObject* norm_rotate(Call& c, PyObject* const* a) {
  const at::Tensor& x = c.tensor(a[0], "x");
  const int code = dtype_code(x);
  if (code < 0 || x.dim() != 3 || x.size(2) < 64 || x.stride(2) != 1) c.refuse("x [tokens, heads, dim], bf16 or fp16, dim of at least 64");
  const int64_t tokens = x.size(0), heads = x.size(1), dim = x.size(2);
  if (heads > INT32_MAX || dim > INT32_MAX) c.refuse("x's sizes out of range");
  c.on_device(x);
  const void* weight = gain(c, a[3], dim, x);
  const float eps = real(c, a[4], "eps");
  const int64_t at = a[5] == Py_None ? dim - 64 : c.integer(a[5], "rope_at");
  const bool split = a[7] != Py_None;
  const int64_t width = split ? dim - 64 : dim;
  const at::Tensor out = a[6] == Py_None ? fresh({tokens, heads, width}, x.scalar_type(), x) : c.tensor(a[6], "out");
  check_rows(c, out, "out", tokens, heads, width, x);
  const at::Tensor rope = split ? c.tensor(a[7], "rope_out") : at::Tensor();
  if (split) check_rows(c, rope, "rope_out", tokens, heads, 64, x);
  const Rope r(c, a[1], a[2], a[8], tokens);
  auto* st = static_cast<uint32_t*>(c.status(a[9]));
  c.run([&](void* stream) {
    return mla_norm_rotate(x.data_ptr(), stride_of(x, 0, dim * heads), stride_of(x, 1, dim), weight, eps, (int)dim, (int)at,
                           width ? out.data_ptr() : nullptr, stride_of(out, 0, width * heads), stride_of(out, 1, width),
                           split ? rope.data_ptr() : nullptr, split ? stride_of(rope, 0, 64 * heads) : 0,
                           split ? stride_of(rope, 1, 64) : 0, code, r.positions, r.table, r.rows, r.style, tokens,
                           (int)heads, st, stream);
  });
  if (split) return pair(out, rope);
  return THPVariable_Wrap(out);
}

// (c_kv, k_rope, weight, kvcache, slots, positions, rope_table, eps, kv_format, rope_style, rows, status)
PyObject* norm_append_kv(Call& c, PyObject* const* a) {
  const int64_t format = c.integer(a[8], "kv_format");
  static constexpr int64_t widths[4] = {MLA_HEAD_DIM_K, MLA_FP8_ROW_BYTES, MLA_FP8_528_ROW_BYTES, MLA_FP4_288_ROW_BYTES};
  if (format < 0 || format > 3) c.refuse("unknown kv_format %lld", (long long)format);
  const at::Tensor &kv = c.tensor(a[0], "c_kv"), &kr = c.tensor(a[1], "k_rope");
  const int64_t latent = format >= MLA_KV_FP8_528 ? 448 : 512, n = kv.dim() ? kv.size(0) : 0;
  const int code = dtype_code(kv);
  if (code < 0 || !is_shape(kv, {n, latent}) || !is_shape(kr, {n, 64}) || kr.scalar_type() != kv.scalar_type() ||
      kv.stride(1) != 1 || kr.stride(1) != 1)
    c.refuse("c_kv [n, %lld] and k_rope [n, 64], bf16 or fp16", (long long)latent);
  c.on_device(kv);
  c.on_device(kr);
  const void* weight = gain(c, a[2], latent, kv);
  const float eps = real(c, a[7], "eps");
  const Cache cache(c, a[3], "kvcache", widths[format], format ? at::kByte : kv.scalar_type());
  const int32_t* slots = int32_vector(c, a[4], "slots", n);
  const Rope r(c, a[5], a[6], a[9], n);
  void* rows = nullptr;
  int64_t rows_stride = latent + 64;
  if (a[10] != Py_None) {
    const at::Tensor& t = c.tensor(a[10], "rows");
    if (t.scalar_type() != kv.scalar_type() || !is_shape(t, {n, latent + 64}) || t.stride(1) != 1)
      c.refuse("rows [n, %lld] of c_kv's type", (long long)latent + 64);
    c.on_device(t);
    rows = t.data_ptr();
    rows_stride = stride_of(t, 0, latent + 64);
  }
  auto* st = static_cast<uint32_t*>(c.status(a[11]));
  c.run([&](void* stream) {
    return mla_norm_append_kv(kv.data_ptr(), stride_of(kv, 0, latent), kr.data_ptr(), stride_of(kr, 0, 64), weight, eps,
                              code, slots, r.positions, r.table, r.rows, r.style, n, cache.data, cache.blocks, cache.page,
                              (int)format, rows, rows_stride, st, stream);
  });
  Py_INCREF(a[3]);
  return a[3];
}

// (kvcache, block_table, offsets, total, starts, kv_format, dtype code, out, status); the code -1: the cache's own type,
// of quantised rows that of `out`, or bf16
PyObject* read_kv(Call& c, PyObject* const* a) {
  const int64_t format = c.integer(a[5], "kv_format");
  static constexpr int64_t widths[4] = {MLA_HEAD_DIM_K, MLA_FP8_ROW_BYTES, MLA_FP8_528_ROW_BYTES, MLA_FP4_288_ROW_BYTES};
  if (format < 0 || format > 3) c.refuse("unknown kv_format %lld", (long long)format);
  const at::Tensor& kv = c.tensor(a[0], "kvcache");
  int64_t code = c.integer(a[6], "dtype");
  if (format == 0) {
    if (dtype_code(kv) < 0 || (code >= 0 && code != dtype_code(kv))) c.refuse("a 16-bit cache is read in its own type");
    code = dtype_code(kv);
  } else if (code < 0) {
    code = a[7] != Py_None && dtype_code(c.tensor(a[7], "out")) == MLA_DTYPE_FP16 ? MLA_DTYPE_FP16 : MLA_DTYPE_BF16;
  }
  const Cache cache(c, a[0], "kvcache", widths[format], format ? at::kByte : kv.scalar_type());
  const at::Tensor& table = c.tensor(a[1], "block_table");
  const int64_t batch = table.dim() == 2 ? table.size(0) : -1;
  if (table.scalar_type() != at::kInt || batch < 0 || batch > INT32_MAX || table.size(1) > INT32_MAX || !table.is_contiguous())
    c.refuse("block_table: int32 [batch, max_blocks]");
  c.on_device(table);
  const int32_t* offsets = int32_vector(c, a[2], "offsets", batch + 1);
  const int32_t* starts = a[4] == Py_None ? nullptr : int32_vector(c, a[4], "starts", batch);
  const int64_t width = format >= MLA_KV_FP8_528 ? 512 : 576;
  const at::ScalarType type = code == MLA_DTYPE_FP16 ? at::kHalf : at::kBFloat16;
  const bool given = a[7] != Py_None;
  int64_t total;
  if (given) {
    const at::Tensor& t = c.tensor(a[7], "out");
    if (t.dim() != 2 || t.size(1) != width || t.scalar_type() != type || t.stride(1) != 1)
      c.refuse("out [total, %lld] of the type read", (long long)width);
    c.on_device(t);
    total = t.size(0);
    if (a[3] != Py_None && c.integer(a[3], "total") != total) c.refuse("out has another number of rows than total");
  } else {
    if (a[3] == Py_None) c.refuse("total (the rows that offsets name), or out");
    total = c.integer(a[3], "total", 0);
  }
  const at::Tensor out = given ? c.tensor(a[7], "out") : fresh({total, width}, type, kv);
  auto* st = static_cast<uint32_t*>(c.status(a[8]));
  c.run([&](void* stream) {
    return mla_read_kv(cache.data, cache.blocks, cache.page, (int)format, static_cast<const int32_t*>(table.data_ptr()),
                       (int)table.size(1), offsets, starts, (int)batch, total, out.data_ptr(), stride_of(out, 0, width),
                       (int)code, st, stream);
  });
  return THPVariable_Wrap(out);
}

// (q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, softmax_scale, causal, prefix_lens, out, lse, status)
PyObject* prefill(Call& c, PyObject* const* a) {
  const at::Tensor &q = c.tensor(a[0], "q"), &k = c.tensor(a[1], "k_nope"), &kr = c.tensor(a[2], "k_rope"), &v = c.tensor(a[3], "v");
  const int code = dtype_code(q);
  if (code < 0 || q.dim() != 3 || q.size(2) != 192 || q.stride(2) != 1) c.refuse("q [tokens, heads, 192], bf16 or fp16");
  const int64_t tq = q.size(0), heads = q.size(1), tk = k.dim() ? k.size(0) : 0;
  if (heads > INT32_MAX) c.refuse("heads out of range");
  for (const at::Tensor* t : {&k, &kr, &v})
    if (t->scalar_type() != q.scalar_type()) c.refuse("k_nope, k_rope and v of q's type");
  if (!is_shape(k, {tk, heads, 128}) || !is_shape(v, {tk, heads, 128}) || !is_shape(kr, {tk, 64}) || k.stride(2) != 1 ||
      v.stride(2) != 1 || kr.stride(1) != 1)
    c.refuse("k_nope and v [tokens, heads, 128], k_rope [tokens, 64], dense rows");
  for (const at::Tensor* t : {&q, &k, &kr, &v}) c.on_device(*t);
  const at::Tensor& cu = c.tensor(a[4], "cu_seqlens_q");
  const int64_t batch = cu.dim() == 1 ? cu.size(0) - 1 : -1;
  if (batch < 0 || batch >= INT32_MAX) c.refuse("cu_seqlens_q: int32 [batch + 1]");
  const int32_t* cu_q = int32_vector(c, a[4], "cu_seqlens_q", batch + 1);
  const int32_t* cu_k = int32_vector(c, a[5], "cu_seqlens_k", batch + 1);
  const float scale = real(c, a[6], "softmax_scale");
  const bool causal = truth(a[7]);
  const int32_t* prefix = a[8] == Py_None ? nullptr : int32_vector(c, a[8], "prefix_lens", batch);
  const at::Tensor out = a[9] == Py_None ? fresh({tq, heads, 128}, q.scalar_type(), q) : c.tensor(a[9], "out");
  check_rows(c, out, "out", tq, heads, 128, q);
  const at::Tensor lse = output(c, a[10], "lse", at::kFloat, {tq, heads}, q);
  auto* st = static_cast<uint32_t*>(c.status(a[11]));
  // partial results of cut units, from the stream's own memory
  const size_t bytes = mla_prefill_workspace_size(tq, tk, (int)batch, (int)heads);
  at::Tensor space;
  if (bytes) space = fresh({(int64_t)bytes}, at::kByte, q);
  c.run([&](void* stream) {
    return mla_prefill(q.data_ptr(), stride_of(q, 0, 192 * heads), stride_of(q, 1, 192), k.data_ptr(),
                       stride_of(k, 0, 128 * heads), stride_of(k, 1, 128), kr.data_ptr(), stride_of(kr, 0, 64), v.data_ptr(),
                       stride_of(v, 0, 128 * heads), stride_of(v, 1, 128), code, cu_q, cu_k, prefix, (int)batch, tq, tk,
                       (int)heads, scale, causal, out.data_ptr(), stride_of(out, 0, 128 * heads), stride_of(out, 1, 128),
                       static_cast<float*>(lse.data_ptr()), bytes ? space.data_ptr() : nullptr, bytes, st, stream);
  });
  return pair(out, lse);
}

template <PyObject* (*kBody)(Call&, PyObject* const*), int kArgs, const char* const& kName>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%s: %d arguments", kName, kArgs);
    return nullptr;
  }
  try {
    Call c{kName};
    return kBody(c, args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

constexpr const char* kAppendKv = "mla_append_kv";
constexpr const char* kRotateQ = "mla_rotate_q";
constexpr const char* kAppendIndexK = "mla_append_index_k";
constexpr const char* kQuantizeIndexQ = "mla_quantize_index_q";
constexpr const char* kIndexScore = "mla_index_score";
constexpr const char* kSelectTopk = "mla_select_topk";
constexpr const char* kNormRotate = "mla_norm_rotate";
constexpr const char* kNormAppendKv = "mla_norm_append_kv";
constexpr const char* kReadKv = "mla_read_kv";
constexpr const char* kPrefill = "mla_prefill";

#define MLA_METHOD(name, body, args) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<body, args, name>)), METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {
    MLA_METHOD(kAppendKv, append_kv, 9),
    MLA_METHOD(kRotateQ, rotate_q, 6),
    MLA_METHOD(kAppendIndexK, append_index_k, 8),
    MLA_METHOD(kQuantizeIndexQ, quantize_index_q, 8),
    MLA_METHOD(kIndexScore, index_score, 11),
    MLA_METHOD(kSelectTopk, select_topk, 10),
    MLA_METHOD(kNormRotate, norm_rotate, 10),
    MLA_METHOD(kNormAppendKv, norm_append_kv, 12),
    MLA_METHOD(kReadKv, read_kv, 9),
    MLA_METHOD(kPrefill, prefill, 12),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&g_module); }
