// calls.cpp -- the Python side of the 4-bit cache, gather, score and eviction
// calls, of the calls on selected pages, page assignment and log probabilities
// (binding.py wraps these functions).  Argument marshalling only: type,
// shape and device checks, output allocation, raw pointers for libsvp.so.
//
// A decode step makes these calls once per layer, and the smallest of them
// run 4 us on the GPU: marshalled in Python a call takes 10-17 us of host
// time, here 4-6, launch included.  Nothing is kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include "svp.h"

namespace {

using at::Tensor;

[[noreturn]] void fail(PyObject *type, const std::string &what) {
  PyErr_SetString(type, what.c_str());
  throw python_error();
}

// ---- arguments ----

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o))
    fail(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

bool given(PyObject *o) { return o != Py_None; }

int integer(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT_MIN || v > INT_MAX)
    fail(PyExc_ValueError, std::string(name) + " is out of range");
  return (int)v;
}

double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "wrong number of arguments");
}

// `t`: a contiguous tensor of that type and shape on CUDA device `dev`.
void want(const Tensor &t, const char *name, at::Device dev, at::ScalarType type,
          at::IntArrayRef shape) {
  if (t.scalar_type() == type && t.sizes() == shape && t.device() == dev &&
      t.is_contiguous() && dev.is_cuda())
    return;
  std::ostringstream s;
  s << name << " must be a contiguous " << type << " CUDA tensor " << shape
    << " on " << dev << ", got " << t.scalar_type() << " " << t.sizes() << " on "
    << t.device() << (t.is_contiguous() ? "" : " (not contiguous)");
  fail(PyExc_ValueError, s.str());
}

void need(bool cond, const char *what) {
  if (!cond) fail(PyExc_ValueError, what);
}

int small(int64_t v, const char *name) {
  if (v > INT_MAX) fail(PyExc_ValueError, std::string(name) + " is out of range");
  return (int)v;
}

struct Cache {
  int code = 0;          // svp_dtype
  int64_t head_dim = 0;  // what a row holds
  at::ScalarType io = at::kBFloat16;  // of q, outputs and new rows
};

Cache cache_kind(const Tensor &k) {
  need(k.dim() == 4, "caches must be [num_blocks, Hkv, block_size, row]");
  Cache c;
  c.head_dim = k.size(3);
  switch (k.scalar_type()) {
    case at::kFloat:
      c.code = SVP_F32;
      c.io = at::kFloat;
      break;
    case at::kBFloat16:
      c.code = SVP_BF16;
      break;
    case at::kByte:
      // a 4-bit row of 36 or 72 bytes is no FP8 head_dim
      if (c.head_dim == 36 || c.head_dim == 72) {
        c.code = SVP_FP4_E2M1;
        c.head_dim = c.head_dim / 9 * 16;
        break;
      }
      [[fallthrough]];
    case at::kFloat8_e4m3fn:
      c.code = SVP_FP8_E4M3;
      break;
    default:
      fail(PyExc_TypeError,
           "caches must be float32, bfloat16, float8_e4m3fn or uint8");
  }
  return c;
}

// The paged arguments of a call for `batch` sequences; the caches' device.
at::Device pages(const Tensor &k, const Tensor *v, const Tensor &table,
                 const Tensor &lens, int64_t batch) {
  const at::Device dev = k.device();
  want(k, "k_cache", dev, k.scalar_type(), k.sizes());
  if (v) want(*v, "v_cache", dev, k.scalar_type(), k.sizes());
  need(table.dim() == 2, "block_table must be int32 [B, max_blocks]");
  want(table, "block_table", dev, at::kInt, {batch, table.size(1)});
  want(lens, "seq_lens", dev, at::kInt, {batch});
  return dev;
}

svp_dims dims_of(const Cache &c, const Tensor &k, const Tensor &table,
                 int64_t batch, int64_t q_heads, double k_scale,
                 double v_scale) {
  svp_dims d = {};
  d.batch = small(batch, "the batch");
  d.num_q_heads = small(q_heads, "the number of heads");
  d.num_kv_heads = small(k.size(1), "the number of kv heads");
  d.head_dim = small(c.head_dim, "head_dim");
  d.block_size = small(k.size(2), "block_size");
  d.max_blocks_per_seq = small(table.size(1), "block_table");
  d.num_blocks = small(k.size(0), "num_blocks");
  d.dtype = c.code;
  d.k_scale = (float)k_scale;
  d.v_scale = (float)v_scale;
  return d;
}

// The call's device made current, and its stream (an integer handle, or
// None: torch's current one), so that what is allocated on the way belongs
// to the stream that uses it.
class Where {
 public:
  Where(at::Device dev, PyObject *stream) : device_(dev) {
    if (given(stream)) {
      const auto h = PyLong_AsUnsignedLongLong(stream);
      if (PyErr_Occurred()) throw python_error();
      handle_ = reinterpret_cast<cudaStream_t>(h);
      guard_.emplace(c10::cuda::getStreamFromExternal(handle_, dev.index()));
    } else {
      handle_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
  }
  cudaStream_t stream() const { return handle_; }

 private:
  c10::cuda::CUDAGuard device_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
  cudaStream_t handle_ = nullptr;
};

Tensor output(PyObject *o, const char *name, at::Device dev, at::ScalarType type,
              at::IntArrayRef shape) {
  if (!given(o)) return Tensor();  // made once the device is current
  const Tensor &t = tensor(o, name);
  want(t, name, dev, type, shape);
  return t;
}

void make(Tensor &t, at::Device dev, at::ScalarType type, at::IntArrayRef shape) {
  if (!t.defined()) t = at::empty(shape, at::TensorOptions(dev).dtype(type));
}

const uint32_t *tree_bits(PyObject *o, at::Device dev, at::IntArrayRef shape) {
  if (!given(o)) return nullptr;
  const Tensor &t = tensor(o, "tree_mask");
  need(t.element_size() == 4 && !t.is_floating_point(),
       "tree_mask must be int32/uint32 [B, q_len]");
  want(t, "tree_mask", dev, t.scalar_type(), shape);
  return static_cast<const uint32_t *>(t.data_ptr());
}

double scale_or(PyObject *o, int64_t d) {
  return given(o) ? real(o) : 1.0 / std::sqrt((double)d);
}

template <typename T>
T *ptr(const Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

template <typename F>
int without_gil(F f) {
  PyThreadState *s = PyEval_SaveThread();
  const int st = f();
  PyEval_RestoreThread(s);
  return st;
}

// a status other than SVP_OK goes back as an integer: binding.py raises it
PyObject *status(int st) {
  if (st != SVP_OK) return PyLong_FromLong(st);
  Py_RETURN_NONE;
}

PyObject *two(int st, const Tensor &a, const Tensor &b) {
  if (st != SVP_OK) return PyLong_FromLong(st);
  PyObject *x = THPVariable_Wrap(a);
  if (!x) return nullptr;
  PyObject *y = THPVariable_Wrap(b);
  if (!y) {
    Py_DECREF(x);
    return nullptr;
  }
  PyObject *t = PyTuple_New(2);
  if (!t) {
    Py_DECREF(x);
    Py_DECREF(y);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, x);
  PyTuple_SET_ITEM(t, 1, y);
  return t;
}

// ---- the calls ----

// k_new, v_new, k_cache, v_cache, block_table, seq_lens, stream, k_scale,
// v_scale
PyObject *append_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor &kn = tensor(a[0], "k_new"), &vn = tensor(a[1], "v_new");
  const Tensor &k = tensor(a[2], "k_cache"), &v = tensor(a[3], "v_cache");
  const Tensor &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "seq_lens");
  need(kn.dim() == 4, "k_new/v_new must be [B, n_new, Hkv, D]");
  const Cache c = cache_kind(k);
  const int64_t batch = kn.size(0);
  const at::Device dev = pages(k, &v, table, lens, batch);
  const int64_t shape[4] = {batch, kn.size(1), k.size(1), c.head_dim};
  want(kn, "k_new", dev, c.io, shape);
  want(vn, "v_new", dev, c.io, shape);
  const svp_dims d =
      dims_of(c, k, table, batch, k.size(1), real(a[7]), real(a[8]));
  const int n_new = small(kn.size(1), "n_new");
  const Where where(dev, a[6]);
  return status(without_gil([&] {
    return kv_append(&d, kn.data_ptr(), vn.data_ptr(), k.data_ptr(), v.data_ptr(),
                     ptr<int32_t>(table), ptr<int32_t>(lens), n_new,
                     where.stream());
  }));
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, seq_lens, n_sink, window, tree_mask, scale,
// out, lse, workspace, split_pages, kernel_path, stream, k_scale, v_scale
PyObject *attention_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 17);
  const Tensor &q = tensor(a[0], "q");
  const Tensor &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
  const Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
  need(q.dim() == 4, "q must be [B, q_len, Hq, D]");
  const Cache c = cache_kind(k);
  const int64_t batch = q.size(0);
  const at::Device dev = pages(k, &v, table, lens, batch);
  want(q, "q", dev, c.io, q.sizes());
  need(q.size(3) == c.head_dim,
       "a 4-bit cache row has 9/16 byte per element of q's head_dim");
  const int64_t rows[3] = {batch, q.size(1), q.size(2)};
  const uint32_t *tree = tree_bits(a[7], dev, {batch, q.size(1)});
  Tensor out = output(a[9], "out", dev, c.io, q.sizes());
  Tensor lse = output(a[10], "lse", dev, at::kFloat, rows);
  Tensor ws;
  if (given(a[11])) {
    ws = tensor(a[11], "workspace");
    want(ws, "workspace", dev, ws.scalar_type(), ws.sizes());
  }
  svp_dims d =
      dims_of(c, k, table, batch, q.size(2), real(a[15]), real(a[16]));
  d.split_pages = integer(a[12], "split_pages");
  d.kernel_path = integer(a[13], "kernel_path");
  const int n_sink = integer(a[5], "n_sink"), window = integer(a[6], "window");
  const int q_len = small(q.size(1), "q_len");
  const float scale = (float)scale_or(a[8], c.head_dim);
  const Where where(dev, a[14]);
  if (!ws.defined()) {
    // a workspace of the call's own: calls on other streams and captured
    // graphs share nothing.  0: an invalid request, which the call reports;
    // a header's size: it uses none
    const size_t bytes = paged_decode_workspace_size(&d, q_len, n_sink, window);
    if (bytes > 256)
      ws = at::empty({(int64_t)bytes}, at::TensorOptions(dev).dtype(at::kByte));
  }
  if (ws.defined()) {
    d.workspace = ws.data_ptr();
    d.workspace_bytes = (size_t)ws.nbytes();
  }
  make(out, dev, c.io, q.sizes());
  make(lse, dev, at::kFloat, rows);
  const int st = without_gil([&] {
    return tree ? paged_tree_attention(&d, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       ptr<int32_t>(table), ptr<int32_t>(lens),
                                       q_len, tree, scale, out.data_ptr(),
                                       ptr<float>(lse), where.stream())
                : paged_decode_attention(&d, q.data_ptr(), k.data_ptr(),
                                         v.data_ptr(), ptr<int32_t>(table),
                                         ptr<int32_t>(lens), q_len, n_sink, window,
                                         scale, out.data_ptr(), ptr<float>(lse),
                                         where.stream());
  });
  return two(st, out, lse);
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, block_table, seq_lens, n_rows, starts, k_out, v_out,
// stream, k_scale, v_scale
PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11);
  const Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache");
  const Tensor &table = tensor(a[2], "block_table"), &lens = tensor(a[3], "seq_lens");
  need(lens.dim() == 1, "seq_lens must be int32 [B]");
  const Cache c = cache_kind(k);
  const int64_t batch = lens.size(0);
  const at::Device dev = pages(k, &v, table, lens, batch);
  const int n_rows = integer(a[4], "n_rows");
  need(n_rows >= 0, "n_rows must not be negative");
  const int64_t shape[4] = {batch, n_rows, k.size(1), c.head_dim};
  const int32_t *starts = nullptr;
  if (given(a[5])) {
    const Tensor &t = tensor(a[5], "starts");
    want(t, "starts", dev, at::kInt, {batch});
    starts = ptr<int32_t>(t);
  }
  Tensor ko = output(a[6], "k_out", dev, c.io, shape);
  Tensor vo = output(a[7], "v_out", dev, c.io, shape);
  const svp_dims d =
      dims_of(c, k, table, batch, k.size(1), real(a[9]), real(a[10]));
  const Where where(dev, a[8]);
  make(ko, dev, c.io, shape);
  make(vo, dev, c.io, shape);
  const int st = without_gil([&] {
    return kv_gather(&d, k.data_ptr(), v.data_ptr(), ptr<int32_t>(table),
                     ptr<int32_t>(lens), starts, n_rows, ko.data_ptr(),
                     vo.data_ptr(), where.stream());
  });
  return two(st, ko, vo);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, lse, block_table, seq_lens, scores, n_fresh, n_sink, window,
// tree_mask, scale, k_scale, stream
PyObject *score_update(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache");
  const Tensor &lse = tensor(a[2], "lse"), &table = tensor(a[3], "block_table");
  const Tensor &lens = tensor(a[4], "seq_lens"), &scores = tensor(a[5], "scores");
  need(q.dim() == 4, "q must be [B, q_len, Hq, D]");
  const Cache c = cache_kind(k);
  const int64_t batch = q.size(0);
  const at::Device dev = pages(k, nullptr, table, lens, batch);
  want(q, "q", dev, c.io, q.sizes());
  need(q.size(3) == c.head_dim, "q and k_cache must share head_dim");
  want(lse, "lse", dev, at::kFloat, {batch, q.size(1), q.size(2)});
  want(scores, "scores", dev, at::kFloat, k.sizes().slice(0, 3));
  const uint32_t *tree = tree_bits(a[9], dev, {batch, q.size(1)});
  const svp_dims d = dims_of(c, k, table, batch, q.size(2), real(a[11]), 1.0);
  const int q_len = small(q.size(1), "q_len");
  const int n_fresh = given(a[6]) ? integer(a[6], "n_fresh") : q_len;
  const int n_sink = integer(a[7], "n_sink"), window = integer(a[8], "window");
  const float scale = (float)scale_or(a[10], c.head_dim);
  const Where where(dev, a[12]);
  return status(without_gil([&] {
    return paged_score_update(&d, q.data_ptr(), k.data_ptr(), ptr<float>(lse),
                              ptr<int32_t>(table), ptr<int32_t>(lens), q_len,
                              n_sink, window, tree, scale, n_fresh,
                              ptr<float>(scores), where.stream());
  }));
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, scores, block_table, seq_lens, budget, n_sink, n_recent,
// dst_block_table, kept, new_lens, stream
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache");
  const Tensor &scores = tensor(a[2], "scores"), &table = tensor(a[3], "block_table");
  const Tensor &lens = tensor(a[4], "seq_lens");
  need(lens.dim() == 1, "seq_lens must be int32 [B]");
  const Cache c = cache_kind(k);
  const int64_t batch = lens.size(0);
  const at::Device dev = pages(k, &v, table, lens, batch);
  want(scores, "scores", dev, at::kFloat, k.sizes().slice(0, 3));
  const int budget = integer(a[5], "budget");
  need(budget >= 1, "budget must be at least 1");
  const int n_sink = integer(a[6], "n_sink"), n_recent = integer(a[7], "n_recent");
  const int32_t *dst = nullptr;
  int dst_blocks = 0;
  if (given(a[8])) {
    const Tensor &t = tensor(a[8], "dst_block_table");
    need(t.dim() == 2, "dst_block_table must be int32 [B, n]");
    want(t, "dst_block_table", dev, at::kInt, {batch, t.size(1)});
    dst = ptr<int32_t>(t);
    dst_blocks = small(t.size(1), "dst_block_table");
  }
  const int64_t shape[3] = {batch, k.size(1), budget};
  Tensor kept = output(a[9], "kept", dev, at::kInt, shape);
  Tensor new_lens = output(a[10], "new_lens", dev, at::kInt, {batch});
  const svp_dims d = dims_of(c, k, table, batch, k.size(1), 1.0, 1.0);
  const Where where(dev, a[11]);
  make(kept, dev, at::kInt, shape);
  make(new_lens, dev, at::kInt, {batch});
  const int st = without_gil([&] {
    return kv_evict(&d, k.data_ptr(), v.data_ptr(), ptr<float>(scores),
                    ptr<int32_t>(table), ptr<int32_t>(lens), budget, n_sink,
                    n_recent, dst, dst_blocks, ptr<int32_t>(kept),
                    ptr<int32_t>(new_lens), where.stream());
  });
  return two(st, kept, new_lens);
  END_HANDLE_TH_ERRORS
}

// k_cache, block_table, seq_lens, bounds, n_new, stream
PyObject *page_bounds(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  const Tensor &k = tensor(a[0], "k_cache"), &table = tensor(a[1], "block_table");
  const Tensor &lens = tensor(a[2], "seq_lens"), &bounds = tensor(a[3], "bounds");
  need(lens.dim() == 1, "seq_lens must be int32 [B]");
  const Cache c = cache_kind(k);
  const int64_t batch = lens.size(0);
  const at::Device dev = pages(k, nullptr, table, lens, batch);
  want(bounds, "bounds", dev, at::kBFloat16, {k.size(0), k.size(1), 2, c.head_dim});
  const int n_new = given(a[4]) ? integer(a[4], "n_new") : INT_MAX;
  const svp_dims d = dims_of(c, k, table, batch, k.size(1), 1.0, 1.0);
  const Where where(dev, a[5]);
  return status(without_gil([&] {
    return kv_page_bounds(&d, k.data_ptr(), ptr<int32_t>(table), ptr<int32_t>(lens),
                          n_new, bounds.data_ptr(), where.stream());
  }));
  END_HANDLE_TH_ERRORS
}

// q, bounds, block_table, seq_lens, scale, k_scale, scores, stream
PyObject *page_scores(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Tensor &q = tensor(a[0], "q"), &bounds = tensor(a[1], "bounds");
  const Tensor &table = tensor(a[2], "block_table"), &lens = tensor(a[3], "seq_lens");
  need(q.dim() == 4, "q must be [B, q_len, Hq, D]");
  need(q.scalar_type() == at::kFloat || q.scalar_type() == at::kBFloat16,
       "q must be float32 or bfloat16");
  need(bounds.dim() == 4, "bounds must be [num_blocks, Hkv, 2, D]");
  need(table.dim() == 2, "block_table must be int32 [B, max_blocks]");
  const at::Device dev = q.device();
  const int64_t batch = q.size(0);
  want(q, "q", dev, q.scalar_type(), q.sizes());
  want(bounds, "bounds", dev, at::kBFloat16,
       {bounds.size(0), bounds.size(1), 2, q.size(3)});
  want(table, "block_table", dev, at::kInt, {batch, table.size(1)});
  want(lens, "seq_lens", dev, at::kInt, {batch});
  const int64_t shape[3] = {batch, bounds.size(1), table.size(1)};
  Tensor scores = output(a[6], "scores", dev, at::kFloat, shape);
  svp_dims d = {};
  d.batch = small(batch, "the batch");
  d.num_q_heads = small(q.size(2), "the number of heads");
  d.num_kv_heads = small(bounds.size(1), "the number of kv heads");
  d.head_dim = small(q.size(3), "head_dim");
  d.block_size = 16;
  d.max_blocks_per_seq = small(table.size(1), "block_table");
  d.num_blocks = small(bounds.size(0), "num_blocks");
  d.dtype = q.scalar_type() == at::kFloat ? SVP_F32 : SVP_BF16;
  const int q_len = small(q.size(1), "q_len");
  const float scale = (float)(scale_or(a[4], q.size(3)) * real(a[5]));
  const Where where(dev, a[7]);
  make(scores, dev, at::kFloat, shape);
  const int st = without_gil([&] {
    return paged_page_scores(&d, q.data_ptr(), bounds.data_ptr(), ptr<int32_t>(table),
                             ptr<int32_t>(lens), q_len, scale, ptr<float>(scores),
                             where.stream());
  });
  return st != SVP_OK ? PyLong_FromLong(st) : THPVariable_Wrap(scores);
  END_HANDLE_TH_ERRORS
}

// scores, seq_lens, n_select, n_sink, n_recent, pages, stream
PyObject *select_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const Tensor &scores = tensor(a[0], "scores"), &lens = tensor(a[1], "seq_lens");
  need(scores.dim() == 3, "scores must be float32 [B, Hkv, max_blocks]");
  const at::Device dev = scores.device();
  want(scores, "scores", dev, at::kFloat, scores.sizes());
  want(lens, "seq_lens", dev, at::kInt, {scores.size(0)});
  const int n_select = integer(a[2], "n_select");
  need(n_select >= 1, "n_select must be at least 1");
  const int n_sink = integer(a[3], "n_sink"), n_recent = integer(a[4], "n_recent");
  const int64_t shape[3] = {scores.size(0), scores.size(1), n_select};
  Tensor pages = output(a[5], "pages", dev, at::kInt, shape);
  const int batch = small(scores.size(0), "the batch");
  const int heads = small(scores.size(1), "the number of kv heads");
  const int blocks = small(scores.size(2), "max_blocks");
  const Where where(dev, a[6]);
  make(pages, dev, at::kInt, shape);
  const int st = without_gil([&] {
    return paged_select_pages(batch, heads, blocks, ptr<float>(scores),
                              ptr<int32_t>(lens), n_select, n_sink, n_recent,
                              ptr<int32_t>(pages), where.stream());
  });
  return st != SVP_OK ? PyLong_FromLong(st) : THPVariable_Wrap(pages);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, seq_lens, pages, tree_mask, scale, out, lse,
// split_pages, stream, k_scale, v_scale
PyObject *sparse_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 14);
  const Tensor &q = tensor(a[0], "q");
  const Tensor &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
  const Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
  const Tensor &list = tensor(a[5], "pages");
  need(q.dim() == 4, "q must be [B, q_len, Hq, D]");
  const Cache c = cache_kind(k);
  const int64_t batch = q.size(0);
  const at::Device dev = pages(k, &v, table, lens, batch);
  want(q, "q", dev, c.io, q.sizes());
  need(q.size(3) == c.head_dim, "q and the caches must share head_dim");
  need(list.dim() == 3, "pages must be int32 [B, Hkv, n_select]");
  want(list, "pages", dev, at::kInt, {batch, k.size(1), list.size(2)});
  const int64_t rows[3] = {batch, q.size(1), q.size(2)};
  const uint32_t *tree = tree_bits(a[6], dev, {batch, q.size(1)});
  Tensor out = output(a[8], "out", dev, c.io, q.sizes());
  Tensor lse = output(a[9], "lse", dev, at::kFloat, rows);
  svp_dims d =
      dims_of(c, k, table, batch, q.size(2), real(a[12]), real(a[13]));
  d.split_pages = integer(a[10], "split_pages");
  const int q_len = small(q.size(1), "q_len");
  const int n_select = small(list.size(2), "n_select");
  const float scale = (float)scale_or(a[7], c.head_dim);
  const Where where(dev, a[11]);
  make(out, dev, c.io, q.sizes());
  make(lse, dev, at::kFloat, rows);
  const int st = without_gil([&] {
    return paged_sparse_attention(&d, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                  ptr<int32_t>(table), ptr<int32_t>(lens), q_len,
                                  ptr<int32_t>(list), n_select, tree, scale,
                                  out.data_ptr(), ptr<float>(lse), where.stream());
  });
  return two(st, out, lse);
  END_HANDLE_TH_ERRORS
}

// block_table, seq_lens, new_lens, free_pages, free_count, n_slots, slots,
// offsets, num_blocks, stream
PyObject *assign_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor &table = tensor(a[0], "block_table"), &lens = tensor(a[1], "seq_lens");
  const Tensor &target = tensor(a[2], "new_lens"), &free = tensor(a[3], "free_pages");
  const Tensor &left = tensor(a[4], "free_count");
  need(table.dim() == 2, "block_table must be int32 [B, max_blocks]");
  need(free.dim() == 1, "free_pages must be int32 [capacity]");
  const at::Device dev = table.device();
  const int64_t batch = table.size(0);
  want(table, "block_table", dev, at::kInt, table.sizes());
  want(lens, "seq_lens", dev, at::kInt, {batch});
  want(target, "new_lens", dev, at::kInt, {batch});
  want(free, "free_pages", dev, at::kInt, free.sizes());
  want(left, "free_count", dev, at::kInt, {1});
  int n_slots = given(a[5]) ? integer(a[5], "n_slots") : 0;
  need(n_slots >= 0, "n_slots must not be negative");
  Tensor slots;
  if (given(a[6])) {
    slots = tensor(a[6], "slots");
    need(slots.dim() == 1, "slots must be int64 [n_slots]");
    want(slots, "slots", dev, at::kLong, slots.sizes());
    need(!given(a[5]) || slots.size(0) == n_slots, "slots must have n_slots entries");
    n_slots = small(slots.size(0), "n_slots");
  }
  const bool map = given(a[5]) || given(a[6]);
  Tensor offsets = output(a[7], "offsets", dev, at::kInt, {batch + 1});
  const int num_blocks = given(a[8]) ? integer(a[8], "num_blocks") : INT_MAX;
  const int b = small(batch, "the batch"), blocks = small(table.size(1), "max_blocks");
  const int capacity = small(free.size(0), "free_pages");
  const Where where(dev, a[9]);
  if (map) make(slots, dev, at::kLong, {n_slots});
  make(offsets, dev, at::kInt, {batch + 1});
  // no entries, yet a map: the limit of zero slots holds
  static int64_t none;
  const int st = without_gil([&] {
    return kv_assign_pages(b, blocks, num_blocks, ptr<int32_t>(table),
                           ptr<int32_t>(lens), ptr<int32_t>(target),
                           ptr<int32_t>(free), ptr<int32_t>(left), capacity,
                           !map ? nullptr : n_slots ? ptr<int64_t>(slots) : &none,
                           n_slots, ptr<int32_t>(offsets), where.stream());
  });
  if (map) return two(st, slots, offsets);
  if (st != SVP_OK) return PyLong_FromLong(st);
  PyObject *o = THPVariable_Wrap(offsets);
  if (!o) return nullptr;
  PyObject *t = PyTuple_New(2);
  if (!t) {
    Py_DECREF(o);
    return nullptr;
  }
  Py_INCREF(Py_None);
  PyTuple_SET_ITEM(t, 0, Py_None);
  PyTuple_SET_ITEM(t, 1, o);
  return t;
  END_HANDLE_TH_ERRORS
}

// k_new, v_new, k_cache, v_cache, slots, stream, k_scale, v_scale
PyObject *append_slots(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Tensor &kn = tensor(a[0], "k_new"), &vn = tensor(a[1], "v_new");
  const Tensor &k = tensor(a[2], "k_cache"), &v = tensor(a[3], "v_cache");
  const Tensor &slots = tensor(a[4], "slots");
  need(kn.dim() == 3, "k_new/v_new must be [n_rows, Hkv, D] with slots");
  const Cache c = cache_kind(k);
  const at::Device dev = k.device();
  want(k, "k_cache", dev, k.scalar_type(), k.sizes());
  want(v, "v_cache", dev, k.scalar_type(), k.sizes());
  const int64_t shape[3] = {kn.size(0), k.size(1), c.head_dim};
  want(kn, "k_new", dev, c.io, shape);
  want(vn, "v_new", dev, c.io, shape);
  want(slots, "slots", dev, at::kLong, {kn.size(0)});
  svp_dims d = {};
  d.num_q_heads = d.num_kv_heads = small(k.size(1), "the number of kv heads");
  d.head_dim = small(c.head_dim, "head_dim");
  d.block_size = small(k.size(2), "block_size");
  d.num_blocks = small(k.size(0), "num_blocks");
  d.dtype = c.code;
  d.k_scale = (float)real(a[6]);
  d.v_scale = (float)real(a[7]);
  const int n_rows = small(kn.size(0), "the number of rows");
  const Where where(dev, a[5]);
  return status(without_gil([&] {
    return kv_append_slots(&d, kn.data_ptr(), vn.data_ptr(), k.data_ptr(),
                           v.data_ptr(), ptr<int64_t>(slots), n_rows,
                           where.stream());
  }));
  END_HANDLE_TH_ERRORS
}

// logits, tokens, n_top, temperature, allowed, logprobs, entropy, ranks,
// top_logprobs, top_tokens, stream
PyObject *logprobs(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11);
  const Tensor &logits = tensor(a[0], "logits"), &tokens = tensor(a[1], "tokens");
  need(logits.dim() >= 1, "logits must be [..., vocab]");
  need(logits.scalar_type() == at::kFloat || logits.scalar_type() == at::kBFloat16,
       "logits must be float32 or bfloat16");
  const at::Device dev = logits.device();
  want(logits, "logits", dev, logits.scalar_type(), logits.sizes());
  const auto lead = logits.sizes().slice(0, logits.dim() - 1);
  want(tokens, "tokens", dev, at::kInt, lead);
  const int n_top = integer(a[2], "n_top");
  need(n_top >= 0, "n_top must not be negative");
  const float temperature = (float)real(a[3]);
  const int vocab = small(logits.size(-1), "the vocabulary");
  const uint32_t *allowed = nullptr;
  if (given(a[4])) {
    const Tensor &t = tensor(a[4], "allowed");
    need(t.element_size() == 4 && !t.is_floating_point(),
         "allowed must be int32/uint32 [..., ceil(vocab / 32)]");
    std::vector<int64_t> shape(lead.begin(), lead.end());
    shape.push_back(((int64_t)vocab + 31) / 32);
    want(t, "allowed", dev, t.scalar_type(), shape);
    allowed = static_cast<const uint32_t *>(t.data_ptr());
  }
  std::vector<int64_t> tops(lead.begin(), lead.end());
  tops.push_back(n_top);
  Tensor lp = output(a[5], "logprobs", dev, at::kFloat, lead);
  Tensor en = output(a[6], "entropy", dev, at::kFloat, lead);
  Tensor rk = output(a[7], "ranks", dev, at::kInt, lead);
  Tensor tl = output(a[8], "top_logprobs", dev, at::kFloat, tops);
  Tensor tt = output(a[9], "top_tokens", dev, at::kInt, tops);
  const int rows = small(tokens.numel(), "the number of rows");
  const int code = logits.scalar_type() == at::kFloat ? SVP_F32 : SVP_BF16;
  const Where where(dev, a[10]);
  make(lp, dev, at::kFloat, lead);
  make(en, dev, at::kFloat, lead);
  make(rk, dev, at::kInt, lead);
  make(tl, dev, at::kFloat, tops);
  make(tt, dev, at::kInt, tops);
  const int st = without_gil([&] {
    return token_logprobs(rows, vocab, code, logits.data_ptr(), ptr<int32_t>(tokens),
                          n_top, temperature, allowed, ptr<float>(lp), ptr<float>(en),
                          ptr<int32_t>(rk), ptr<float>(tl), ptr<int32_t>(tt),
                          where.stream());
  });
  if (st != SVP_OK) return PyLong_FromLong(st);
  PyObject *t = PyTuple_New(5);
  if (!t) return nullptr;
  const Tensor *const all[5] = {&lp, &en, &rk, &tl, &tt};
  for (int i = 0; i < 5; ++i) {
    PyObject *x = THPVariable_Wrap(*all[i]);
    if (!x) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i, x);
  }
  return t;
  END_HANDLE_TH_ERRORS
}

#define SVP_FAST(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {SVP_FAST("append_fp4", append_fp4),
                          SVP_FAST("attention_fp4", attention_fp4),
                          SVP_FAST("gather", gather),
                          SVP_FAST("score_update", score_update),
                          SVP_FAST("evict", evict),
                          SVP_FAST("page_bounds", page_bounds),
                          SVP_FAST("page_scores", page_scores),
                          SVP_FAST("select_pages", select_pages),
                          SVP_FAST("sparse_attention", sparse_attention),
                          SVP_FAST("assign_pages", assign_pages),
                          SVP_FAST("append_slots", append_slots),
                          SVP_FAST("logprobs", logprobs),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "svp_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_svp_calls(void) {
  PyObject *m = PyModule_Create(&kModule);
  // the torch whose headers this was compiled against
  if (m && PyModule_AddStringConstant(m, "torch_version", SVP_TORCH) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
