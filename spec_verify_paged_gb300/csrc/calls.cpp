// calls.cpp -- the Python side of the 4-bit cache, gather, score and eviction
// calls (binding.py wraps these functions).  Argument marshalling only: type,
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

#define SVP_FAST(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {SVP_FAST("append_fp4", append_fp4),
                          SVP_FAST("attention_fp4", attention_fp4),
                          SVP_FAST("gather", gather),
                          SVP_FAST("score_update", score_update),
                          SVP_FAST("evict", evict),
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
