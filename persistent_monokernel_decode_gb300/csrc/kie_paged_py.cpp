// Marshalling of the paged-cache operators and the log probabilities from tensors to the C ABI (include/kie.h): types,
// shapes and devices are checked, outputs and the workspace allocated, and the call made on the current stream of the
// tensors' device. A call of
// the attention takes 6.5 us of the host's time, of the append 3.4, of the release 5, of extend 8; marshalled in Python
// they took 22, 12, 24 and 31 us, several times what the kernels of a small step do.
//
// paged.py documents the functions; they take their arguments by position. bind() receives the addresses of the C entry
// points and the exception class of the package.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/DeviceGuard.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>

#include <stdexcept>
#include <string>

#include "kie.h"

namespace {

decltype(&kie_paged_extend) g_extend;
decltype(&kie_paged_release) g_release;
decltype(&kie_paged_append) g_append;
decltype(&kie_paged_attention) g_attention;
decltype(&kie_paged_attention_workspace) g_workspace;
decltype(&kie_paged_prefix_attention) g_prefix_attention;
decltype(&kie_paged_prefix_attention_workspace) g_prefix_workspace;
decltype(&kie_paged_fork) g_fork;
decltype(&kie_paged_copy) g_copy;
decltype(&kie_paged_compact) g_compact;
decltype(&kie_token_logprobs) g_logprobs;
decltype(&kie_paged_last_error) g_last_error;
PyObject *g_error;  // KieError(code, message)

struct Refused : std::runtime_error {  // becomes a ValueError
  using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python exception is set

void need(bool ok, const char *what) {
  if (!ok) throw Refused(what);
}

void check(int rc) {
  if (rc == KIE_OK) return;
  if (PyObject *e = PyObject_CallFunction(g_error, "is", rc, g_last_error())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " is out of range");
  return v;
}

int kind(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kHalf: return KIE_F16;
    case at::kBFloat16: return KIE_BF16;
    case at::kFloat: return KIE_F32;
    case at::kFloat8_e4m3fn: return KIE_E4M3;
    default: return -1;
  }
}

// Address of a contiguous int32 tensor of n values (n < 0: any number) on the device.
int32_t *ints(const at::Tensor &t, const char *name, const at::Device &dev, int64_t n = -1) {
  if (t.scalar_type() != at::kInt || !t.is_contiguous() || t.device() != dev || (n >= 0 && t.numel() != n))
    throw Refused(std::string(name) + " must be a contiguous int32 tensor" +
                  (n >= 0 ? " of " + std::to_string(n) : std::string()) + " on " + dev.str());
  return static_cast<int32_t *>(t.data_ptr());
}

int32_t *table(const at::Tensor &t, const at::Device &dev, int64_t n_seqs) {
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != n_seqs || t.size(1) < 1 || t.stride(1) != 1 ||
      t.device() != dev)
    throw Refused("block_table must be an int32 [" + std::to_string(n_seqs) + ", max_blocks] tensor on " + dev.str() +
                  " with contiguous rows");
  return static_cast<int32_t *>(t.data_ptr());
}

// Address and first two strides of a tensor [n, heads, head_dim] of rows.
void *rows(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType type, const at::Device &dev,
           int64_t (&stride)[2]) {
  if (t.sizes() != shape || t.scalar_type() != type || t.device() != dev || t.stride(2) != 1) {
    std::string s;
    for (int64_t x : shape) s += (s.empty() ? "" : ", ") + std::to_string(x);
    throw Refused(std::string(name) + " must be a [" + s + "] " + c10::toString(type) + " tensor on " + dev.str() +
                  " with contiguous rows");
  }
  stride[0] = t.stride(0);
  stride[1] = t.stride(1);
  return t.data_ptr();
}

int size_of(int64_t v, const char *name) {
  if (v > INT32_MAX) throw Refused(std::string(name) + " is out of range");
  return (int)v;
}

// Page tensors [n_blocks, n_kv_heads, block_size, head_dim] (any outer strides) with their scales.
kie_pages pages(const at::Tensor &k, const at::Tensor &v, PyObject *k_scale, PyObject *v_scale, const at::Device &dev) {
  kie_pages p = {};
  need(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() && k.stride(3) == 1 && v.stride(3) == 1,
       "the pages are two tensors [n_blocks, n_kv_heads, block_size, head_dim] of one type whose last dimension is contiguous");
  p.dtype = kind(k);
  need(p.dtype >= 0 && p.dtype != KIE_F32, "pages are float16, bfloat16 or float8_e4m3fn");
  need(dev.is_cuda() && k.device() == dev && v.device() == dev, "the pages and the rows must be on one CUDA device");
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  for (int i = 0; i < 3; ++i) p.k_stride[i] = k.stride(i), p.v_stride[i] = v.stride(i);
  p.n_blocks = size_of(k.size(0), "n_blocks");
  p.n_kv_heads = size_of(k.size(1), "n_kv_heads");
  p.block_size = size_of(k.size(2), "block_size");
  p.head_dim = size_of(k.size(3), "head_dim");
  if (p.dtype != KIE_E4M3) {
    need(k_scale == Py_None && v_scale == Py_None, "only float8_e4m3fn pages have scales");
    return p;
  }
  need(k_scale != Py_None && v_scale != Py_None, "float8_e4m3fn pages need k_scale and v_scale");
  const at::Tensor &ks = tensor(k_scale, "k_scale"), &vs = tensor(v_scale, "v_scale");
  for (const at::Tensor *s : {&ks, &vs})
    need(s->scalar_type() == at::kFloat && s->dim() == 3 && s->size(0) == k.size(0) && s->size(1) == k.size(1) &&
             s->size(2) == k.size(2) && s->device() == dev,
         "the scales are float32 [n_blocks, n_kv_heads, block_size] tensors on the pages' device");
  p.k_scale = static_cast<float *>(ks.data_ptr());
  p.v_scale = static_cast<float *>(vs.data_ptr());
  for (int i = 0; i < 3; ++i) p.k_scale_stride[i] = ks.stride(i), p.v_scale_stride[i] = vs.stride(i);
  return p;
}

void *stream_of(const at::Device &dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev) {
  return at::Tensor(at::detail::empty_cuda(shape, at::TensorOptions().dtype(type).device(dev)));
}

// Elements [at, at + n) of a new buffer as a tensor of its own on the same storage.
at::Tensor part(const at::Tensor &buffer, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(), buffer.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

PyObject *wrap(at::Tensor t) {
  PyObject *o = THPVariable_Wrap(std::move(t));
  if (!o) throw Raised();
  return o;
}

template <class... T>
PyObject *wrap_all(T... t) {
  PyObject *items[] = {THPVariable_Wrap(std::move(t))...};
  PyObject *out = PyTuple_New(sizeof...(t));
  bool ok = out != nullptr;
  for (size_t i = 0; i < sizeof...(t); ++i) {
    ok = ok && items[i];
    if (out)
      PyTuple_SET_ITEM(out, i, items[i]);  // takes the reference
    else
      Py_XDECREF(items[i]);
  }
  if (!ok) {
    Py_XDECREF(out);
    throw Raised();
  }
  return out;
}

// extend(new_lens, lens, block_table, free_blocks, n_free, block_size, n_rows)
PyObject *extend(PyObject *const *x) {
  const at::Tensor &fresh = tensor(x[0], "new_lens"), &lens = tensor(x[1], "lens"), &tab = tensor(x[2], "block_table"),
                   &free = tensor(x[3], "free_blocks"), &n_free = tensor(x[4], "n_free");
  const at::Device dev = lens.device();
  const int64_t R = lens.numel();
  need(dev.is_cuda(), "lens must be a CUDA tensor");
  kie_paged_extend_args a = {};
  a.n_rows = (int)integer(x[6], "n_rows");
  need(a.n_rows >= 0, "n_rows must be >= 0");
  a.lens = ints(lens, "lens", dev);
  a.new_lens = ints(fresh, "new_lens", dev, R);
  a.free_blocks = ints(free, "free_blocks", dev);
  a.n_free = ints(n_free, "n_free", dev, 1);
  a.block_table = table(tab, dev, R);
  a.table_stride = tab.stride(0);
  a.n_seqs = size_of(R, "the number of requests");
  a.max_blocks = size_of(tab.size(1), "max_blocks");
  a.block_size = (int)integer(x[5], "block_size");
  a.free_capacity = size_of(free.numel(), "the length of free_blocks");
  const c10::DeviceGuard guard(dev);
  const at::Tensor admitted = empty({R}, at::kBool, dev), buffer = empty({2 * R + 2 + 3ll * a.n_rows}, at::kInt, dev);
  const int64_t at[] = {0, R, R + 1, 2 * R + 2, 2 * R + 2 + a.n_rows, 2 * R + 2 + 2ll * a.n_rows};
  int32_t *p = static_cast<int32_t *>(buffer.data_ptr());
  a.admitted = static_cast<uint8_t *>(admitted.data_ptr());
  a.lens_out = p + at[0];
  a.n_free_out = p + at[1];
  a.row_start = p + at[2];
  a.slots = p + at[3];
  a.positions = p + at[4];
  a.seqs = p + at[5];
  check(g_extend(&a, stream_of(dev)));
  return wrap_all(part(buffer, at[0], R), part(buffer, at[1], 1), admitted, part(buffer, at[2], R + 1),
                  part(buffer, at[3], a.n_rows), part(buffer, at[4], a.n_rows), part(buffer, at[5], a.n_rows));
}

// release(done, lens, block_table, free_blocks, n_free, block_size, shares)
PyObject *release(PyObject *const *x) {
  const at::Tensor &done = tensor(x[0], "done"), &lens = tensor(x[1], "lens"), &tab = tensor(x[2], "block_table"),
                   &free = tensor(x[3], "free_blocks"), &n_free = tensor(x[4], "n_free");
  const at::Device dev = lens.device();
  const int64_t R = lens.numel();
  need(dev.is_cuda(), "lens must be a CUDA tensor");
  need(done.scalar_type() == at::kBool && done.numel() == R && done.is_contiguous() && done.device() == dev,
       "done must be a contiguous bool tensor of a value per request on lens' device");
  kie_paged_release_args a = {};
  a.done = static_cast<uint8_t *>(done.data_ptr());
  a.lens = ints(lens, "lens", dev);
  a.n_free = ints(n_free, "n_free", dev, 1);
  a.block_table = table(tab, dev, R);
  a.table_stride = tab.stride(0);
  a.free_blocks = ints(free, "free_blocks", dev);
  a.n_seqs = size_of(R, "the number of requests");
  a.max_blocks = size_of(tab.size(1), "max_blocks");
  a.block_size = (int)integer(x[5], "block_size");
  a.free_capacity = size_of(free.numel(), "the length of free_blocks");
  if (x[6] != Py_None) {
    const at::Tensor &shares = tensor(x[6], "shares");
    a.shares = ints(shares, "shares", dev);
    a.n_blocks = size_of(shares.numel(), "the length of shares");
  }
  const c10::DeviceGuard guard(dev);
  const at::Tensor buffer = empty({R + 1}, at::kInt, dev);
  a.lens_out = static_cast<int32_t *>(buffer.data_ptr());
  a.n_free_out = a.lens_out + R;
  check(g_release(&a, stream_of(dev)));
  return wrap_all(part(buffer, 0, R), part(buffer, R, 1));
}

// append(k, v, k_cache, v_cache, slots, positions, rope, q, q_out, k_scale, v_scale, k_pairs)
PyObject *append(PyObject *const *x) {
  const at::Tensor &k = tensor(x[0], "k"), &v = tensor(x[1], "v"), &kc = tensor(x[2], "k_cache"), &vc = tensor(x[3], "v_cache"),
                   &slots = tensor(x[4], "slots");
  const at::Device dev = k.device();
  kie_paged_append_args a = {};
  a.pages = pages(kc, vc, x[9], x[10], dev);
  need(k.dim() == 3 && k.size(1) == kc.size(1) && k.size(2) == kc.size(3),
       "k must be [rows, n_kv_heads, head_dim] like the pages");
  const int64_t T = k.size(0), dh = k.size(2);
  a.n_rows = size_of(T, "the number of rows");
  a.x_dtype = kind(k);
  a.k = rows(k, "k", k.sizes(), k.scalar_type(), dev, a.k_stride);
  a.v = rows(v, "v", k.sizes(), k.scalar_type(), dev, a.v_stride);
  a.slots = ints(slots, "slots", dev, T);
  if (x[6] != Py_None) {
    need(x[5] != Py_None, "a rope table needs positions");
    const at::Tensor &rope = tensor(x[6], "rope");
    need(rope.scalar_type() == at::kFloat && rope.dim() == 3 && rope.size(1) == dh / 2 && rope.size(2) == 2 &&
             rope.is_contiguous() && rope.device() == dev,
         "rope must be a contiguous float32 [n_pos, head_dim / 2, 2] tensor on the rows' device");
    a.positions = ints(tensor(x[5], "positions"), "positions", dev, T);
    a.rope = static_cast<const float *>(rope.data_ptr());
    a.n_pos = size_of(rope.size(0), "n_pos");
  }
  const int pairs = PyObject_IsTrue(x[11]);
  if (pairs < 0) throw Raised();
  a.k_pairs = pairs;
  const c10::DeviceGuard guard(dev);
  at::Tensor q_out;
  PyObject *result = x[8];
  if (x[7] != Py_None) {
    const at::Tensor &q = tensor(x[7], "q");
    need(q.dim() == 3 && q.size(0) == T && q.size(2) == dh, "q must be [rows, n_heads, head_dim] like k");
    a.n_heads = size_of(q.size(1), "n_heads");
    a.q = rows(q, "q", q.sizes(), k.scalar_type(), dev, a.q_stride);
    q_out = x[8] != Py_None ? tensor(x[8], "q_out") : empty(q.sizes(), q.scalar_type(), dev);
    a.q_out = rows(q_out, "q_out", q.sizes(), k.scalar_type(), dev, a.q_out_stride);
  }
  check(g_append(&a, stream_of(dev)));
  if (x[7] != Py_None && x[8] == Py_None) return wrap(q_out);
  Py_INCREF(result);
  return result;
}

// What attention and prefix_attention have in common: arguments 0 .. 12, checked, and outputs; all but the workspace.
struct Attention {
  kie_paged_attention_args a = {};
  at::Tensor out, lse;
};
void prepare(PyObject *const *x, const at::Device &dev, Attention &t) {
  kie_paged_attention_args &a = t.a;
  const at::Tensor &q = tensor(x[0], "q"), &kc = tensor(x[1], "k_cache"), &vc = tensor(x[2], "v_cache"),
                   &tab = tensor(x[3], "block_table");
  a.pages = pages(kc, vc, x[7], x[8], dev);
  need(q.dim() == 3 && q.size(2) == kc.size(3), "q must be [sequences, n_heads, head_dim] like the pages");
  const int64_t B = q.size(0), H = q.size(1), dh = q.size(2);
  a.n_seqs = size_of(B, "the number of sequences");
  a.n_heads = size_of(H, "n_heads");
  a.q_dtype = kind(q);
  a.q = rows(q, "q", q.sizes(), q.scalar_type(), dev, a.q_stride);
  if (x[11] != Py_None || x[12] != Py_None) {
    need(x[4] == Py_None && x[11] != Py_None && x[12] != Py_None, "either lens or both seqs and positions are needed");
    a.seqs = ints(tensor(x[11], "seqs"), "seqs", dev, B);
    a.positions = ints(tensor(x[12], "positions"), "positions", dev, B);
    a.n_table = size_of(tab.dim() > 0 ? tab.size(0) : 0, "the number of the block table's rows");
  } else {
    a.lens = ints(tensor(x[4], "lens"), "lens", dev, B);
  }
  a.block_table = table(tab, dev, a.seqs ? a.n_table : B);
  a.table_stride = tab.stride(0);
  a.max_blocks = size_of(tab.size(1), "max_blocks");
  a.window = (int)integer(x[6], "window");
  double scale = 0.0;
  if (x[5] != Py_None) {
    scale = PyFloat_AsDouble(x[5]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised();
  }
  a.scale = x[5] != Py_None ? (float)scale : dh == 64 ? 0.125f : dh == 128 ? 0.08838834764831845f : 0.f;
  const int with_lse = PyObject_IsTrue(x[10]);
  if (with_lse < 0) throw Raised();
  t.out = x[9] != Py_None ? tensor(x[9], "out") : empty(q.sizes(), q.scalar_type(), dev);
  a.out = rows(t.out, "out", q.sizes(), q.scalar_type(), dev, a.out_stride);
  if (with_lse) {
    t.lse = empty({B, H}, at::kFloat, dev);
    a.lse = static_cast<float *>(t.lse.data_ptr());
  }
}

// out, as it was given or new, and lse if it was asked for.
PyObject *results(PyObject *given, Attention &t) {
  PyObject *o = given;
  if (o == Py_None)
    o = wrap(t.out);
  else
    Py_INCREF(o);
  if (!t.lse.defined()) return o;
  PyObject *l = THPVariable_Wrap(t.lse), *both = l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(l);
  if (!both) throw Raised();
  return both;
}

// attention(q, k_cache, v_cache, block_table, lens, scale, window, k_scale, v_scale, out, return_lse, seqs, positions)
PyObject *attention(PyObject *const *x) {
  const at::Device dev = tensor(x[0], "q").device();
  need(dev.is_cuda(), "q must be a CUDA tensor");
  const c10::DeviceGuard guard(dev);
  Attention t;
  prepare(x, dev, t);
  kie_paged_attention_args &a = t.a;
  a.workspace_bytes = g_workspace(a.n_heads, a.pages.n_kv_heads, a.pages.head_dim);
  const at::Tensor workspace = empty({(int64_t)a.workspace_bytes}, at::kByte, dev);
  a.workspace = workspace.data_ptr();
  check(g_attention(&a, stream_of(dev)));
  return results(x[9], t);
}

// prefix_attention(the arguments of attention, group_start, prefix_lens)
PyObject *prefix_attention(PyObject *const *x) {
  const at::Device dev = tensor(x[0], "q").device();
  need(dev.is_cuda(), "q must be a CUDA tensor");
  const c10::DeviceGuard guard(dev);
  Attention t;
  prepare(x, dev, t);
  kie_paged_prefix_attention_args p = {};
  const at::Tensor &start = tensor(x[13], "group_start"), &prefix = tensor(x[14], "prefix_lens");
  p.n_groups = size_of(prefix.numel(), "the number of groups");
  p.prefix_lens = ints(prefix, "prefix_lens", dev);
  p.group_start = ints(start, "group_start", dev, (int64_t)p.n_groups + 1);
  t.a.workspace_bytes = g_prefix_workspace(t.a.n_seqs, t.a.n_heads, t.a.pages.n_kv_heads, t.a.pages.head_dim);
  const at::Tensor workspace = empty({(int64_t)t.a.workspace_bytes}, at::kByte, dev);
  t.a.workspace = workspace.data_ptr();
  p.a = t.a;
  check(g_prefix_attention(&p, stream_of(dev)));
  return results(x[9], t);
}

// fork(parents, lens, block_table, shares, free_blocks, n_free, block_size)
PyObject *fork(PyObject *const *x) {
  const at::Tensor &parents = tensor(x[0], "parents"), &lens = tensor(x[1], "lens"), &tab = tensor(x[2], "block_table"),
                   &shares = tensor(x[3], "shares"), &free = tensor(x[4], "free_blocks"), &n_free = tensor(x[5], "n_free");
  const at::Device dev = lens.device();
  const int64_t R = lens.numel();
  need(dev.is_cuda(), "lens must be a CUDA tensor");
  kie_paged_fork_args a = {};
  a.lens = ints(lens, "lens", dev);
  a.parents = ints(parents, "parents", dev, R);
  a.shares = ints(shares, "shares", dev);
  a.free_blocks = ints(free, "free_blocks", dev);
  a.n_free = ints(n_free, "n_free", dev, 1);
  a.block_table = table(tab, dev, R);
  a.table_stride = tab.stride(0);
  a.n_seqs = size_of(R, "the number of requests");
  a.max_blocks = size_of(tab.size(1), "max_blocks");
  a.block_size = (int)integer(x[6], "block_size");
  a.n_blocks = size_of(shares.numel(), "the length of shares");
  a.free_capacity = size_of(free.numel(), "the length of free_blocks");
  const c10::DeviceGuard guard(dev);
  const at::Tensor ok = empty({1}, at::kBool, dev), buffer = empty({4 * R + 1}, at::kInt, dev);
  a.workspace_bytes = (size_t)R * a.max_blocks * 4;
  const at::Tensor workspace = empty({(int64_t)a.workspace_bytes}, at::kByte, dev);
  a.workspace = workspace.data_ptr();
  a.ok = static_cast<uint8_t *>(ok.data_ptr());
  a.lens_out = static_cast<int32_t *>(buffer.data_ptr());
  a.n_free_out = a.lens_out + R;
  a.copy_src = a.n_free_out + 1;
  a.copy_dst = a.copy_src + R;
  a.copy_rows = a.copy_dst + R;
  check(g_fork(&a, stream_of(dev)));
  return wrap_all(part(buffer, 0, R), part(buffer, R, 1), ok, part(buffer, R + 1, R), part(buffer, 2 * R + 1, R),
                  part(buffer, 3 * R + 1, R));
}

// copy(src, dst, k_cache, v_cache, rows, k_scale, v_scale): caches [n_layers, n_blocks, ...] or one layer's
PyObject *copy(PyObject *const *x) {
  const at::Tensor &src = tensor(x[0], "src"), &dst = tensor(x[1], "dst"), &kc = tensor(x[2], "k_cache"),
                   &vc = tensor(x[3], "v_cache");
  const at::Device dev = kc.device();
  kie_paged_copy_args a = {};
  a.n_layers = 1;
  const bool layers = kc.dim() == 5;
  if (layers) {
    need(vc.sizes() == kc.sizes(), "k_cache and v_cache must have one shape");
    need(kc.size(0) >= 1, "the cache has no layers");
    a.n_layers = size_of(kc.size(0), "the number of layers");
    a.k_layer_stride = kc.stride(0);
    a.v_layer_stride = vc.stride(0);
    at::Tensor ks, vs;  // layer 0's, as pages() takes them
    PyObject *scales[2] = {x[5], x[6]};
    for (int i = 0; i < 2; ++i) {
      if (scales[i] == Py_None) continue;
      const at::Tensor &s = tensor(scales[i], "a scale");
      need(s.dim() == 4 && s.size(0) == kc.size(0), "the scales are float32 [n_layers, n_blocks, n_kv_heads, block_size] tensors");
      (i ? a.v_scale_layer_stride : a.k_scale_layer_stride) = s.stride(0);
      (i ? vs : ks) = s.select(0, 0);
    }
    PyObject *k0 = ks.defined() ? wrap(ks) : Py_None, *v0 = nullptr;
    try {
      v0 = vs.defined() ? wrap(vs) : Py_None;
      a.pages = pages(kc.select(0, 0), vc.select(0, 0), k0, v0, dev);
    } catch (...) {
      if (ks.defined()) Py_DECREF(k0);
      if (vs.defined()) Py_XDECREF(v0);
      throw;
    }
    if (ks.defined()) Py_DECREF(k0);
    if (vs.defined()) Py_DECREF(v0);
  } else {
    a.pages = pages(kc, vc, x[5], x[6], dev);
  }
  a.n_pairs = size_of(src.numel(), "the number of pairs");
  a.src = ints(src, "src", dev);
  a.dst = ints(dst, "dst", dev, a.n_pairs);
  if (x[4] != Py_None) a.rows = ints(tensor(x[4], "rows"), "rows", dev, a.n_pairs);
  const c10::DeviceGuard guard(dev);
  check(g_copy(&a, stream_of(dev)));
  Py_RETURN_NONE;
}

// compact(lens, block_table, shares, free_blocks, n_free, block_size)
PyObject *compact(PyObject *const *x) {
  const at::Tensor &lens = tensor(x[0], "lens"), &tab = tensor(x[1], "block_table"), &shares = tensor(x[2], "shares"),
                   &free = tensor(x[3], "free_blocks"), &n_free = tensor(x[4], "n_free");
  const at::Device dev = lens.device();
  const int64_t R = lens.numel(), n = shares.numel(), most = n / 2;
  need(dev.is_cuda(), "lens must be a CUDA tensor");
  kie_paged_compact_args a = {};
  a.lens = ints(lens, "lens", dev);
  a.shares = ints(shares, "shares", dev);
  a.free_blocks = ints(free, "free_blocks", dev);
  a.n_free = ints(n_free, "n_free", dev, 1);
  a.block_table = table(tab, dev, R);
  a.table_stride = tab.stride(0);
  a.n_seqs = size_of(R, "the number of requests");
  a.max_blocks = size_of(tab.size(1), "max_blocks");
  a.block_size = (int)integer(x[5], "block_size");
  a.n_blocks = size_of(n, "the length of shares");
  a.free_capacity = size_of(free.numel(), "the length of free_blocks");
  const c10::DeviceGuard guard(dev);
  const at::Tensor buffer = empty({1 + 2 * most + n}, at::kInt, dev);
  a.n_free_out = static_cast<int32_t *>(buffer.data_ptr());
  a.src = a.n_free_out + 1;
  a.dst = a.src + most;
  a.page_map = a.dst + most;
  check(g_compact(&a, stream_of(dev)));
  return wrap_all(part(buffer, 0, 1), part(buffer, 1, most), part(buffer, 1 + most, most), part(buffer, 1 + 2 * most, n));
}

// logprobs(logits, tokens, top)
PyObject *logprobs(PyObject *const *x) {
  const at::Tensor &logits = tensor(x[0], "logits");
  const at::Device dev = logits.device();
  kie_token_logprobs_args a = {};
  need(dev.is_cuda() && logits.dim() == 2 && logits.stride(1) == 1, "logits must be a CUDA tensor [rows, vocab] with contiguous rows");
  a.dtype = kind(logits);
  need(a.dtype >= 0 && a.dtype != KIE_E4M3, "logits are float16, bfloat16 or float32");
  const int64_t N = logits.size(0);
  a.n_rows = size_of(N, "the number of rows");
  a.vocab = size_of(logits.size(1), "vocab");
  a.logits = logits.data_ptr();
  a.row_stride = logits.stride(0);
  a.tokens = ints(tensor(x[1], "tokens"), "tokens", dev, N);
  a.top = (int)integer(x[2], "top");
  need(a.top >= 0 && a.top <= KIE_MAX_TOP && a.top <= a.vocab, "top must be from 0 to 32 and at most vocab");
  const c10::DeviceGuard guard(dev);
  const int64_t k = a.top;
  const at::Tensor floats = empty({(2 + k) * N}, at::kFloat, dev), top_ids = empty({N, k}, at::kInt, dev);
  float *f = static_cast<float *>(floats.data_ptr());
  a.logprob = f;
  a.entropy = f + N;
  a.top_logprobs = f + 2 * N;
  a.top_ids = static_cast<int32_t *>(top_ids.data_ptr());
  check(g_logprobs(&a, stream_of(dev)));
  at::Tensor top = part(floats, 2 * N, k * N);
  top.unsafeGetTensorImpl()->set_sizes_contiguous({N, k});
  return wrap_all(part(floats, 0, N), part(floats, N, N), top_ids, top);
}

// No C++ exception passes into Python.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are expected, not %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised &) {
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// bind(extend, release, append, attention, attention_workspace, last_error, prefix_attention, prefix_attention_workspace,
// fork, copy, compact, token_logprobs, KieError)
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long p[12];
  PyObject *error;
  if (!PyArg_ParseTuple(args, "KKKKKKKKKKKKO", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7], &p[8], &p[9], &p[10],
                        &p[11], &error))
    return nullptr;
  g_extend = reinterpret_cast<decltype(g_extend)>(p[0]);
  g_release = reinterpret_cast<decltype(g_release)>(p[1]);
  g_append = reinterpret_cast<decltype(g_append)>(p[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[3]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[4]);
  g_last_error = reinterpret_cast<decltype(g_last_error)>(p[5]);
  g_prefix_attention = reinterpret_cast<decltype(g_prefix_attention)>(p[6]);
  g_prefix_workspace = reinterpret_cast<decltype(g_prefix_workspace)>(p[7]);
  g_fork = reinterpret_cast<decltype(g_fork)>(p[8]);
  g_copy = reinterpret_cast<decltype(g_copy)>(p[9]);
  g_compact = reinterpret_cast<decltype(g_compact)>(p[10]);
  g_logprobs = reinterpret_cast<decltype(g_logprobs)>(p[11]);
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

#define FAST(f, n) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<f, n>)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"extend", FAST(extend, 7), nullptr},
                         {"release", FAST(release, 7), nullptr},
                         {"append", FAST(append, 12), nullptr},
                         {"attention", FAST(attention, 13), nullptr},
                         {"prefix_attention", FAST(prefix_attention, 15), nullptr},
                         {"fork", FAST(fork, 7), nullptr},
                         {"copy", FAST(copy, 7), nullptr},
                         {"compact", FAST(compact, 6), nullptr},
                         {"logprobs", FAST(logprobs, 3), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
