// The Python side of the serving-pass operators (serving.py) as a CPython
// module: argument checks, output allocation and the call of the C entry point
// in one function each.  A pass makes these calls once a layer, and at small
// batches the host's time is what they cost: checked and marshalled in Python
// through ctypes they took 8.4-14.6 us each, more than their kernels; here
// kv_write takes 3.3, process_logits 4.5, batch_layout 5.4 and tree_attention
// 6.8 us, launches included.  Only host code: the compute is behind
// include/awq.h.
#include <torch/csrc/python_headers.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <map>
#include <string>
#include <utility>

#include "awq.h"

namespace {

using at::Tensor;

// A refused argument: becomes the Python exception `kind`.
struct Refused {
  PyObject* kind;
  std::string what;
};
[[noreturn]] void value_error(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }
[[noreturn]] void type_error(std::string what) { throw Refused{PyExc_TypeError, std::move(what)}; }
struct PythonError {};  // already set

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}
std::string text(at::ScalarType t) {
  return std::string("torch.") + torch::getTHPDtype(t)->name;
}

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor* maybe(const char* name, PyObject* o) {
  return o == Py_None ? nullptr : &tensor(name, o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}

void on_device(const char* name, const Tensor& t, at::Device device) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be on a HIP device (no CPU fallback)");
  if (t.device() != device)
    value_error(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
}

// Checks a small contiguous operand (a copy would be made on every call and an
// output could not be copied at all, so none is made).
void need(const char* name, const Tensor& t, at::ScalarType dtype, at::IntArrayRef shape,
          at::Device device) {
  on_device(name, t, device);
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " must be " + text(dtype) + ", got " + text(t.scalar_type()));
  if (t.sizes() != shape)
    value_error(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}
// Words of the masks of n tokens, at least one: no words would be no mask.
int64_t need_mask(const Tensor& t, int64_t n, at::Device device) {
  const int64_t words = t.dim() ? t.size(-1) : 0;
  need("tree_mask", t, at::kLong, {n, words}, device);
  if (words == 0 && n > 0) value_error("tree_mask must have a word or more for each token");
  return words;
}
const void* pointer(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

int act_dtype(at::ScalarType t) {
  return t == at::kHalf ? AWQ_F16 : t == at::kBFloat16 ? AWQ_BF16 : -1;
}
int cache_dtype(at::ScalarType t) {
  return t == at::kFloat8_e4m3fn ? AWQ_E4M3 : act_dtype(t);
}

Tensor new_tensor(at::IntArrayRef shape, at::ScalarType dtype, at::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
}
// `n` elements of a 1-D tensor from `from` on, as a tensor of their own.
Tensor slice(const Tensor& t, int64_t from, int64_t n) {
  Tensor v = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(t.storage()),
                                                      t.key_set(), t.dtype());
  v.unsafeGetTensorImpl()->set_storage_offset(from);
  v.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return v;
}

void* stream_of(at::Device device) {
  return c10::hip::getCurrentHIPStream(device.index()).stream();
}

// Calls f, which returns a new reference, and turns what it throws into a
// Python exception.
template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.kind, r.what.c_str());
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}
// The C call without the interpreter's lock, as ctypes makes it, and with the
// tensors' device current: a launch goes to the current one, and the null
// stream is that one's.  f reads no tensor: another thread may change one, and
// one without memory throws.
template <class F>
int unlocked(at::Device device, F f) {
  const c10::hip::HIPGuard guard(device.index());
  const struct Release {
    PyThreadState* state = PyEval_SaveThread();
    ~Release() { PyEval_RestoreThread(state); }
  } release;
  return f();
}
PyObject* status(int st) { return PyLong_FromLong(st); }

// (cached_lens, new_counts, blocks_held, free_blocks, block_table, block_size,
// num_blocks, num_tokens, parents, mask_words, free_start) -> the fields of
// BatchLayout, or a status.
PyObject* batch_layout(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded(count, 11, [&]() -> PyObject* {
    const Tensor& table = tensor("block_table", args[4]);
    const at::Device device = table.device();
    if (!table.is_cuda()) on_device("block_table", table, device);
    if (table.dim() != 2) value_error("block_table must be (B, W), got " + text(table.sizes()));
    const int64_t B = table.size(0), W = table.size(1), T = integer(args[7]);
    if (T < 0) value_error("num_tokens must not be negative");
    const at::ScalarType i32 = at::kInt;
    const Tensor &cached = tensor("cached_lens", args[0]), &counts = tensor("new_counts", args[1]),
                 &held = tensor("blocks_held", args[2]), &free = tensor("free_blocks", args[3]);
    const Tensor *parents = maybe("parents", args[8]), *start = maybe("free_start", args[10]);
    need("block_table", table, i32, {B, W}, device);
    need("cached_lens", cached, i32, {B}, device);
    need("new_counts", counts, i32, {B}, device);
    need("blocks_held", held, i32, {B}, device);
    need("free_blocks", free, i32, {free.numel()}, device);
    if (parents) need("parents", *parents, i32, {T}, device);
    if (start) need("free_start", *start, i32, {1}, device);
    const int64_t words = args[9] == Py_None ? (parents ? 1 : 0) : integer(args[9]);
    if (words < 0) value_error("mask_words must not be negative");
    const int64_t block_size = integer(args[5]), num_blocks = integer(args[6]);
    if (T > (int64_t{1} << 31)) return status(AWQ_ERROR_SHAPE);   // before it is allocated
    const Tensor whole = new_tensor({3 * T + 2 * B + 5}, i32, device);
    Tensor mask;
    if (words) mask = new_tensor({T, words}, at::kLong, device);
    // slots, positions, requests, q_start, blocks_held, status
    const std::array<int64_t, 6> sizes = {T, T, T, B + 1, B, 4};
    std::array<Tensor, 6> part;
    int64_t at = 0;
    for (size_t i = 0; i < 6; ++i) {
      part[i] = slice(whole, at, sizes[i]);
      at += sizes[i];
    }
    int32_t* p = whole.data_ptr<int32_t>();
    const void *pc = cached.data_ptr(), *pn = counts.data_ptr(), *ph = held.data_ptr(),
               *pf = free.data_ptr(), *ps = pointer(start), *pp = pointer(parents);
    void *pt = table.data_ptr(), *pm = words ? mask.data_ptr() : nullptr;
    const int64_t num_free = free.numel();
    void* stream = stream_of(device);
    const int st = unlocked(device, [&] {
      return awq_batch_layout(pc, pn, ph, pf, ps, pp, pt, p + 3 * T, p, p + T, p + 2 * T, pm,
                              p + 3 * T + B + 1, p + 3 * T + 2 * B + 1, B, T, num_free, W,
                              block_size, num_blocks, words, stream);
    });
    if (st != AWQ_SUCCESS) return status(st);
    PyObject* out = PyTuple_New(7);
    if (!out) throw PythonError{};
    const int order[] = {3, 0, 1, 2, -1, 4, 5};
    for (int i = 0; i < 7; ++i) {
      PyObject* o = nullptr;
      if (order[i] >= 0) {
        o = THPVariable_Wrap(part[order[i]]);
      } else if (words) {
        o = THPVariable_Wrap(mask);
      } else {
        Py_INCREF(Py_None);
        o = Py_None;
      }
      PyTuple_SET_ITEM(out, i, o);
    }
    return out;
  });
}

awq_kv_cache cache_of(const Tensor& k, const Tensor& v, const Tensor* k_scale, const Tensor* v_scale) {
  const at::Device device = k.device();
  if (!k.is_cuda() || v.device() != device) {
    on_device("k_cache", k, device);
    on_device("v_cache", v, device);
  }
  if (k.dim() != 4 || v.sizes() != k.sizes())
    value_error("k_cache and v_cache must both be (num_blocks, block_size, heads, head_dim), got " +
                text(k.sizes()) + " and " + text(v.sizes()));
  if (v.scalar_type() != k.scalar_type() || cache_dtype(k.scalar_type()) < 0)
    type_error("k_cache and v_cache must both be float16, bfloat16 or float8_e4m3fn");
  const at::IntArrayRef ks = k.strides(), vs = v.strides();
  if (ks[3] != 1 || vs[3] != 1) value_error("the channels of k_cache and v_cache must be contiguous");
  if (k_scale) need("k_scale", *k_scale, at::kFloat, {k.size(2)}, device);
  if (v_scale) need("v_scale", *v_scale, at::kFloat, {k.size(2)}, device);
  awq_kv_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.k_scale = pointer(k_scale);
  c.v_scale = pointer(v_scale);
  c.num_blocks = k.size(0);
  c.block_size = k.size(1);
  c.heads = k.size(2);
  c.head_dim = k.size(3);
  c.k_block_stride = ks[0];
  c.k_slot_stride = ks[1];
  c.k_head_stride = ks[2];
  c.v_block_stride = vs[0];
  c.v_slot_stride = vs[1];
  c.v_head_stride = vs[2];
  c.dtype = cache_dtype(k.scalar_type());
  return c;
}

// (k, v, slots, k_cache, v_cache, k_scale, v_scale) -> status
PyObject* kv_write(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded(count, 7, [&]() -> PyObject* {
    const Tensor &k = tensor("k", args[0]), &v = tensor("v", args[1]), &slots = tensor("slots", args[2]),
                 &kc = tensor("k_cache", args[3]), &vc = tensor("v_cache", args[4]);
    const awq_kv_cache cache = cache_of(kc, vc, maybe("k_scale", args[5]), maybe("v_scale", args[6]));
    const at::Device device = kc.device();
    on_device("k", k, device);
    on_device("v", v, device);
    const int dtype = act_dtype(k.scalar_type());
    if (dtype < 0 || v.scalar_type() != k.scalar_type())
      type_error("k and v must both be float16 or bfloat16");
    if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(1) != cache.heads || k.size(2) != cache.head_dim)
      value_error("k and v must both be (T, " + std::to_string(cache.heads) + ", " +
                  std::to_string(cache.head_dim) + "), got " + text(k.sizes()) + " and " + text(v.sizes()));
    const int64_t T = k.size(0);
    need("slots", slots, at::kInt, {T}, device);
    const at::IntArrayRef ks = k.strides(), vs = v.strides();
    if (ks[2] != 1 || vs[2] != 1) value_error("the channels of k and v must be contiguous");
    const void *pk = k.data_ptr(), *pv = v.data_ptr(), *ps = slots.data_ptr();
    const int64_t kts = ks[0], khs = ks[1], vts = vs[0], vhs = vs[1];
    void* stream = stream_of(device);
    return status(unlocked(device, [&] {
      return awq_kv_write(pk, pv, ps, &cache, T, kts, khs, vts, vhs, dtype, stream);
    }));
  });
}

// Workspaces by device and stream, from the function that serving.py sets (the
// one that awq_gemm's come from).  A buffer that it has replaced by a larger
// one stays allocated, so one held here stays valid.  While that function
// runs, another thread may come here for the same stream: each takes the
// buffer that it was given.
PyObject* workspace_source = nullptr;
Tensor workspace_for(at::Device device, void* stream, size_t bytes) {
  static auto* held = new std::map<std::pair<int, void*>, Tensor>;   // lives as long as the process
  Tensor& t = (*held)[{device.index(), stream}];
  if (t.defined() && static_cast<size_t>(t.numel()) >= bytes) return t;
  if (!workspace_source) throw Refused{PyExc_RuntimeError, "no source of workspaces"};
  PyObject* o = PyObject_CallFunction(workspace_source, "iKK", static_cast<int>(device.index()),
                                      static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(stream)),
                                      static_cast<unsigned long long>(bytes));
  if (!o) throw PythonError{};
  const Tensor given = tensor("workspace", o);
  Py_DECREF(o);
  t = given;
  return given;
}
PyObject* set_workspace_source(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(workspace_source, f);
  Py_RETURN_NONE;
}

// (q, k_cache, v_cache, block_table, cached_lens, q_start, tree_mask, k_scale,
// v_scale, scale, out, workspace) -> out, or a status
PyObject* tree_attention(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded(count, 12, [&]() -> PyObject* {
    const Tensor &q = tensor("q", args[0]), &kc = tensor("k_cache", args[1]),
                 &vc = tensor("v_cache", args[2]), &table = tensor("block_table", args[3]),
                 &cached = tensor("cached_lens", args[4]), &q_start = tensor("q_start", args[5]);
    const awq_kv_cache cache = cache_of(kc, vc, maybe("k_scale", args[7]), maybe("v_scale", args[8]));
    const at::Device device = kc.device();
    on_device("q", q, device);
    const int dtype = act_dtype(q.scalar_type());
    if (dtype < 0 || (kc.scalar_type() != q.scalar_type() && kc.scalar_type() != at::kFloat8_e4m3fn))
      type_error("q must be float16 or bfloat16, and the cache the same or float8_e4m3fn");
    if (q.dim() != 3 || q.size(2) != cache.head_dim)
      value_error("q must be (T, heads, " + std::to_string(cache.head_dim) + "), got " + text(q.sizes()));
    const int64_t T = q.size(0), heads = q.size(1), dim = q.size(2);
    const at::IntArrayRef qs = q.strides();
    if (qs[2] != 1) value_error("the channels of q must be contiguous");
    if (table.dim() != 2 || table.scalar_type() != at::kInt)
      type_error("block_table must be a 2-D int32 tensor");
    on_device("block_table", table, device);
    const int64_t B = table.size(0), W = table.size(1);
    if (table.stride(1) != 1 && W > 1) value_error("the rows of block_table must be contiguous");
    need("cached_lens", cached, at::kInt, {B}, device);
    need("q_start", q_start, at::kInt, {B + 1}, device);
    const Tensor* mask = maybe("tree_mask", args[6]);
    const int64_t words = mask ? need_mask(*mask, T, device) : 0;
    double scale = 0.0;
    if (args[9] == Py_None) {
      scale = 1.0 / std::sqrt(static_cast<double>(dim));
    } else {
      scale = PyFloat_AsDouble(args[9]);
      if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
    }
    const Tensor* given = maybe("out", args[10]);
    if (given) need("out", *given, q.scalar_type(), {T, heads, dim}, device);
    const Tensor* ws = maybe("workspace", args[11]);
    if (ws) {
      on_device("workspace", *ws, device);
      if (!ws->is_contiguous()) value_error("workspace must be contiguous");
    }
    void* stream = stream_of(device);
    const size_t bytes = awq_tree_attention_workspace_size(B, T, heads, cache.heads, dim);
    const Tensor own = !ws && bytes ? workspace_for(device, stream, bytes) : Tensor();
    if (own.defined()) ws = &own;
    void* const ws_data = ws ? ws->data_ptr() : nullptr;
    const size_t ws_bytes = ws ? ws->nbytes() : 0;
    const Tensor out = given ? *given : new_tensor({T, heads, dim}, q.scalar_type(), device);
    const void *pq = q.data_ptr(), *pt = table.data_ptr(), *pc = cached.data_ptr(),
               *ps = q_start.data_ptr(), *pm = pointer(mask);
    void* po = out.data_ptr();
    const int64_t row = table.stride(0), qts = qs[0], qhs = qs[1];
    const int st = unlocked(device, [&] {
      return awq_tree_attention(pq, &cache, pt, pc, ps, pm, po, B, T, heads, W, row, words, qts, qhs,
                                scale, dtype, ws_data, ws_bytes, stream);
    });
    if (st != AWQ_SUCCESS) return status(st);
    if (given) {
      Py_INCREF(args[10]);
      return args[10];
    }
    return THPVariable_Wrap(out);
  });
}

// (logits, tokens, prompt_lens, lens, requests, repetition, frequency,
// presence, bias_ids, bias_values, grammar_mask, draft_tokens, tree_mask,
// q_start, out) -> out, or a status
PyObject* process_logits(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded(count, 15, [&]() -> PyObject* {
    const Tensor& logits = tensor("logits", args[0]);
    const at::Device device = logits.device();
    on_device("logits", logits, device);
    const at::ScalarType dtype = logits.scalar_type();
    if (act_dtype(dtype) < 0 && dtype != at::kFloat)
      type_error("logits must be float16, bfloat16 or float32");
    if (logits.dim() != 2 || logits.size(1) == 0) value_error("logits must be (rows, vocab)");
    const int64_t R = logits.size(0), V = logits.size(1);
    if (logits.stride(1) != 1 && V > 1) value_error("the entries of a row of logits must be contiguous");
    const Tensor* given = maybe("out", args[14]);
    if (given) {
      on_device("out", *given, device);
      if (given->scalar_type() != dtype || given->sizes() != logits.sizes() ||
          (given->stride(1) != 1 && V > 1))
        value_error("out must be like logits, with contiguous rows");
    }
    const Tensor *tokens = maybe("tokens", args[1]), *prompt_lens = maybe("prompt_lens", args[2]),
                 *lens = maybe("lens", args[3]), *requests = maybe("requests", args[4]),
                 *repetition = maybe("repetition", args[5]), *frequency = maybe("frequency", args[6]),
                 *presence = maybe("presence", args[7]), *bias_ids = maybe("bias_ids", args[8]),
                 *bias_values = maybe("bias_values", args[9]), *grammar = maybe("grammar_mask", args[10]),
                 *draft = maybe("draft_tokens", args[11]), *mask = maybe("tree_mask", args[12]),
                 *q_start = maybe("q_start", args[13]);
    // The batch is what any per-request operand says; all have to agree.
    int64_t B = -1;
    for (const Tensor* t : {lens, repetition, frequency, presence, bias_ids})
      if (t && B < 0 && t->dim() > 0) B = t->size(0);
    if (B < 0) B = q_start && q_start->dim() > 0 ? q_start->size(0) - 1 : R;
    awq_logits a{};
    a.rows = R;
    a.vocab = V;
    a.batch = B;
    a.logits_stride = logits.stride(0);
    a.dtype = dtype == at::kFloat ? AWQ_F32 : act_dtype(dtype);
    a.logits = R ? logits.data_ptr() : nullptr;
    if (requests) {
      need("requests", *requests, at::kInt, {R}, device);
      a.requests = requests->data_ptr();
    } else if ((tokens || repetition || frequency || presence || bias_ids) && B < R) {
      value_error(std::to_string(R) + " rows need requests: the batch has " + std::to_string(B));
    }
    if (tokens) {
      if (!prompt_lens || !lens) value_error("tokens needs prompt_lens and lens");
      on_device("tokens", *tokens, device);
      if (tokens->scalar_type() != at::kInt || tokens->dim() != 2 || tokens->size(0) != B ||
          (tokens->stride(1) != 1 && tokens->size(1) > 1))
        value_error("tokens must be int32 (" + std::to_string(B) + ", history) with contiguous rows");
      need("prompt_lens", *prompt_lens, at::kInt, {B}, device);
      need("lens", *lens, at::kInt, {B}, device);
      if (tokens->size(1)) {
        a.tokens = tokens->data_ptr();
        a.tokens_stride = tokens->stride(0);
        a.history = tokens->size(1);
        a.prompt_lens = prompt_lens->data_ptr();
        a.lens = lens->data_ptr();
      }
    }
    const auto per_request = [&](const char* name, const Tensor* t) -> const void* {
      if (t) need(name, *t, at::kFloat, {B}, device);
      return pointer(t);
    };
    a.repetition = per_request("repetition", repetition);
    a.frequency = per_request("frequency", frequency);
    a.presence = per_request("presence", presence);
    if ((bias_ids == nullptr) != (bias_values == nullptr))
      value_error("bias_ids and bias_values come together");
    if (bias_ids) {
      const int64_t n = bias_ids->dim() ? bias_ids->size(-1) : 0;
      need("bias_ids", *bias_ids, at::kInt, {B, n}, device);
      need("bias_values", *bias_values, at::kFloat, {B, n}, device);
      if (n) {
        a.bias_ids = bias_ids->data_ptr();
        a.bias_values = bias_values->data_ptr();
        a.biases = n;
      }
    }
    if (grammar) {
      on_device("grammar_mask", *grammar, device);
      const int64_t words = (V + 31) / 32;
      if (grammar->scalar_type() != at::kInt || grammar->sizes() != at::IntArrayRef({R, words}) ||
          (grammar->stride(1) != 1 && words > 1))
        value_error("grammar_mask must be int32 (" + std::to_string(R) + ", " + std::to_string(words) +
                    ") with contiguous rows");
      a.grammar_mask = grammar->data_ptr();
      a.grammar_stride = grammar->stride(0);
    }
    if (draft || mask || q_start) {
      if (!draft || !mask || !q_start)
        value_error("draft_tokens, tree_mask and q_start come together");
      need("draft_tokens", *draft, at::kInt, {R}, device);
      const int64_t words = need_mask(*mask, R, device);
      need("q_start", *q_start, at::kInt, {B + 1}, device);
      if (R) {
        a.draft_tokens = draft->data_ptr();
        a.tree_mask = mask->data_ptr();
        a.q_start = q_start->data_ptr();
        a.mask_words = words;
      }
    }
    const Tensor out = given ? *given : new_tensor({R, V}, dtype, device);
    a.out = R ? out.data_ptr() : nullptr;
    a.out_stride = out.stride(0);
    void* stream = stream_of(device);
    const int st = unlocked(device, [&] { return awq_process_logits(&a, stream); });
    if (st != AWQ_SUCCESS) return status(st);
    if (given) {
      Py_INCREF(args[14]);
      return args[14];
    }
    return THPVariable_Wrap(out);
  });
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {
    {"batch_layout", fast(batch_layout), METH_FASTCALL, nullptr},
    {"kv_write", fast(kv_write), METH_FASTCALL, nullptr},
    {"tree_attention", fast(tree_attention), METH_FASTCALL, nullptr},
    {"process_logits", fast(process_logits), METH_FASTCALL, nullptr},
    {"set_workspace_source", set_workspace_source, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__serving() {
  return PyModule_Create(&module);
}
