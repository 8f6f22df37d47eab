// The host side of the calls with axes, score rules and drafts: torch tensors in, one C entry
// point called.  Kernels of a decode step take 2 to 20 us; read from Python, a call's tensors
// and its 20 to 30 arguments cost 9 us of the host, here 1.  The checks are those of what the
// C entry cannot see (types, shapes, contiguity); their refusals are ValueErrors.
//
// Functions take their arguments by position, None for what is left out, and return the
// entry's status.  The module binds to the torch that is loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <limits>
#include <stdexcept>
#include <string>

#include "pkvqk.h"

namespace {

struct PythonRaised {};                        // the Python error is set already

[[noreturn]] void refuse(const std::string& words) { throw std::invalid_argument(words); }

// ------------------------------------------------------------- arguments

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %.100s", name, Py_TYPE(o)->tp_name);
    throw PythonRaised{};
  }
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, int64_t least, int64_t most, const char* name) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw PythonRaised{};
  if (n < least || n > most) refuse(std::string(name) + " is out of range");
  return n;
}
int32_t int32(PyObject* o, const char* name) {
  return static_cast<int32_t>(integer(o, std::numeric_limits<int32_t>::min(),
                                      std::numeric_limits<int32_t>::max(), name));
}
int32_t count32(int64_t n, const char* name) {
  if (n > std::numeric_limits<int32_t>::max()) refuse(std::string(name) + " is out of range");
  return static_cast<int32_t>(n);
}
float float32(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonRaised{};
  return static_cast<float>(x);
}
// The same where the entry takes 0 as a word of its own: what fp32 only has as 0 is refused.
float float32_or_0(PyObject* o, const char* name) {
  const float x = float32(o);
  if (x == 0.f && PyFloat_AsDouble(o) != 0.0) refuse(std::string(name) + " is out of range");
  return x;
}

template <typename T = void>
T* data(const at::Tensor& x) {
  return static_cast<T*>(x.data_ptr());
}

// n contiguous values of a type
template <typename T>
T* values(PyObject* o, at::ScalarType type, int64_t n, const char* name) {
  const at::Tensor& x = tensor(o, name);
  if (x.scalar_type() != type || !x.is_contiguous() || x.numel() != n) {
    const char* word = type == at::kInt ? "int32" : type == at::kLong ? "int64" : "float32";
    refuse(std::string(name) + " must be " + std::to_string(n) + " contiguous " + word +
           " values");
  }
  return data<T>(x);
}
template <typename T>
T* values_or_none(PyObject* o, at::ScalarType type, int64_t n, const char* name) {
  return o == Py_None ? nullptr : values<T>(o, type, n, name);
}

struct Heads {
  void* p;
  int64_t tokens, heads, stride_t, stride_h;
};
Heads heads(PyObject* o, const char* name) {
  const at::Tensor& x = tensor(o, name);
  if (x.scalar_type() != at::kBFloat16 || x.dim() != 3 || x.size(2) != 128 || x.stride(2) != 1)
    refuse(std::string(name) + " must be bfloat16 [tokens, heads, 128], head_dim the contiguous "
           "axis");
  return {data(x), x.size(0), x.size(1), x.stride(0), x.stride(1)};
}

const void* gains(PyObject* o, const char* name) {
  const at::Tensor& x = tensor(o, name);
  if (x.scalar_type() != at::kBFloat16 || x.numel() != 128 || !x.is_contiguous())
    refuse(std::string(name) + " must be 128 contiguous bfloat16 values");
  return data(x);
}

struct Caches {
  void *k, *v;
  pkvqk_cache_layout layout;
};
Caches caches(PyObject* ko, PyObject* vo) {
  const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  if (k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16)
    refuse("k_cache and v_cache must be bfloat16");
  if (k.sizes() != v.sizes() || k.strides() != v.strides())
    refuse("k_cache and v_cache must share one layout");
  if (k.dim() != 4 || k.stride(3) != 1)
    refuse("caches must be [num_blocks, block_size, num_kv_heads, head_dim], head_dim the "
           "contiguous axis");
  return {data(k), data(v),
          {k.size(0), count32(k.size(1), "block_size"), count32(k.size(2), "num_kv_heads"),
           count32(k.size(3), "head_dim"), 0, k.stride(0), k.stride(1), k.stride(2)}};
}

int32_t* flags(PyObject* o) {
  if (o == Py_None) return nullptr;
  const at::Tensor& x = tensor(o, "status_flags");
  if (x.scalar_type() != at::kInt || x.numel() < 1) refuse("status_flags must be int32");
  return data<int32_t>(x);
}

// The stream given, or the current one of q's device.
pkvqk_stream_t stream_of(PyObject* stream, PyObject* q) {
  if (stream != Py_None) {
    PyObject* handle = PyObject_GetAttrString(stream, "cuda_stream");
    if (handle == nullptr) throw PythonRaised{};
    const unsigned long long n = PyLong_AsUnsignedLongLong(handle);
    Py_DECREF(handle);
    if (n == static_cast<unsigned long long>(-1) && PyErr_Occurred()) throw PythonRaised{};
    return reinterpret_cast<pkvqk_stream_t>(static_cast<uintptr_t>(n));
  }
  const at::Tensor& x = THPVariable_Unpack(q);
  if (!x.is_cuda()) return nullptr;            // a host tensor is refused by the entry
  return reinterpret_cast<pkvqk_stream_t>(
      c10::cuda::getCurrentCUDAStream(x.get_device()).stream());
}

// A function of the module: refusals become ValueErrors, no exception leaves.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", wanted, given);
    return nullptr;
  }
  try {
    return PyLong_FromLong(static_cast<long>(f()));
  } catch (const PythonRaised&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// Without the interpreter's lock: a launch may wait for room in the stream's queue.
template <typename F>
pkvqk_status unlocked(F&& f) {
  pkvqk_status status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  return status;
}

// ---------------------------------------------------------------- append

PyObject* append_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    const Heads q = heads(a[0], "q");
    const Heads o = a[12] == Py_None ? q : heads(a[12], "q_out");
    const Heads k = heads(a[1], "k"), v = heads(a[2], "v");
    const Caches c = caches(a[10], a[11]);
    if (o.tokens != q.tokens || o.heads != q.heads || k.tokens != q.tokens ||
        v.tokens != q.tokens || k.heads != v.heads || k.heads != c.layout.num_kv_heads)
      refuse("q, q_out, k and v must agree in tokens, and k, v and the cache in heads");
    const at::Tensor& pos = tensor(a[3], "positions");
    if (pos.scalar_type() != at::kLong || pos.dim() != 2 || pos.size(1) != q.tokens ||
        (q.tokens > 1 && pos.stride(1) != 1))
      refuse("positions must be int64 [axes, tokens], the tokens contiguous");
    if (!PyBytes_Check(a[4]) || PyBytes_GET_SIZE(a[4]) != 64) refuse("freq_axes must be 64 bytes");
    const int32_t table_positions = int32(a[14], "table_positions");
    const void* table = nullptr;
    if (a[13] != Py_None) {
      static const size_t row_bytes = pkvqk_rope_table_bytes(1);
      const at::Tensor& x = tensor(a[13], "rope_table");
      if (!x.is_contiguous() ||
          static_cast<int64_t>(x.nbytes()) < table_positions * static_cast<int64_t>(row_bytes))
        refuse("rope_table must be contiguous and hold " + std::to_string(table_positions) +
               " positions");
      table = data(x);
    }
    const auto* axes = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[4]));
    const auto* slots = values<int64_t>(a[5], at::kLong, q.tokens, "slot_mapping");
    const void *gq = gains(a[6], "gamma_q"), *gk = gains(a[7], "gamma_k");
    const float theta = float32(a[8]), eps = float32(a[9]);
    const int32_t tokens = count32(q.tokens, "tokens"), num_heads = count32(q.heads, "heads");
    const int32_t num_axes = count32(pos.size(0), "axes");
    int32_t* status_flags = flags(a[15]);
    const pkvqk_stream_t stream = stream_of(a[16], a[0]);
    const auto* positions = data<int64_t>(pos);
    const int64_t stride_a = pos.stride(0);
    return unlocked([&] {
      return pkvqk_norm_rope_append_axes(
          q.p, q.stride_t, q.stride_h, o.p, o.stride_t, o.stride_h, k.p, k.stride_t, k.stride_h,
          v.p, v.stride_t, v.stride_h, positions, stride_a, num_axes, axes, slots, gq, gk, theta,
          eps, tokens, num_heads, c.k, c.v, &c.layout, table, table_positions, status_flags,
          stream);
    });
  });
}

// ------------------------------------------------------------- attention

// What the three entry points under score rules share, from the arguments behind their own.
struct Attention {
  Heads q;
  Caches c;
  const int32_t *table, *seq_lens;
  int32_t width, batch, splits, hint;
  float scale;
  pkvqk_score_rules rules;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int32_t* status_flags;
  pkvqk_stream_t stream;
};

// shared: k_cache, v_cache, block_tables, seq_lens, out; then softcap, window, slopes,
// first_keys, prefix_lens, num_splits, max_seq_len_hint, scale, lse_out, workspace,
// status_flags, stream
constexpr int kTensors = 5, kOptions = 12;

Attention attention(PyObject* q, int64_t q_len, PyObject* const* x, PyObject* const* r) {
  Attention t;
  t.q = heads(q, "q");
  const at::Tensor& lens = tensor(x[3], "seq_lens");
  const int64_t batch = lens.dim() > 0 ? lens.size(0) : -1;
  if (batch < 0) refuse("seq_lens must be int32 [batch]");
  if (q_len >= 0 && q_len * batch != t.q.tokens)
    refuse("q must hold q_len rows for each sequence of seq_lens");
  const at::Tensor& table = tensor(x[2], "block_tables");
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != batch ||
      !table.is_contiguous())
    refuse("block_tables must be contiguous int32 [batch, max_blocks_per_seq]");
  t.table = data<int32_t>(table);
  t.width = count32(table.size(1), "max_blocks_per_seq");
  // out and lse_out may hold more rows, which are left as they are
  const int64_t rows = t.q.tokens * t.q.heads;
  const at::Tensor& out = tensor(x[4], "out");
  if (out.scalar_type() != at::kBFloat16 || !out.is_contiguous() || out.numel() < rows * 128)
    refuse("out must be contiguous bfloat16, one value per value of q");
  t.out = data(out);
  t.lse = nullptr;
  if (r[8] != Py_None) {
    const at::Tensor& lse = tensor(r[8], "lse_out");
    if (lse.scalar_type() != at::kFloat || !lse.is_contiguous() || lse.numel() < rows)
      refuse("lse_out must be contiguous float32, one value per row and head");
    t.lse = data<float>(lse);
  }
  t.c = caches(x[0], x[1]);
  t.seq_lens = values<int32_t>(x[3], at::kInt, batch, "seq_lens");
  t.batch = count32(batch, "batch");
  t.rules.softcap = float32_or_0(r[0], "softcap");
  t.rules.window = int32(r[1], "window");
  t.rules.slopes = values_or_none<float>(r[2], at::kFloat, t.q.heads, "slopes");
  t.rules.first_keys = values_or_none<int32_t>(r[3], at::kInt, t.q.tokens, "first_keys");
  t.rules.prefix_lens = values_or_none<int32_t>(r[4], at::kInt, batch, "prefix_lens");
  t.splits = int32(r[5], "num_splits");
  t.hint = int32(r[6], "max_seq_len_hint");
  t.scale = float32_or_0(r[7], "scale");
  t.workspace = nullptr;
  t.workspace_bytes = 0;
  if (r[9] != Py_None) {
    const at::Tensor& ws = tensor(r[9], "workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
    t.workspace = data(ws);
    t.workspace_bytes = ws.nbytes();
  }
  t.status_flags = flags(r[10]);
  t.stream = stream_of(r[11], q);
  return t;
}

// q, the shared tensors, q_len, the options
template <typename Entry>
PyObject* even_rows(PyObject* const* a, Py_ssize_t n, Entry entry) {
  return guarded(n, 1 + kTensors + 1 + kOptions, [&] {
    const int32_t q_len = int32(a[1 + kTensors], "q_len");
    if (q_len < 0) refuse("q_len is out of range");
    const Attention t = attention(a[0], q_len, a + 1, a + 2 + kTensors);
    const int32_t num_heads = count32(t.q.heads, "heads");
    return unlocked([&] {
      return entry(t.q.p, t.q.stride_t, t.q.stride_h, t.c.k, t.c.v, &t.c.layout, t.table, t.width,
                   t.seq_lens, t.batch, q_len, num_heads, t.splits, t.hint, t.scale, &t.rules,
                   t.out, t.lse, t.workspace, t.workspace_bytes, t.status_flags, t.stream);
    });
  });
}
PyObject* decode_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return even_rows(a, n, pkvqk_paged_decode_scored);
}
PyObject* prefill_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return even_rows(a, n, pkvqk_paged_prefill_scored);
}

// q, cu_seqlens_q, max_q_len, the shared tensors, the options
PyObject* prefill_varlen_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3 + kTensors + kOptions, [&] {
    const Attention t = attention(a[0], -1, a + 3, a + 3 + kTensors);
    const auto* cu = values<int32_t>(a[1], at::kInt, t.batch + 1ll, "cu_seqlens_q");
    const int32_t longest = int32(a[2], "max_q_len");
    const int32_t num_heads = count32(t.q.heads, "heads");
    return unlocked([&] {
      return pkvqk_paged_prefill_varlen_scored(
          t.q.p, t.q.stride_t, t.q.stride_h, cu, longest, t.q.tokens, t.c.k, t.c.v, &t.c.layout,
          t.table, t.width, t.seq_lens, t.batch, num_heads, t.splits, t.hint, t.scale, &t.rules,
          t.out, t.lse, t.workspace, t.workspace_bytes, t.status_flags, t.stream);
    });
  });
}

// ---------------------------------------------------------------- drafts

// A [batch, >= rows, vocab] view whose rows are contiguous.
void rows_of(const at::Tensor& x, int64_t batch, int64_t rows, int64_t vocab, const char* name) {
  if (x.dim() != 3 || x.size(0) != batch || x.size(1) < rows || x.size(2) != vocab ||
      (vocab > 1 && x.stride(2) != 1))
    refuse(std::string(name) + " must be [batch, drafts, vocab], the vocabulary contiguous");
}

PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& target = tensor(a[0], "target_probs");
    const at::Tensor& drafted = tensor(a[2], "draft_tokens");
    if (drafted.dim() != 2) refuse("draft_tokens must be int32 [batch, drafts]");
    const int64_t B = drafted.size(0), K = drafted.size(1);
    const int64_t V = target.dim() > 0 ? target.size(-1) : 0;
    const at::ScalarType type = target.scalar_type();
    int32_t kind = 0;
    if (type == at::kFloat) kind = PKVQK_PROB_FP32;
    else if (type == at::kBFloat16) kind = PKVQK_PROB_BF16;
    else if (type == at::kHalf) kind = PKVQK_PROB_FP16;
    else refuse("target_probs must be float32, bfloat16 or float16");
    rows_of(target, B, K + 1, V, "target_probs");
    const void* draft = nullptr;
    int64_t draft_b = 0, draft_t = 0;
    if (a[1] != Py_None) {
      const at::Tensor& x = tensor(a[1], "draft_probs");
      if (x.scalar_type() != type) refuse("draft_probs must have target_probs' type");
      if (K > 0) {                             // without drafts none of it is read
        rows_of(x, B, K, V, "draft_probs");
        draft = data(x);
        draft_b = x.stride(0);
        draft_t = x.stride(1);
      }
    }
    const auto* tokens_in = values<int32_t>(a[2], at::kInt, B * K, "draft_tokens");
    const auto* lens = values_or_none<int32_t>(a[6], at::kInt, B, "draft_lens");
    const auto* uniforms = values<float>(a[3], at::kFloat, B * (K + 1), "uniforms");
    auto* tokens = values<int32_t>(a[4], at::kInt, B * (K + 1), "tokens");
    auto* accepted = values<int32_t>(a[5], at::kInt, B, "num_accepted");
    const auto* seq_lens = values_or_none<int32_t>(a[7], at::kInt, B, "seq_lens");
    auto* kept = values_or_none<int32_t>(a[8], at::kInt, B, "kept_lens");
    const int32_t b = count32(B, "batch"), k = count32(K, "drafts"), v = count32(V, "vocab");
    int32_t* status_flags = flags(a[9]);
    const pkvqk_stream_t stream = stream_of(a[10], a[0]);
    const void* p = data(target);
    const int64_t stride_b = target.stride(0), stride_t = target.stride(1);
    return unlocked([&] {
      return pkvqk_verify_drafts(p, stride_b, stride_t, draft, draft_b, draft_t, kind, tokens_in,
                                 lens, uniforms, b, k, v, tokens, accepted, seq_lens, kept,
                                 status_flags, stream);
    });
  });
}

// ---------------------------------------------------------------- module

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {
    method<append_axes>("append_axes"),
    method<decode_scored>("decode_scored"),
    method<prefill_scored>("prefill_scored"),
    method<prefill_varlen_scored>("prefill_varlen_scored"),
    method<verify_drafts>("verify_drafts"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "torch_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_torch_calls() { return PyModule_Create(&module); }
