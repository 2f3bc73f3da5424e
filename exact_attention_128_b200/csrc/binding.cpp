// binding.cpp — the Python side of the passes around attention, in C++ against torch: checks
// the tensors of a call, allocates what was not given, fills the call's struct (include/fa.h) and
// calls the C ABI on the current stream.  The library stays free of torch; its entry points come in
// as addresses (connect).
//
// These are the calls of a decode loop, a few microseconds on the device each.  Checked and packed
// in Python a call took 13 to 25 us of host time, most of it in reading tensors' attributes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <array>
#include <climits>
#include <initializer_list>

#include "../../include/fa.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// ---- the library

struct Api {
  decltype(&::fa_qk_norm_rope) qk_norm_rope;
  decltype(&::fa_qk_norm_rope_append) qk_norm_rope_append;
  decltype(&::fa_qk_norm_rope_bwd) qk_norm_rope_bwd;
  decltype(&::fa_qk_norm_rope_bwd_workspace_size) qk_norm_rope_bwd_workspace_size;
  decltype(&::fa_paged_decode_shared) paged_decode_shared;
  decltype(&::fa_paged_decode_shared_workspace_size) paged_decode_shared_workspace_size;
  decltype(&::fa_paged_decode_scored) paged_decode_scored;
  decltype(&::fa_paged_decode_scored_workspace_size) paged_decode_scored_workspace_size;
  decltype(&::fa_paged_evict) paged_evict;
  decltype(&::fa_paged_evict_workspace_size) paged_evict_workspace_size;
} api;
PyObject* error_class;  // FAError(name, status)

// ---- arguments

// What was given in a tensor's place, for messages.
std::string described(PyObject* o) {
  if (!THPVariable_Check(o)) return Py_TYPE(o)->tp_name;
  const Tensor& t = THPVariable_Unpack(o);
  return c10::str(t.scalar_type(), " ", t.sizes(), " with strides ", t.strides(), " on ", t.device());
}

const Tensor& tensor(PyObject* o, const char* name, int64_t dim) {
  TORCH_CHECK_VALUE(THPVariable_Check(o) && THPVariable_Unpack(o).dim() == dim, name, " must be a CUDA tensor of ",
                    dim, " dimensions, got ", described(o));
  return THPVariable_Unpack(o);
}

// The tensor that a call's others are held against.
const Tensor& first_tensor(PyObject* o, const char* name, int64_t dim) {
  const Tensor& t = tensor(o, name, dim);
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor, got ", described(o));
  return t;
}

// Address of a contiguous tensor of this shape and type on the CUDA device of this index.
template <typename P = void>
P* expect(PyObject* o, const char* name, IntArrayRef shape, ScalarType dtype, int64_t device) {
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == dtype && t.is_cuda() && t.get_device() == device && t.sizes() == shape && t.is_contiguous())
      return static_cast<P*>(t.data_ptr());
  }
  TORCH_CHECK_VALUE(false, name, " must be a contiguous ", dtype, " CUDA tensor of shape ", shape, " on device ", device,
                    ", got ", described(o));
}

// Address of a [B,H,N,d] view whose rows are contiguous, and its {batch, head, token} strides.
void* rows(PyObject* o, const char* name, IntArrayRef shape, ScalarType dtype, int64_t device, int64_t (&strides)[3]) {
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == dtype && t.is_cuda() && t.get_device() == device && t.sizes() == shape &&
        (t.stride(3) == 1 || shape[3] == 1)) {
      for (int i = 0; i < 3; ++i) strides[i] = shape[i] > 1 ? t.stride(i) : 0;  // (size 1: no stride of its own)
      return t.data_ptr();
    }
  }
  TORCH_CHECK_VALUE(false, name, " must be ", dtype, " ", shape, " with a contiguous last dimension on device ", device,
                    ", got ", described(o));
}

int integer(PyObject* o, const char* name) {
  int overflow = 0;
  PyObject* index = PyNumber_Index(o);
  if (!index) PyErr_Clear();
  const long long v = index ? PyLong_AsLongLongAndOverflow(index, &overflow) : 0;
  Py_XDECREF(index);
  TORCH_CHECK_VALUE(index && !overflow && v >= INT_MIN && v <= INT_MAX, name, " must be an integer of 32 bits, got ",
                    index ? "one past them" : Py_TYPE(o)->tp_name);
  return int(v);
}

// A size of a tensor (a dimension past 32 bits is refused).
int size32(int64_t v, const char* name) {
  TORCH_CHECK_VALUE(v <= INT_MAX, name, " is too large: ", v);
  return int(v);
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    TORCH_CHECK_VALUE(false, name, " must be a number, got ", Py_TYPE(o)->tp_name);
  }
  return float(v);
}

bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

int dtype_code(ScalarType t, const char* name) {
  TORCH_CHECK_VALUE(t == at::kFloat || t == at::kBFloat16, name, ": unsupported dtype ", t);
  return t == at::kFloat ? FA_DTYPE_F32 : FA_DTYPE_BF16;
}

// What was given, or a new contiguous tensor.
struct Output {
  Tensor made;
  PyObject* given;
  Output(PyObject* o, IntArrayRef shape, const at::TensorOptions& options) : given(o) {
    if (o == Py_None) made = at::empty(shape, options);
  }
  template <typename P = void>
  P* expect(const char* name, IntArrayRef shape, ScalarType dtype, int64_t device) {
    return made.defined() ? static_cast<P*>(made.data_ptr()) : ::expect<P>(given, name, shape, dtype, device);
  }
  PyObject* object() {  // a new reference
    if (made.defined()) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
  }
};

// The caller's workspace, or a new one, which lives until the call's work is in its stream.
struct Workspace {
  Tensor made;
  void* at = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, size_t need, const Tensor& like) {
    if (o == Py_None) {
      if (!need) return;
      made = at::empty({int64_t(need)}, like.options().dtype(at::kByte));
      at = made.data_ptr();
      bytes = need;
      return;
    }
    TORCH_CHECK_VALUE(THPVariable_Check(o), "workspace must be a tensor, got ", described(o));
    const Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == like.get_device() && t.is_contiguous(),
                      "workspace must be a contiguous tensor on ", like.device(), ", got ", described(o));
    at = t.data_ptr();
    bytes = t.nbytes();
  }
};

// Run one entry point on the device and its current stream.
template <typename A>
void call(const char* name, fa_status (*fn)(const A*, void*), const A& args, int64_t device) {
  fa_status status;
  {
    const c10::DeviceIndex index(static_cast<c10::DeviceIndex>(device));
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != index) guard.set_index(index);
    void* stream = c10::cuda::getCurrentCUDAStream(index).stream();
    Py_BEGIN_ALLOW_THREADS;
    status = fn(&args, stream);
    Py_END_ALLOW_THREADS;
  }
  if (status == FA_OK) return;
  PyObject* e = PyObject_CallFunction(error_class, "si", name, int(status));
  if (e) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  throw python_error();
}

PyObject* pack(std::initializer_list<PyObject*> items) {  // steals them
  PyObject* t = PyTuple_New(Py_ssize_t(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
  return t;
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// ---- norm and rotation

// The arguments that every rotary call shares: positions, frequencies, sections, pairing.
template <typename A>
void rope_arguments(A& a, PyObject* positions, PyObject* inv_freq, PyObject* sections, PyObject* interleaved,
                    PyObject* eps, int64_t B, int64_t N, int64_t device) {
  const int64_t half = tensor(inv_freq, "inv_freq", 1).size(0);
  a.inv_freq = expect<const double>(inv_freq, "inv_freq", {half}, at::kDouble, device);
  a.rotary_dim = size32(2 * half, "rotary_dim");
  TORCH_CHECK_VALUE(THPVariable_Check(positions), "positions must be a tensor, got ", described(positions));
  const Tensor& t = THPVariable_Unpack(positions);
  const int64_t dims = t.dim(), axes = dims == 3 ? t.size(0) : 1;
  const std::array<int64_t, 3> want{axes, B, N};
  TORCH_CHECK_VALUE(dims >= 1 && dims <= 3 && t.sizes() == IntArrayRef(want).slice(3 - dims),
                    "positions must be [N], [B,N] or [axes,B,N] with B = ", B, " and N = ", N, ", got ",
                    described(positions));
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.is_cuda() && t.get_device() == device &&
                        (N <= 1 || t.stride(dims - 1) == 1),
                    "positions must be int32 on device ", device, " with a contiguous last dimension, got ",
                    described(positions));
  a.positions = t.data_ptr<int>();
  a.pos_axis_stride = axes > 1 ? t.stride(0) : 0;
  a.pos_batch_stride = dims > 1 && B > 1 ? t.stride(dims - 2) : 0;
  TORCH_CHECK_VALUE(axes >= 1 && axes <= 3, "positions have 1 to 3 axes, got ", axes);
  a.n_axes = int(axes);
  int64_t sum = 0;
  if (sections == Py_None) {
    a.sections[0] = int(half);
    sum = axes == 1 ? half : -1;
  } else {
    const THPObjectPtr list(PySequence_Fast(sections, "sections must be a sequence of integers"));
    if (!list) throw python_error();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(list.get());
    for (Py_ssize_t i = 0; i < n && i < 3; ++i)
      sum += a.sections[i] = integer(PySequence_Fast_GET_ITEM(list.get(), i), "a section");
    if (n != axes) sum = -1;
  }
  TORCH_CHECK_VALUE(sum == half, axes, " axes of positions need as many sections that sum to ", half);
  a.interleaved = flag(interleaved);
  a.eps = number(eps, "eps");
}

// Both weights [d], or neither.
template <typename A>
bool rope_weights(A& a, PyObject* q_weight, PyObject* k_weight, int64_t d, ScalarType dtype, int64_t device) {
  TORCH_CHECK_VALUE((q_weight == Py_None) == (k_weight == Py_None), "q_weight and k_weight come together, or neither");
  if (q_weight == Py_None) return false;
  a.q_weight = expect(q_weight, "q_weight", {d}, dtype, device);
  a.k_weight = expect(k_weight, "k_weight", {d}, dtype, device);
  return true;
}

// q, k, q_weight, k_weight, positions, inv_freq, sections, interleaved, eps, q_out, k_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* o, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Tensor& q = first_tensor(o[0], "q", 4);
  const int64_t device = q.get_device(), B = q.size(0), Hq = q.size(1), N = q.size(2), d = q.size(3);
  const int64_t Hkv = tensor(o[1], "k", 4).size(1);
  const ScalarType dtype = q.scalar_type();
  const std::array<int64_t, 4> shape{B, Hq, N, d}, kshape{B, Hkv, N, d};
  fa_qk_norm_rope_args a = {};
  a.dtype = dtype_code(dtype, "q");
  a.q = rows(o[0], "q", shape, dtype, device, a.q_strides);
  a.k = rows(o[1], "k", kshape, dtype, device, a.k_strides);
  rope_arguments(a, o[4], o[5], o[6], o[7], o[8], B, N, device);
  rope_weights(a, o[2], o[3], d, dtype, device);
  Output q_out(o[9], shape, q.options()), k_out(o[10], kshape, q.options());
  a.q_out = q_out.expect("q_out", shape, dtype, device);
  a.k_out = k_out.expect("k_out", kshape, dtype, device);
  a.B = size32(B, "B"), a.Hq = size32(Hq, "Hq"), a.Hkv = size32(Hkv, "Hkv"), a.N = size32(N, "N"), a.d = size32(d, "d");
  call("fa_qk_norm_rope", api.qk_norm_rope, a, device);
  return pack({q_out.object(), k_out.object()});
  END_HANDLE_TH_ERRORS
}

// dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, sections, interleaved, eps, grad_dtype, dq, dk,
// workspace
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* o, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Tensor& q = first_tensor(o[2], "q", 4);
  const Tensor& k = tensor(o[3], "k", 4);
  const int64_t device = q.get_device(), B = q.size(0), Hq = q.size(1), N = q.size(2), d = q.size(3), Hkv = k.size(1);
  const ScalarType dtype = q.scalar_type();
  const ScalarType dout = tensor(o[0], "dq_out", 4).scalar_type();
  TORCH_CHECK_VALUE(o[11] == Py_None || THPDtype_Check(o[11]), "grad_dtype must be a torch.dtype, got ",
                    Py_TYPE(o[11])->tp_name);
  const ScalarType grad = o[11] == Py_None ? dtype : reinterpret_cast<THPDtype*>(o[11])->scalar_type;
  const std::array<int64_t, 4> shape{B, Hq, N, d}, kshape{B, Hkv, N, d};
  fa_qk_norm_rope_bwd_args a = {};
  a.dtype = dtype_code(dtype, "q");
  a.dout_dtype = dtype_code(dout, "dq_out"), a.grad_dtype = dtype_code(grad, "grad_dtype");
  a.q = rows(o[2], "q", shape, dtype, device, a.q_strides);
  a.k = rows(o[3], "k", kshape, dtype, device, a.k_strides);
  a.dq_out = expect(o[0], "dq_out", shape, dout, device);
  a.dk_out = expect(o[1], "dk_out", kshape, dout, device);
  rope_arguments(a, o[6], o[7], o[8], o[9], o[10], B, N, device);
  const bool norm = rope_weights(a, o[4], o[5], d, dtype, device);
  // new gradients are dense, their dimensions in the order of q's and k's
  PyObject* given[2] = {o[12], o[13]};
  Tensor made[2], weights[2];
  for (int i = 0; i < 2; ++i) {
    const Tensor& x = i ? k : q;
    int64_t(&strides)[3] = i ? a.dk_strides : a.dq_strides;
    void* at;
    if (given[i] == Py_None) {
      made[i] = at::empty_like(x, x.options().dtype(grad));
      for (int j = 0; j < 3; ++j) strides[j] = x.size(j) > 1 ? made[i].stride(j) : 0;
      TORCH_INTERNAL_ASSERT(made[i].stride(3) == 1 || d == 1);
      at = made[i].data_ptr();
    } else {
      at = rows(given[i], i ? "dk" : "dq", i ? kshape : shape, grad, device, strides);
    }
    (i ? a.dk : a.dq) = at;
    if (norm) {
      weights[i] = at::empty({d}, q.options().dtype(at::kFloat));
      (i ? a.dk_weight : a.dq_weight) = weights[i].data_ptr<float>();
    }
  }
  a.B = size32(B, "B"), a.Hq = size32(Hq, "Hq"), a.Hkv = size32(Hkv, "Hkv"), a.N = size32(N, "N"), a.d = size32(d, "d");
  const Workspace ws(norm ? o[14] : Py_None, norm ? api.qk_norm_rope_bwd_workspace_size(a.d) : 0, q);
  a.workspace = ws.at, a.workspace_bytes = ws.bytes;
  call("fa_qk_norm_rope_bwd", api.qk_norm_rope_bwd, a, device);
  PyObject* out[4];
  for (int i = 0; i < 2; ++i) {
    out[i] = made[i].defined() ? THPVariable_Wrap(made[i]) : given[i];
    if (!made[i].defined()) Py_INCREF(given[i]);
    out[2 + i] = norm ? THPVariable_Wrap(weights[i]) : none();
  }
  return pack({out[0], out[1], out[2], out[3]});
  END_HANDLE_TH_ERRORS
}

// ---- over the paged cache

template <typename A>
void cache_arguments(A& a, PyObject* k_cache, PyObject* v_cache, PyObject* block_table, PyObject* ctx_lens, int64_t R,
                     int64_t Hkv, int64_t d, int64_t device) {
  const Tensor& k = tensor(k_cache, "k_cache", 4);
  const int64_t num_blocks = k.size(0), bs = k.size(2), maxb = tensor(block_table, "block_table", 2).size(1);
  const std::array<int64_t, 4> shape{num_blocks, Hkv, bs, d};
  using Cache = std::remove_pointer_t<decltype(a.k_cache)>;  // (const where it is only read)
  a.k_cache = expect<Cache>(k_cache, "k_cache", shape, at::kBFloat16, device);
  a.v_cache = expect<Cache>(v_cache, "v_cache", shape, at::kBFloat16, device);
  a.block_table = expect<const int>(block_table, "block_table", {R, maxb}, at::kInt, device);
  a.ctx_lens = expect<const int>(ctx_lens, "ctx_lens", {R}, at::kInt, device);
  a.num_blocks = size32(num_blocks, "num_blocks"), a.block_size = size32(bs, "block_size");
  a.max_blocks_per_seq = size32(maxb, "max_blocks"), a.R = size32(R, "R"), a.Hkv = size32(Hkv, "Hkv");
  a.d = size32(d, "d"), a.dtype = FA_DTYPE_BF16;
}

// q, k, v, q_weight, k_weight, positions, inv_freq, k_cache, v_cache, block_table, ctx_lens, q_lens, sections,
// interleaved, eps, q_out
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* o, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Tensor& q = first_tensor(o[0], "q", 4);
  const int64_t device = q.get_device(), R = q.size(0), Hq = q.size(1), N = q.size(2), d = q.size(3);
  const int64_t Hkv = tensor(o[1], "k", 4).size(1);
  const std::array<int64_t, 4> shape{R, Hq, N, d}, kshape{R, Hkv, N, d};
  fa_qk_norm_rope_append_args a = {};
  a.q = rows(o[0], "q", shape, at::kBFloat16, device, a.q_strides);
  a.k = rows(o[1], "k", kshape, at::kBFloat16, device, a.k_strides);
  a.v = rows(o[2], "v", kshape, at::kBFloat16, device, a.v_strides);
  rope_arguments(a, o[5], o[6], o[12], o[13], o[14], R, N, device);
  rope_weights(a, o[3], o[4], d, at::kBFloat16, device);
  cache_arguments(a, o[7], o[8], o[9], o[10], R, Hkv, d, device);
  a.q_lens = expect<const int>(o[11], "q_lens", {R}, at::kInt, device);
  Output q_out(o[15], shape, q.options());
  a.q_out = q_out.expect("q_out", shape, at::kBFloat16, device);
  a.Hq = size32(Hq, "Hq"), a.Nq_max = size32(N, "Nq_max");
  call("fa_qk_norm_rope_append", api.qk_norm_rope_append, a, device);
  return q_out.object();
  END_HANDLE_TH_ERRORS
}

// What both decode calls share: q, scale and the outputs.
struct Decode {
  const Tensor& q;
  const int64_t device, R, Hq, d, Hkv;
  Tensor lse;
  Output out;
  Decode(PyObject* q_, PyObject* k_cache, PyObject* with_lse, PyObject* out_)
      : q(first_tensor(q_, "q", 3)), device(q.get_device()), R(q.size(0)), Hq(q.size(1)), d(q.size(2)),
        Hkv(tensor(k_cache, "k_cache", 4).size(1)), out(out_, q.sizes(), q.options()) {
    if (flag(with_lse)) lse = at::empty({R, Hq}, q.options().dtype(at::kFloat));
  }
  template <typename A>
  void fill(A& a, PyObject* q_, PyObject* scale) {
    a.q = expect(q_, "q", {R, Hq, d}, at::kBFloat16, device);
    a.o = out.expect("out", {R, Hq, d}, at::kBFloat16, device);
    a.lse = lse.defined() ? lse.data_ptr<float>() : nullptr;
    a.Hq = size32(Hq, "Hq");
    a.scale = scale == Py_None ? float(1.0 / std::sqrt(double(d))) : number(scale, "scale");
  }
  PyObject* results() { return pack({out.object(), lse.defined() ? THPVariable_Wrap(lse) : none()}); }
};

// q, k_cache, v_cache, prefix_table, prefix_len, block_table, ctx_lens, scale, with_lse, workspace, out
PyObject* paged_decode_shared(PyObject*, PyObject* const* o, Py_ssize_t) {
  HANDLE_TH_ERRORS
  Decode s(o[0], o[1], o[8], o[10]);
  fa_paged_decode_shared_args a = {};
  s.fill(a, o[0], o[7]);
  cache_arguments(a, o[1], o[2], o[5], o[6], s.R, s.Hkv, s.d, s.device);
  const int64_t pb = tensor(o[3], "prefix_table", 1).size(0);
  a.prefix_table = expect<const int>(o[3], "prefix_table", {pb}, at::kInt, s.device);
  a.prefix_len = expect<const int>(o[4], "prefix_len", {1}, at::kInt, s.device);
  a.max_prefix_blocks = size32(pb, "max_prefix_blocks");
  const Workspace ws(o[9], api.paged_decode_shared_workspace_size(a.R, a.Hq, a.Hkv, a.d, a.max_prefix_blocks,
                                                                  a.max_blocks_per_seq, a.block_size), s.q);
  a.workspace = ws.at, a.workspace_bytes = ws.bytes;
  call("fa_paged_decode_shared", api.paged_decode_shared, a, s.device);
  return s.results();
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, ctx_lens, weights, scale, with_lse, workspace, out
PyObject* paged_decode_scored(PyObject*, PyObject* const* o, Py_ssize_t) {
  HANDLE_TH_ERRORS
  Decode s(o[0], o[1], o[7], o[9]);
  fa_paged_decode_scored_args a = {};
  s.fill(a, o[0], o[6]);
  cache_arguments(a, o[1], o[2], o[3], o[4], s.R, s.Hkv, s.d, s.device);
  const int64_t M = int64_t(a.max_blocks_per_seq) * a.block_size;
  a.weights = expect<float>(o[5], "weights", {s.R, s.Hkv, M}, at::kFloat, s.device);
  const Workspace ws(o[8], api.paged_decode_scored_workspace_size(a.R, a.Hq, a.Hkv, a.d, a.max_blocks_per_seq,
                                                                  a.block_size), s.q);
  a.workspace = ws.at, a.workspace_bytes = ws.bytes;
  call("fa_paged_decode_scored", api.paged_decode_scored, a, s.device);
  return s.results();
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, block_table, ctx_lens, seq_lens, weights, slot_pos, keep, recent, weights_out, slot_pos_out,
// new_ctx, workspace
PyObject* paged_evict(PyObject*, PyObject* const* o, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Tensor& k = first_tensor(o[0], "k_cache", 4);
  const int64_t device = k.get_device(), Hkv = k.size(1), d = k.size(3), R = tensor(o[2], "block_table", 2).size(0);
  fa_paged_evict_args a = {};
  cache_arguments(a, o[0], o[1], o[2], o[3], R, Hkv, d, device);
  const std::array<int64_t, 3> shape{R, Hkv, int64_t(a.max_blocks_per_seq) * a.block_size};
  a.seq_lens = expect<const int>(o[4], "seq_lens", {R}, at::kInt, device);
  a.weights = expect<const float>(o[5], "weights", shape, at::kFloat, device);
  a.slot_pos = expect<const int>(o[6], "slot_pos", shape, at::kInt, device);
  a.keep = integer(o[7], "keep"), a.recent = integer(o[8], "recent");
  Output weights_out(o[9], shape, k.options().dtype(at::kFloat));
  Output slot_pos_out(o[10], shape, k.options().dtype(at::kInt));
  Output new_ctx(o[11], {R}, k.options().dtype(at::kInt));
  a.weights_out = weights_out.expect<float>("weights_out", shape, at::kFloat, device);
  a.slot_pos_out = slot_pos_out.expect<int>("slot_pos_out", shape, at::kInt, device);
  a.new_ctx = new_ctx.expect<int>("new_ctx", {R}, at::kInt, device);
  const Workspace ws(o[12], api.paged_evict_workspace_size(a.R, a.Hkv, a.max_blocks_per_seq, a.keep), k);
  a.workspace = ws.at, a.workspace_bytes = ws.bytes;
  call("fa_paged_evict", api.paged_evict, a, device);
  return pack({new_ctx.object(), weights_out.object(), slot_pos_out.object()});
  END_HANDLE_TH_ERRORS
}

// ---- the module

template <typename F>
bool take(PyObject* addresses, const char* name, F& fn) {
  PyObject* v = PyDict_GetItemString(addresses, name);  // borrowed
  if (!v) {
    PyErr_SetString(PyExc_KeyError, name);
    return false;
  }
  fn = reinterpret_cast<F>(PyLong_AsVoidPtr(v));
  return fn != nullptr;
}

// connect(addresses of the entry points by name, FAError)
PyObject* connect(PyObject*, PyObject* const* o, Py_ssize_t n) {
  if (n != 2 || !PyDict_Check(o[0])) {
    PyErr_SetString(PyExc_TypeError, "connect(addresses, error class)");
    return nullptr;
  }
#define FA_TAKE(name) \
  if (!take(o[0], "fa_" #name, api.name)) return nullptr
  FA_TAKE(qk_norm_rope);
  FA_TAKE(qk_norm_rope_append);
  FA_TAKE(qk_norm_rope_bwd);
  FA_TAKE(qk_norm_rope_bwd_workspace_size);
  FA_TAKE(paged_decode_shared);
  FA_TAKE(paged_decode_shared_workspace_size);
  FA_TAKE(paged_decode_scored);
  FA_TAKE(paged_decode_scored_workspace_size);
  FA_TAKE(paged_evict);
  FA_TAKE(paged_evict_workspace_size);
#undef FA_TAKE
  Py_INCREF(o[1]);
  Py_XDECREF(error_class);
  error_class = o[1];
  return none();
}

// F with the number of arguments that its caller, the package, passes.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), Py_ssize_t N>
PyObject* with(PyObject* self, PyObject* const* o, Py_ssize_t n) {
  if (n != N || !error_class) {
    PyErr_SetString(PyExc_TypeError, n != N ? "wrong number of arguments" : "the library is not connected");
    return nullptr;
  }
  return F(self, o, n);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&with<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&connect)), METH_FASTCALL, nullptr},
    method<qk_norm_rope, 11>("qk_norm_rope"),
    method<qk_norm_rope_bwd, 15>("qk_norm_rope_bwd"),
    method<qk_norm_rope_append, 16>("qk_norm_rope_append"),
    method<paged_decode_shared, 11>("paged_decode_shared"),
    method<paged_decode_scored, 10>("paged_decode_scored"),
    method<paged_evict, 13>("paged_evict"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
