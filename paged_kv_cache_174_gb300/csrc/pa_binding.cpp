// pa_binding.cpp -- the short way from Python into libpagedattn for the calls
// around a step (step inputs, rotary positions, sliding-window attention) and those
// for long contexts (bounds, choice and attention of blocks, weights, eviction).
//
// Those calls take a few microseconds on the GPU, and reading a dozen tensors'
// types, shapes and addresses through Python and ctypes takes longer than that
// (13 to 22 us a call on the GB300 host, 3 to 6 here).  Each function below makes
// the same checks on the tensors themselves and calls the library on the
// current stream.  Whatever is not the plain case (another type, shape, layout,
// device or number, a tensor subclass) returns None, and ops.py goes through its
// own checks, which name what is wrong or deal with it.  A status other than
// PA_OK comes back as an int.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "pagedattn.h"

namespace {

constexpr auto kInt = at::kInt;
constexpr auto kBf16 = at::kBFloat16;

// The tensor of a torch.Tensor (no subclass), or null.
const at::Tensor* tensor(PyObject* o) {
  return Py_TYPE(o) == reinterpret_cast<PyTypeObject*>(THPVariableClass)
             ? &THPVariable_Unpack(o)
             : nullptr;
}

// A contiguous tensor of this type and number of dimensions on the device.
const at::Tensor* plain(PyObject* o, at::ScalarType type, int64_t dims, int device) {
  const at::Tensor* t = tensor(o);
  return t && t->scalar_type() == type && t->dim() == dims && t->is_cuda() &&
                 t->get_device() == device && t->is_contiguous()
             ? t
             : nullptr;
}

// The device of a CUDA tensor if it is the current one, else -1.
int current_device_of(PyObject* o) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda()) return -1;
  const int device = t->get_device();
  return device == c10::cuda::current_device() ? device : -1;
}

bool number(PyObject* o, int32_t* out) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (overflow || v < INT32_MIN || v > INT32_MAX) return false;
  *out = static_cast<int32_t>(v);
  return true;
}

// Without Python's lock while it lives: allocation and launch may wait (a full
// launch queue, an allocation that has to free), and other Python threads run on
// meanwhile, as they do during torch's own operators.  Nothing in its scope touches
// a PyObject; the caller's references keep the tensors.  (No call got measurably
// longer: 3.6 to 5.8 us.)
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

int32_t* ints(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// An int32 output of a call: the caller's (of that shape), or one to be made.
struct Output {
  at::IntArrayRef shape;
  at::Tensor tensor;
  bool take(PyObject* o, int device) {
    if (o == Py_None) return true;
    const at::Tensor* t = plain(o, kInt, static_cast<int64_t>(shape.size()), device);
    if (!t || t->sizes() != shape) return false;
    tensor = *t;
    return true;
  }
};

// Makes the outputs that the caller did not give, in one allocation, each at a
// multiple of 16 bytes (build_step's four: 3.2 us on the GB300 host, 5.0 with an
// allocation each, 2.6 the rest of the call).
void make(Output* const* outputs, int n, int device) {
  const auto whole = [](const Output& o) {
    return (c10::multiply_integers(o.shape) + 3) / 4 * 4;
  };
  int64_t total = 0, at = 0;
  for (int i = 0; i < n; ++i)
    if (!outputs[i]->tensor.defined()) total += whole(*outputs[i]);
  at::Tensor all;
  for (int i = 0; i < n; ++i) {
    Output& o = *outputs[i];
    if (o.tensor.defined()) continue;
    if (!all.defined())
      all = at::empty({total}, at::TensorOptions(kInt).device(at::kCUDA, device));
    o.tensor = at::detail::make_tensor<c10::TensorImpl>(
        c10::TensorImpl::VIEW, c10::Storage(all.storage()), all.key_set(), all.dtype());
    c10::TensorImpl* t = o.tensor.unsafeGetTensorImpl();
    t->set_storage_offset(at);
    t->set_sizes_contiguous(o.shape);
    at += whole(o);
  }
}

// build_step(context_lens, new_lens, block_tables, free_blocks, free_count,
//   free_count_out, position_offsets, seq_lens, query_start_loc, slot_mapping,
//   positions, block_size, num_tokens, num_axes)
PyObject* build_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) Py_RETURN_NONE;
  const int device = current_device_of(a[0]);
  if (device < 0) Py_RETURN_NONE;
  const at::Tensor *ctx = plain(a[0], kInt, 1, device), *len = plain(a[1], kInt, 1, device),
                   *tables = plain(a[2], kInt, 2, device), *free = plain(a[3], kInt, 1, device),
                   *count = plain(a[4], kInt, 1, device);
  const at::Tensor* count_out = a[5] == Py_None ? count : plain(a[5], kInt, 1, device);
  const at::Tensor* offsets = a[6] == Py_None ? nullptr : plain(a[6], kInt, 1, device);
  int32_t block, T, A;
  if (!ctx || !len || !tables || !free || !count || !count_out ||
      (a[6] != Py_None && !offsets) || !number(a[11], &block) || !number(a[12], &T) ||
      !number(a[13], &A) || T < 0 || A < 0 || A > 1024)
    Py_RETURN_NONE;
  const int64_t S = ctx->size(0);
  if (len->size(0) != S || tables->size(0) != S || count->size(0) != 1 ||
      count_out->size(0) != 1 || (offsets && offsets->size(0) != S) || S > INT32_MAX ||
      tables->size(1) > INT32_MAX || free->size(0) > INT32_MAX)
    Py_RETURN_NONE;
  const int64_t lens_shape[] = {S}, starts_shape[] = {S + 1}, slots_shape[] = {T},
                pos_shape[] = {A, T};
  Output lens{lens_shape, {}}, starts{starts_shape, {}}, slots{slots_shape, {}}, pos{pos_shape, {}};
  Output* const outputs[4] = {&lens, &starts, &slots, &pos};
  for (int i = 0; i < 4; ++i)
    if (!outputs[i]->take(a[7 + i], device)) Py_RETURN_NONE;
  int st;
  {
    Unlocked unlocked;
    make(outputs, 4, device);
    st = pa_build_step(
        ints(*ctx), ints(*len), offsets ? ints(*offsets) : nullptr, static_cast<int32_t>(S), T, A,
        ints(*tables), static_cast<int32_t>(tables->size(1)), block, ints(*free), ints(*count),
        ints(*count_out), static_cast<int32_t>(free->size(0)), ints(lens.tensor),
        ints(starts.tensor), ints(slots.tensor), ints(pos.tensor),
        c10::cuda::getCurrentCUDAStream(device).stream());
  }
  if (st != PA_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(4);
  if (!r) return nullptr;
  for (int i = 0; i < 4; ++i) {
    PyObject* x = a[7 + i];
    if (x == Py_None)
      x = THPVariable_Wrap(outputs[i]->tensor);
    else
      Py_INCREF(x);
    PyTuple_SET_ITEM(r, i, x);
  }
  return r;
  END_HANDLE_TH_ERRORS
}

// bf16 [T, heads, d], heads contiguous within a token, tokens at a stride.
bool token_rows(PyObject* o, int device, int64_t T, int64_t d, int64_t* heads, int64_t* stride,
                const pa_bf16** at_) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != kBf16 || t->dim() != 3 || !t->is_cuda() ||
      t->get_device() != device || t->size(0) != T || t->size(2) != d)
    return false;
  const int64_t h = t->size(1);
  if ((t->stride(2) != 1 && d > 1) || (t->stride(1) != d && h > 1)) return false;
  *heads = h;
  *stride = T > 1 ? t->stride(0) : h * d;
  if (T > 1 && (*stride < h * d || *stride % 8)) return false;
  *at_ = static_cast<const pa_bf16*>(t->data_ptr());
  return true;
}

// Blocks and block size of a pair of caches for n_kv heads of d.
bool caches(PyObject* k, PyObject* v, bool fp8, int64_t n_kv, int64_t d, int device,
            int64_t* blocks, int64_t* block, void** k_at, void** v_at) {
  const int dims = fp8 ? 3 : 4;
  const auto type = fp8 ? at::kByte : kBf16;
  const at::Tensor *kc = plain(k, type, dims, device), *vc = plain(v, type, dims, device);
  if (!kc || !vc || kc->sizes() != vc->sizes()) return false;
  if (fp8) {
    if (kc->size(2) != 16 * n_kv * (d + 4)) return false;
    *block = kc->size(1) * 16;
  } else {
    if (kc->size(2) != n_kv || kc->size(3) != d) return false;
    *block = kc->size(1);
  }
  *blocks = kc->size(0);
  *k_at = kc->data_ptr();
  *v_at = vc->data_ptr();
  return *blocks <= INT32_MAX && *block <= INT32_MAX;
}

// rotary(fp8, q, k, v, positions, inv_freq, k_cache, v_cache, slot_mapping,
//   axes, interleaved, q_out)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) Py_RETURN_NONE;
  const bool fp8 = a[0] == Py_True;
  const int device = current_device_of(a[1]);
  const at::Tensor* q = tensor(a[1]);
  if (device < 0 || q->dim() != 3) Py_RETURN_NONE;
  const int64_t T = q->size(0), d = q->size(2);
  int64_t nq, nkv, nv, qs, ks, vs, blocks, block;
  const pa_bf16 *qp, *kp, *vp;
  void *kc, *vc;
  if (T > INT32_MAX || !token_rows(a[1], device, T, d, &nq, &qs, &qp) ||
      !token_rows(a[2], device, T, d, &nkv, &ks, &kp) ||
      !token_rows(a[3], device, T, d, &nv, &vs, &vp) || nkv != nv ||
      !caches(a[6], a[7], fp8, nkv, d, device, &blocks, &block, &kc, &vc))
    Py_RETURN_NONE;
  const at::Tensor* pos = tensor(a[4]);
  if (!pos || pos->scalar_type() != kInt || !pos->is_cuda() || pos->get_device() != device)
    Py_RETURN_NONE;
  int64_t A = 1, pstride = T;
  if (pos->dim() == 2) {
    A = pos->size(0);
    if (A > 1) pstride = pos->stride(0);
    if (pstride < T) Py_RETURN_NONE;
  } else if (pos->dim() != 1) {
    Py_RETURN_NONE;
  }
  if (pos->size(-1) != T || (T > 1 && pos->stride(-1) != 1) || A > INT32_MAX) Py_RETURN_NONE;
  const at::Tensor *freq = plain(a[5], at::kDouble, 1, device),
                   *slots = plain(a[8], kInt, 1, device);
  const at::Tensor* axes = a[9] == Py_None ? nullptr : plain(a[9], kInt, 1, device);
  if (!freq || !slots || slots->size(0) != T || (a[9] != Py_None && !axes) ||
      (axes && axes->size(0) != freq->size(0)) || freq->size(0) > 1024 ||
      (a[10] != Py_True && a[10] != Py_False))
    Py_RETURN_NONE;
  at::Tensor made;
  const at::Tensor* out = nullptr;
  if (a[11] != Py_None) {
    out = plain(a[11], kBf16, 3, device);
    if (!out || out->sizes() != q->sizes()) Py_RETURN_NONE;
  }
  const auto* f = static_cast<const double*>(freq->data_ptr());
  const int32_t* ax = axes ? ints(*axes) : nullptr;
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(device).stream();
  const auto t32 = static_cast<int32_t>(T), a32 = static_cast<int32_t>(A),
             rot = static_cast<int32_t>(2 * freq->size(0)), nb = static_cast<int32_t>(blocks),
             bs = static_cast<int32_t>(block), hq = static_cast<int32_t>(nq),
             hk = static_cast<int32_t>(nkv), d32 = static_cast<int32_t>(d);
  const int inter = a[10] == Py_True;
  int st;
  {
    Unlocked unlocked;
    if (!out) {
      made = at::empty({T, nq, d}, q->options());
      out = &made;
    }
    auto* o = static_cast<pa_bf16*>(out->data_ptr());
    st = fp8 ? pa_rotary_reshape_and_cache_fp8(
                   qp, qs, kp, ks, vp, vs, t32, ints(*pos), pstride, a32, f, ax, rot, inter, o,
                   static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc), nb, bs, hq, hk, d32,
                   ints(*slots), s)
             : pa_rotary_reshape_and_cache(
                   qp, qs, kp, ks, vp, vs, t32, ints(*pos), pstride, a32, f, ax, rot, inter, o,
                   static_cast<pa_bf16*>(kc), static_cast<pa_bf16*>(vc), nb, bs, hq, hk, d32,
                   ints(*slots), s);
  }
  if (st != PA_OK) return PyLong_FromLong(st);
  if (a[11] == Py_None) return THPVariable_Wrap(made);
  Py_INCREF(a[11]);
  return a[11];
  END_HANDLE_TH_ERRORS
}

// window(fp8, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc,
//   scale, window, num_sinks, min_q_len, max_q_len, max_seq_len, out, workspace)
PyObject* window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15 || !PyFloat_CheckExact(a[7])) Py_RETURN_NONE;
  const bool fp8 = a[0] == Py_True;
  const int device = current_device_of(a[1]);
  if (device < 0) Py_RETURN_NONE;
  const at::Tensor *q = plain(a[1], kBf16, 3, device), *bt = plain(a[4], kInt, 2, device),
                   *sl = plain(a[5], kInt, 1, device), *qsl = plain(a[6], kInt, 1, device),
                   *ws = plain(a[14], at::kByte, 1, device);
  const at::Tensor* k = tensor(a[2]);
  int32_t win, sinks, minq, maxq, maxl;
  if (!q || !bt || !sl || !qsl || !ws || !k || k->dim() != (fp8 ? 3 : 4) ||
      !number(a[8], &win) || !number(a[9], &sinks) || !number(a[10], &minq) ||
      !number(a[11], &maxq) || !number(a[12], &maxl))
    Py_RETURN_NONE;
  const int64_t T = q->size(0), nq = q->size(1), d = q->size(2), S = bt->size(0);
  const int64_t nkv = fp8 ? k->size(2) / (16 * (d + 4)) : k->size(2);
  int64_t blocks, block;
  void *kc, *vc;
  if (nkv <= 0 || nq % nkv || sl->size(0) != S || qsl->size(0) != S + 1 || T > INT32_MAX ||
      S > INT32_MAX || bt->size(1) > INT32_MAX ||
      !caches(a[2], a[3], fp8, nkv, d, device, &blocks, &block, &kc, &vc))
    Py_RETURN_NONE;
  at::Tensor made;
  const at::Tensor* out = nullptr;
  if (a[13] != Py_None) {
    out = plain(a[13], kBf16, 3, device);
    if (!out || out->sizes() != q->sizes()) Py_RETURN_NONE;
  }
  const auto* qp = static_cast<const pa_bf16*>(q->data_ptr());
  const auto nb = static_cast<int32_t>(blocks), bs = static_cast<int32_t>(block),
             hq = static_cast<int32_t>(nq), hk = static_cast<int32_t>(nkv),
             d32 = static_cast<int32_t>(d), mb = static_cast<int32_t>(bt->size(1)),
             s32 = static_cast<int32_t>(S), t32 = static_cast<int32_t>(T);
  const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[7]));
  const auto bytes = static_cast<size_t>(ws->numel());
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(device).stream();
  int st;
  {
    Unlocked unlocked;
    if (!out) {
      made = at::empty(q->sizes(), q->options());
      out = &made;
    }
    auto* o = static_cast<pa_bf16*>(out->data_ptr());
    st = fp8 ? pa_paged_attention_window_fp8(
                   qp, static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc), nb, bs, hq, hk, d32,
                   ints(*bt), mb, ints(*sl), ints(*qsl), s32, t32, minq, maxq, maxl, win, sinks,
                   scale, o, ws->data_ptr(), bytes, s)
             : pa_paged_attention_window(
                   qp, static_cast<pa_bf16*>(kc), static_cast<pa_bf16*>(vc), nb, bs, hq, hk, d32,
                   ints(*bt), mb, ints(*sl), ints(*qsl), s32, t32, minq, maxq, maxl, win, sinks,
                   scale, o, ws->data_ptr(), bytes, s);
  }
  if (st != PA_OK) return PyLong_FromLong(st);
  if (a[13] == Py_None) return THPVariable_Wrap(made);
  Py_INCREF(a[13]);
  return a[13];
  END_HANDLE_TH_ERRORS
}

// The q heads, kv heads and head_dim that q and a cache agree on, and the step's arrays.
struct Step {
  const at::Tensor *q, *tables, *lens, *starts;
  int64_t T, nq, d, S, blocks, block;
  void *kc, *vc;
  // a: q, k_cache, v_cache, block_tables, seq_lens, query_start_loc; n_kv from elsewhere
  bool take(PyObject* const* a, bool fp8, int64_t nkv, int device) {
    q = plain(a[0], kBf16, 3, device);
    tables = plain(a[3], kInt, 2, device);
    lens = plain(a[4], kInt, 1, device);
    starts = plain(a[5], kInt, 1, device);
    if (!q || !tables || !lens || !starts) return false;
    T = q->size(0), nq = q->size(1), d = q->size(2), S = tables->size(0);
    return nkv > 0 && nq % nkv == 0 && lens->size(0) == S && starts->size(0) == S + 1 &&
           T <= INT32_MAX && S <= INT32_MAX && nq <= INT32_MAX && tables->size(1) <= INT32_MAX &&
           caches(a[1], a[2], fp8, nkv, d, device, &blocks, &block, &kc, &vc);
  }
};

int32_t narrow(int64_t n) { return static_cast<int32_t>(n); }

// The output beside q: the caller's (of q's shape), one to be made, or no plain case.
bool output(PyObject* o, const at::Tensor& q, int device, const at::Tensor** out) {
  if (o == Py_None) return true;
  *out = plain(o, kBf16, 3, device);
  return *out && (*out)->sizes() == q.sizes();
}

PyObject* returned(PyObject* given, const at::Tensor& made) {
  if (given == Py_None) return THPVariable_Wrap(made);
  Py_INCREF(given);
  return given;
}

// summarize(fp8, k_cache, block_tables, seq_lens, query_start_loc, bounds,
//   bound_scales, num_tokens)
PyObject* summarize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  const bool fp8 = a[0] == Py_True;
  const int device = current_device_of(a[1]);
  if (device < 0) Py_RETURN_NONE;
  const at::Tensor *bt = plain(a[2], kInt, 2, device), *sl = plain(a[3], kInt, 1, device),
                   *qsl = a[4] == Py_None ? nullptr : plain(a[4], kInt, 1, device),
                   *bounds = plain(a[5], at::kChar, 4, device),
                   *scales = plain(a[6], at::kFloat, 2, device);
  int32_t T;
  if (!bt || !sl || (a[4] != Py_None && !qsl) || !bounds || !scales || !number(a[7], &T))
    Py_RETURN_NONE;
  const int64_t S = bt->size(0), nb = bounds->size(0), nkv = bounds->size(1), d = bounds->size(3);
  int64_t blocks, block;
  void *kc, *vc;
  if (sl->size(0) != S || (qsl && qsl->size(0) != S + 1) || bounds->size(2) != 2 ||
      scales->size(0) != nb || scales->size(1) != nkv || S > INT32_MAX || nkv > INT32_MAX ||
      d > INT32_MAX || bt->size(1) > INT32_MAX ||
      !caches(a[1], a[1], fp8, nkv, d, device, &blocks, &block, &kc, &vc) || blocks != nb)
    Py_RETURN_NONE;
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(device).stream();
  auto* b = static_cast<int8_t*>(bounds->data_ptr());
  auto* sc = static_cast<float*>(scales->data_ptr());
  int st;
  {
    Unlocked unlocked;
    const int32_t* starts = qsl ? ints(*qsl) : nullptr;
    st = fp8 ? pa_summarize_blocks_fp8(static_cast<uint8_t*>(kc), narrow(nb), narrow(block),
                                       narrow(nkv), narrow(d), ints(*bt), narrow(bt->size(1)),
                                       ints(*sl), starts, narrow(S), T, b, sc, s)
             : pa_summarize_blocks(static_cast<pa_bf16*>(kc), narrow(nb), narrow(block),
                                   narrow(nkv), narrow(d), ints(*bt), narrow(bt->size(1)),
                                   ints(*sl), starts, narrow(S), T, b, sc, s);
  }
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// select_blocks(q, bounds, bound_scales, block_tables, seq_lens, query_start_loc,
//   num_selected, num_sinks, num_recent, block_size, max_seq_len, out)
PyObject* select_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) Py_RETURN_NONE;
  const int device = current_device_of(a[0]);
  if (device < 0) Py_RETURN_NONE;
  const at::Tensor *q = plain(a[0], kBf16, 3, device), *bounds = plain(a[1], at::kChar, 4, device),
                   *scales = plain(a[2], at::kFloat, 2, device), *bt = plain(a[3], kInt, 2, device),
                   *sl = plain(a[4], kInt, 1, device), *qsl = plain(a[5], kInt, 1, device);
  int32_t K, sinks, recent, block, maxl;
  if (!q || !bounds || !scales || !bt || !sl || !qsl || !number(a[6], &K) ||
      !number(a[7], &sinks) || !number(a[8], &recent) || !number(a[9], &block) ||
      !number(a[10], &maxl) || K < 1)
    Py_RETURN_NONE;
  const int64_t T = q->size(0), nq = q->size(1), d = q->size(2), S = bt->size(0),
                nb = bounds->size(0), nkv = bounds->size(1);
  if (bounds->size(2) != 2 || bounds->size(3) != d || nkv <= 0 || nq % nkv ||
      scales->size(0) != nb || scales->size(1) != nkv || sl->size(0) != S ||
      qsl->size(0) != S + 1 || T > INT32_MAX || S > INT32_MAX || nb > INT32_MAX ||
      nq > INT32_MAX || d > INT32_MAX || bt->size(1) > INT32_MAX)
    Py_RETURN_NONE;
  at::Tensor made;
  const at::Tensor* out = nullptr;
  const int64_t shape[] = {T, nkv, K};
  if (a[11] != Py_None) {
    out = plain(a[11], kInt, 3, device);
    if (!out || out->sizes() != at::IntArrayRef(shape)) Py_RETURN_NONE;
  }
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(device).stream();
  int st;
  {
    Unlocked unlocked;
    if (!out) {
      made = at::empty(shape, sl->options());
      out = &made;
    }
    st = pa_select_blocks(static_cast<const pa_bf16*>(q->data_ptr()),
                          static_cast<const int8_t*>(bounds->data_ptr()),
                          static_cast<const float*>(scales->data_ptr()), narrow(nb), block,
                          narrow(nq), narrow(nkv), narrow(d), ints(*bt), narrow(bt->size(1)),
                          ints(*sl), ints(*qsl), narrow(S), narrow(T), maxl, K, sinks, recent,
                          ints(*out), s);
  }
  if (st != PA_OK) return PyLong_FromLong(st);
  return returned(a[11], made);
  END_HANDLE_TH_ERRORS
}

// blocks(fp8, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale,
//   selected, out)
PyObject* blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10 || !PyFloat_CheckExact(a[7])) Py_RETURN_NONE;
  const bool fp8 = a[0] == Py_True;
  const int device = current_device_of(a[1]);
  if (device < 0) Py_RETURN_NONE;
  const at::Tensor* sel = plain(a[8], kInt, 3, device);
  Step x;
  if (!sel || !x.take(a + 1, fp8, sel->size(1), device) || sel->size(0) != x.T ||
      sel->size(2) > INT32_MAX)
    Py_RETURN_NONE;
  at::Tensor made;
  const at::Tensor* out = nullptr;
  if (!output(a[9], *x.q, device, &out)) Py_RETURN_NONE;
  const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[7]));
  const int32_t nkv = narrow(sel->size(1)), K = narrow(sel->size(2));
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(device).stream();
  int st;
  {
    Unlocked unlocked;
    if (!out) {
      made = at::empty(x.q->sizes(), x.q->options());
      out = &made;
    }
    const auto* q = static_cast<const pa_bf16*>(x.q->data_ptr());
    auto* o = static_cast<pa_bf16*>(out->data_ptr());
    st = fp8 ? pa_paged_attention_blocks_fp8(
                   q, static_cast<uint8_t*>(x.kc), static_cast<uint8_t*>(x.vc), narrow(x.blocks),
                   narrow(x.block), narrow(x.nq), nkv, narrow(x.d), ints(*x.tables),
                   narrow(x.tables->size(1)), ints(*x.lens), ints(*x.starts), narrow(x.S),
                   narrow(x.T), scale, ints(*sel), K, o, s)
             : pa_paged_attention_blocks(
                   q, static_cast<pa_bf16*>(x.kc), static_cast<pa_bf16*>(x.vc), narrow(x.blocks),
                   narrow(x.block), narrow(x.nq), nkv, narrow(x.d), ints(*x.tables),
                   narrow(x.tables->size(1)), ints(*x.lens), ints(*x.starts), narrow(x.S),
                   narrow(x.T), scale, ints(*sel), K, o, s);
  }
  if (st != PA_OK) return PyLong_FromLong(st);
  return returned(a[9], made);
  END_HANDLE_TH_ERRORS
}

// weights(fp8, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale,
//   weights, min_q_len, max_q_len, max_seq_len, out, workspace)
PyObject* weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14 || !PyFloat_CheckExact(a[7])) Py_RETURN_NONE;
  const bool fp8 = a[0] == Py_True;
  const int device = current_device_of(a[1]);
  if (device < 0) Py_RETURN_NONE;
  const at::Tensor* w = plain(a[8], at::kFloat, 3, device);
  const at::Tensor* ws = a[13] == Py_None ? nullptr : plain(a[13], at::kByte, 1, device);
  int32_t minq, maxq, maxl;
  Step x;
  if (!w || (a[13] != Py_None && !ws) || !number(a[9], &minq) || !number(a[10], &maxq) ||
      !number(a[11], &maxl) || (!ws && maxq > 1) || !x.take(a + 1, fp8, w->size(1), device) ||
      w->size(0) != x.S || w->size(2) > INT32_MAX)
    Py_RETURN_NONE;
  at::Tensor made;
  const at::Tensor* out = nullptr;
  if (!output(a[12], *x.q, device, &out)) Py_RETURN_NONE;
  const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[7]));
  const int32_t nkv = narrow(w->size(1)), length = narrow(w->size(2));
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(device).stream();
  int st;
  {
    Unlocked unlocked;
    if (!out) {
      made = at::empty(x.q->sizes(), x.q->options());
      out = &made;
    }
    const auto* q = static_cast<const pa_bf16*>(x.q->data_ptr());
    auto* o = static_cast<pa_bf16*>(out->data_ptr());
    auto* f = static_cast<float*>(w->data_ptr());
    void* space = ws ? ws->data_ptr() : nullptr;
    const size_t bytes = ws ? static_cast<size_t>(ws->numel()) : 0;
    st = fp8 ? pa_paged_attention_weights_fp8(
                   q, static_cast<uint8_t*>(x.kc), static_cast<uint8_t*>(x.vc), narrow(x.blocks),
                   narrow(x.block), narrow(x.nq), nkv, narrow(x.d), ints(*x.tables),
                   narrow(x.tables->size(1)), ints(*x.lens), ints(*x.starts), narrow(x.S),
                   narrow(x.T), minq, maxq, maxl, scale, f, length, o, space, bytes, s)
             : pa_paged_attention_weights(
                   q, static_cast<pa_bf16*>(x.kc), static_cast<pa_bf16*>(x.vc), narrow(x.blocks),
                   narrow(x.block), narrow(x.nq), nkv, narrow(x.d), ints(*x.tables),
                   narrow(x.tables->size(1)), ints(*x.lens), ints(*x.starts), narrow(x.S),
                   narrow(x.T), minq, maxq, maxl, scale, f, length, o, space, bytes, s);
  }
  if (st != PA_OK) return PyLong_FromLong(st);
  return returned(a[12], made);
  END_HANDLE_TH_ERRORS
}

// evict(fp8, k_cache, v_cache, weights, block_tables, seq_lens, budgets, free_blocks,
//   free_count, num_sinks, num_recent, max_seq_len, seq_lens_out, free_count_out,
//   position_offsets)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15) Py_RETURN_NONE;
  const bool fp8 = a[0] == Py_True;
  const int device = current_device_of(a[1]);
  const at::Tensor* k = tensor(a[1]);
  if (device < 0 || k->dim() != (fp8 ? 3 : 4)) Py_RETURN_NONE;
  const at::Tensor *w = plain(a[3], at::kFloat, 3, device), *bt = plain(a[4], kInt, 2, device),
                   *sl = plain(a[5], kInt, 1, device), *budgets = plain(a[6], kInt, 1, device),
                   *free = plain(a[7], kInt, 1, device), *count = plain(a[8], kInt, 1, device);
  const at::Tensor* lens_out = a[12] == Py_None ? sl : plain(a[12], kInt, 1, device);
  const at::Tensor* count_out = a[13] == Py_None ? count : plain(a[13], kInt, 1, device);
  const at::Tensor* offsets = a[14] == Py_None ? nullptr : plain(a[14], kInt, 1, device);
  int32_t sinks, recent, maxl;
  if (!w || !bt || !sl || !budgets || !free || !count || !lens_out || !count_out ||
      (a[14] != Py_None && !offsets) || !number(a[9], &sinks) || !number(a[10], &recent) ||
      !number(a[11], &maxl))
    Py_RETURN_NONE;
  const int64_t S = bt->size(0), nkv = w->size(1), length = w->size(2);
  const int64_t d = fp8 ? (nkv > 0 ? k->size(2) / (16 * nkv) - 4 : 0) : k->size(3);
  int64_t blocks, block;
  void *kc, *vc;
  if (w->size(0) != S || sl->size(0) != S || budgets->size(0) != S || count->size(0) != 1 ||
      lens_out->size(0) != S || count_out->size(0) != 1 || (offsets && offsets->size(0) != S) ||
      S > INT32_MAX || length > INT32_MAX || bt->size(1) > INT32_MAX || nkv > INT32_MAX ||
      d > INT32_MAX || !caches(a[1], a[2], fp8, nkv, d, device, &blocks, &block, &kc, &vc) ||
      free->size(0) != blocks)
    Py_RETURN_NONE;
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(device).stream();
  int st;
  {
    Unlocked unlocked;
    auto* f = static_cast<float*>(w->data_ptr());
    int32_t* off = offsets ? ints(*offsets) : nullptr;
    st = fp8 ? pa_evict_tokens_fp8(
                   static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc), f, narrow(length),
                   narrow(blocks), narrow(block), narrow(nkv), narrow(d), ints(*bt),
                   narrow(bt->size(1)), ints(*sl), ints(*budgets), narrow(S), maxl, sinks, recent,
                   ints(*free), ints(*count), ints(*lens_out), ints(*count_out), off, s)
             : pa_evict_tokens(
                   static_cast<pa_bf16*>(kc), static_cast<pa_bf16*>(vc), f, narrow(length),
                   narrow(blocks), narrow(block), narrow(nkv), narrow(d), ints(*bt),
                   narrow(bt->size(1)), ints(*sl), ints(*budgets), narrow(S), maxl, sinks, recent,
                   ints(*free), ints(*count), ints(*lens_out), ints(*count_out), off, s);
  }
  if (st != PA_OK) return PyLong_FromLong(st);
  PyObject* r = a[12] == Py_None ? a[5] : a[12];
  Py_INCREF(r);
  return r;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef kMethods[] = {
    {"build_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(build_step)),
     METH_FASTCALL, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL,
     nullptr},
    {"window", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(window)), METH_FASTCALL,
     nullptr},
    method<summarize>("summarize"),
    method<select_blocks>("select_blocks"),
    method<blocks>("blocks"),
    method<weights>("weights"),
    method<evict>("evict"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "pa_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_binding(void) { return PyModule_Create(&kModule); }
