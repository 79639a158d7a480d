// Calls of the grouped-head, 8-bit cache and rotary entry points from PyTorch without
// the interpreter in between: what the Python helpers of the same names do
// (check the tensors, allocate the outputs and the workspace, call the C ABI on
// the current stream), for the plain case in which all arguments are in order.
// A decoding step's calls take the host longer than the GPU: through Python
// and ctypes 24 us for a token's attention whose kernels run 7 us.
//
// Every function returns its tensors, or None if anything is not as the C ABI
// wants it (or an allocation or the call failed), or while PyTorch's operations
// are recorded, which none of these is: the caller then takes the Python path,
// which names what is wrong.  No C++ exception leaves a function.
// Allocations and launches, which may have to wait (for memory, for room in the
// launch queue), run without the interpreter lock.
#include <Python.h>

#include <cmath>
#include <limits>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/jit/frontend/tracer.h>

#include "fa.h"

namespace {

using at::Tensor;

// Lets other Python threads run while in scope (also left by an exception).
class WithoutLock {
 public:
  WithoutLock() : state_(PyEval_SaveThread()) {}
  ~WithoutLock() { PyEval_RestoreThread(state_); }
  WithoutLock(const WithoutLock&) = delete;
  WithoutLock& operator=(const WithoutLock&) = delete;

 private:
  PyThreadState* state_;
};

// torch.jit.trace or make_fx is at work on this thread.
bool recording() {
  using c10::impl::TorchDispatchModeKey;
  using c10::impl::TorchDispatchModeTLS;
  return torch::jit::tracer::isTracing() ||
         (TorchDispatchModeTLS::any_modes_set() && TorchDispatchModeTLS::get_mode(TorchDispatchModeKey::PROXY).has_value());
}

// A tensor argument; nullptr if it is something else.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool dense(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.scalar_type() == type &&
         t.sizes() == shape && t.is_contiguous();
}

// Row stride of a bf16 [rows, heads, d] tensor whose rows may lie further apart than heads·d; -1 if it is none.
int64_t rows_stride(const Tensor& t, int64_t rows, int64_t heads, int64_t d, int dev) {
  if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kBFloat16 ||
      t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != d)
    return -1;
  const int64_t n = heads * d;
  if (t.is_contiguous()) return n;
  const int64_t s0 = t.stride(0);
  if ((d > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != d)) return -1;
  if (rows <= 1) return n;
  return s0 >= n && s0 % 8 == 0 ? s0 : -1;
}

bool to_int(PyObject* o, int* v) {
  const long long x = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  if (x == -1 && PyErr_Occurred()) PyErr_Clear();
  *v = static_cast<int>(x);
  return x > 0 && x <= std::numeric_limits<int>::max();
}

// scale: None is 1 / sqrt(d).
bool to_scale(PyObject* o, int64_t d, float* v) {
  if (o == Py_None) {
    *v = static_cast<float>(std::pow(static_cast<double>(d), -0.5));
    return true;
  }
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *v = static_cast<float>(x);
  return true;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

bool fits(int64_t n) { return n >= 0 && n <= std::numeric_limits<int>::max(); }

PyObject* pair(Tensor a, Tensor b) {
  PyObject* x = THPVariable_Wrap(std::move(a));
  PyObject* y = THPVariable_Wrap(std::move(b));
  if (!x || !y) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    return nullptr;
  }
  PyObject* r = PyTuple_Pack(2, x, y);
  Py_DECREF(x);
  Py_DECREF(y);
  return r;
}

// ----------------------------------------------------------------------------
// Grouped heads over packed batches
// ----------------------------------------------------------------------------
struct Grouped {
  int dev, T, H, Hk, d, nseq, max_seqlen;
  int64_t ldq, ldk, ldv;
  float scale;
  bool causal;
};

bool check_grouped(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, Grouped* g) {
  if (!q.is_cuda() || q.dim() != 3 || k.dim() != 3 || cu.dim() != 1) return false;
  g->dev = q.get_device();
  const int64_t T = q.size(0), H = q.size(1), d = q.size(2), Hk = k.size(1), n = cu.size(0) - 1;
  if (!fits(T) || !fits(H) || !fits(d) || !fits(Hk) || !fits(n)) return false;
  g->T = static_cast<int>(T), g->H = static_cast<int>(H), g->d = static_cast<int>(d);
  g->Hk = static_cast<int>(Hk), g->nseq = static_cast<int>(n);
  g->ldq = rows_stride(q, T, H, d, g->dev);
  g->ldk = rows_stride(k, T, Hk, d, g->dev);
  g->ldv = rows_stride(v, T, Hk, d, g->dev);
  return g->ldq > 0 && g->ldk > 0 && g->ldv > 0 && dense(cu, at::kInt, cu.sizes(), g->dev);
}

fa_status forward_grouped(const Grouped& g, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu,
                          Tensor* o, Tensor* lse) {
  *o = at::empty({g.T, g.H, g.d}, q.options().requires_grad(false));
  *lse = at::empty({g.H, g.T}, q.options().requires_grad(false).dtype(at::kFloat));
  return fa_fwd_grouped(q.data_ptr(), k.data_ptr(), v.data_ptr(), o->data_ptr(), static_cast<float*>(lse->data_ptr()),
                        static_cast<const int*>(cu.data_ptr()), g.nseq, g.max_seqlen, g.T, g.H, g.Hk, g.d, g.ldq,
                        g.ldk, g.ldv, g.scale, g.causal, 1, stream_of(g.dev));
}

fa_status backward_grouped(const Grouped& g, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o,
                           const Tensor& dout, const Tensor& lse, const Tensor& cu, Tensor* dq, Tensor* dk,
                           Tensor* dv) {
  const auto opt = q.options().requires_grad(false);
  *dq = at::empty({g.T, g.H, g.d}, opt);
  *dk = at::empty({g.T, g.Hk, g.d}, opt);
  *dv = at::empty({g.T, g.Hk, g.d}, opt);
  const size_t n = fa_bwd_grouped_workspace_bytes(g.nseq, g.max_seqlen, g.T, g.H, g.Hk, g.d, g.causal);
  Tensor ws = at::empty({static_cast<int64_t>(n)}, opt.dtype(at::kByte));
  return fa_bwd_grouped(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                        static_cast<const float*>(lse.data_ptr()), dq->data_ptr(), dk->data_ptr(), dv->data_ptr(),
                        ws.data_ptr(), n, static_cast<const int*>(cu.data_ptr()), g.nseq, g.max_seqlen, g.T, g.H, g.Hk,
                        g.d, g.ldq, g.ldk, g.ldv, g.scale, g.causal, 1, stream_of(g.dev));
}

// (q, k, v, cu_seqlens, max_seqlen, causal, scale) of `args`.
bool grouped_args(PyObject* const* args, Py_ssize_t n, const Tensor* (&t)[4], Grouped* g) {
  if (n != 7 || recording()) return false;
  for (int i = 0; i < 4; ++i)
    if (!(t[i] = tensor(args[i]))) return false;
  if (!check_grouped(*t[0], *t[1], *t[2], *t[3], g)) return false;
  const int causal = PyObject_IsTrue(args[5]);
  if (causal < 0) {
    PyErr_Clear();
    return false;
  }
  g->causal = causal != 0;
  return to_int(args[4], &g->max_seqlen) && to_scale(args[6], g->d, &g->scale);
}

PyObject* py_forward_grouped(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    const Tensor* t[4];
    Grouped g;
    Tensor o, lse;
    if (grouped_args(args, n, t, &g)) {
      fa_status st;
      {
        WithoutLock unlocked;
        st = forward_grouped(g, *t[0], *t[1], *t[2], *t[3], &o, &lse);
      }
      if (st == FA_OK) return pair(std::move(o), std::move(lse));
    }
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

// The autograd function; differentiable once, like its Python counterpart.
struct FlashAttentionGrouped : torch::autograd::Function<FlashAttentionGrouped> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& v,
                        const Tensor& cu, int64_t max_seqlen, bool causal, double scale) {
    Grouped g;
    TORCH_CHECK(check_grouped(q, k, v, cu, &g), "flash_attention_grouped: arguments out of order");
    g.max_seqlen = static_cast<int>(max_seqlen);
    g.causal = causal;
    g.scale = static_cast<float>(scale);
    Tensor o, lse;
    const fa_status st = forward_grouped(g, q, k, v, cu, &o, &lse);
    TORCH_CHECK(st == FA_OK, "fa_fwd_grouped failed: ", fa_status_string(st), " ", fa_last_error_detail());
    ctx->save_for_backward({q, k, v, o, lse, cu});
    ctx->saved_data["max_seqlen"] = max_seqlen;
    ctx->saved_data["causal"] = causal;
    ctx->saved_data["scale"] = scale;
    return o;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto s = ctx->get_saved_variables();
    Grouped g;
    // (what was saved comes back through hooks that the user may have set)
    TORCH_CHECK(check_grouped(s[0], s[1], s[2], s[5], &g) && dense(s[3], at::kBFloat16, {g.T, g.H, g.d}, g.dev) &&
                    dense(s[4], at::kFloat, {g.H, g.T}, g.dev),
                "flash_attention_grouped: saved tensors out of order");
    g.max_seqlen = static_cast<int>(ctx->saved_data["max_seqlen"].toInt());
    g.causal = ctx->saved_data["causal"].toBool();
    g.scale = static_cast<float>(ctx->saved_data["scale"].toDouble());
    const Tensor dout = grads[0].contiguous();
    TORCH_CHECK(dense(dout, at::kBFloat16, {g.T, g.H, g.d}, g.dev), "flash_attention_grouped: gradient of o must be a "
                "bfloat16 tensor of o's shape on its device");
    const bool again = at::GradMode::is_enabled();
    torch::autograd::variable_list out(7);
    {
      at::AutoGradMode no_grad(false);
      const fa_status st = backward_grouped(g, s[0], s[1], s[2], s[3], dout, s[4], s[5], &out[0], &out[1], &out[2]);
      TORCH_CHECK(st == FA_OK, "fa_bwd_grouped failed: ", fa_status_string(st), " ", fa_last_error_detail());
    }
    if (again) {  // the gradients are wanted for differentiation: that, not this, is the error
      torch::autograd::variable_list three(out.begin(), out.begin() + 3);
      for (auto& x : three) x = x.requires_grad_(true);
      auto err = std::make_shared<torch::autograd::DelayedError>("flash_attention_grouped is differentiable once", 3);
      three = (*err)(std::move(three));
      for (int i = 0; i < 3; ++i) out[i] = three[i];
    }
    return out;
  }
};

PyObject* py_flash_attention_grouped(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    const Tensor* t[4];
    Grouped g;
    if (grouped_args(args, n, t, &g)) {
      Tensor o;
      {
        WithoutLock unlocked;
        o = FlashAttentionGrouped::apply(*t[0], *t[1], *t[2], *t[3], static_cast<int64_t>(g.max_seqlen), g.causal,
                                         static_cast<double>(g.scale));
      }
      return THPVariable_Wrap(std::move(o));
    }
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

PyObject* py_backward_grouped(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    const Tensor* t[4];
    Grouped g;
    if (n == 10 && grouped_args(args, 7, t, &g)) {
      const Tensor *o = tensor(args[7]), *dout = tensor(args[8]), *lse = tensor(args[9]);
      if (o && dout && lse && dense(*o, at::kBFloat16, {g.T, g.H, g.d}, g.dev) &&
          dense(*dout, at::kBFloat16, {g.T, g.H, g.d}, g.dev) && dense(*lse, at::kFloat, {g.H, g.T}, g.dev)) {
        Tensor d[3];
        fa_status st;
        {
          WithoutLock unlocked;
          st = backward_grouped(g, *t[0], *t[1], *t[2], *o, *dout, *lse, *t[3], &d[0], &d[1], &d[2]);
        }
        if (st == FA_OK) {
          PyObject* r = PyTuple_New(3);
          for (int i = 0; r && i < 3; ++i) {
            PyObject* x = THPVariable_Wrap(std::move(d[i]));
            if (!x) {
              Py_DECREF(r);
              return nullptr;
            }
            PyTuple_SET_ITEM(r, i, x);
          }
          return r;
        }
      }
    }
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

// ----------------------------------------------------------------------------
// 8-bit paged cache
// ----------------------------------------------------------------------------
struct Cache {
  const Tensor* t[4];  // k, v, k_scale, v_scale
  int num_blocks, Hk, block, d;
};

bool cache_args(PyObject* cache, int dev, Cache* c) {
  if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 4) return false;
  for (int i = 0; i < 4; ++i)
    if (!(c->t[i] = tensor(PyTuple_GET_ITEM(cache, i)))) return false;
  const Tensor& k = *c->t[0];
  if (k.dim() != 4) return false;
  const auto s = k.sizes();
  for (int i = 0; i < 4; ++i)
    if (!fits(s[i])) return false;
  c->num_blocks = static_cast<int>(s[0]), c->Hk = static_cast<int>(s[1]);
  c->block = static_cast<int>(s[2]), c->d = static_cast<int>(s[3]);
  const auto heads = s.slice(0, 2);
  return dense(k, at::kFloat8_e4m3fn, s, dev) && dense(*c->t[1], at::kFloat8_e4m3fn, s, dev) &&
         dense(*c->t[2], at::kFloat, heads, dev) && dense(*c->t[3], at::kFloat, heads, dev);
}

// (k, v, cache, block_table, cu_seqlens, start, max_new) -> True
PyObject* py_cache8_store(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != 7 || recording()) Py_RETURN_NONE;
    const Tensor *k = tensor(args[0]), *v = tensor(args[1]), *table = tensor(args[3]), *cu = tensor(args[4]),
                 *start = tensor(args[5]);
    Cache c;
    int max_new = 0;
    if (!k || !v || !table || !cu || !start || !k->is_cuda() || k->dim() != 3) Py_RETURN_NONE;
    const int dev = k->get_device();
    if (!cache_args(args[2], dev, &c) || !to_int(args[6], &max_new)) Py_RETURN_NONE;
    const int64_t T = k->size(0), B = start->numel();
    const int64_t ldk = rows_stride(*k, T, c.Hk, c.d, dev), ldv = rows_stride(*v, T, c.Hk, c.d, dev);
    if (ldk < 0 || ldv < 0 || table->dim() != 2 || !fits(T) || !fits(B) || !fits(table->size(1)) ||
        !dense(*table, at::kInt, {B, table->size(1)}, dev) || !dense(*cu, at::kInt, {B + 1}, dev) ||
        !dense(*start, at::kInt, {B}, dev))
      Py_RETURN_NONE;
    fa_status st;
    {
      WithoutLock unlocked;
      st = fa_cache8_store(
          k->data_ptr(), v->data_ptr(), c.t[0]->data_ptr(), c.t[1]->data_ptr(), static_cast<float*>(c.t[2]->data_ptr()),
          static_cast<float*>(c.t[3]->data_ptr()), static_cast<const int*>(table->data_ptr()),
          static_cast<const int*>(cu->data_ptr()), static_cast<const int*>(start->data_ptr()), static_cast<int>(B), max_new,
          static_cast<int>(T), c.num_blocks, static_cast<int>(table->size(1)), c.Hk, c.block, c.d, ldk, ldv,
          stream_of(dev));
    }
    if (st == FA_OK) Py_RETURN_TRUE;
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

// (q, cache, block_table, seqlens, max_seqlen, causal, scale) -> (o, lse)
PyObject* py_decode_cache8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != 7 || recording()) Py_RETURN_NONE;
    const Tensor *q = tensor(args[0]), *table = tensor(args[2]), *lens = tensor(args[3]);
    Cache c;
    int max_seqlen = 0;
    float scale = 0.f;
    if (!q || !table || !lens || !q->is_cuda() || q->dim() != 4) Py_RETURN_NONE;
    const int dev = q->get_device();
    const int64_t B = q->size(0), Nq = q->size(1), H = q->size(2), d = q->size(3);
    const int causal = PyObject_IsTrue(args[5]);
    if (causal < 0) PyErr_Clear();
    if (causal < 0 || !cache_args(args[1], dev, &c) || !to_int(args[4], &max_seqlen) || !to_scale(args[6], d, &scale))
      Py_RETURN_NONE;
    if (!fits(B) || !fits(Nq) || !fits(H) || d != c.d || !dense(*q, at::kBFloat16, q->sizes(), dev) || table->dim() != 2 ||
        !fits(table->size(1)) || !dense(*table, at::kInt, {B, table->size(1)}, dev) || !dense(*lens, at::kInt, {B}, dev))
      Py_RETURN_NONE;
    const int b = static_cast<int>(B), nq = static_cast<int>(Nq), h = static_cast<int>(H);
    const size_t bytes = fa_decode_cache8_workspace_bytes(b, nq, h, c.Hk, max_seqlen, c.d);
    if (bytes == 0) Py_RETURN_NONE;
    Tensor o, lse;
    fa_status st;
    {
      WithoutLock unlocked;
      const auto opt = q->options().requires_grad(false);
      o = at::empty(q->sizes(), opt);
      lse = at::empty({B, H, Nq}, opt.dtype(at::kFloat));
      Tensor ws = at::empty({static_cast<int64_t>(bytes)}, opt.dtype(at::kByte));
      st = fa_fwd_decode_cache8(
          q->data_ptr(), c.t[0]->data_ptr(), c.t[1]->data_ptr(), static_cast<const float*>(c.t[2]->data_ptr()),
          static_cast<const float*>(c.t[3]->data_ptr()), static_cast<const int*>(table->data_ptr()),
          static_cast<const int*>(lens->data_ptr()), o.data_ptr(), static_cast<float*>(lse.data_ptr()), ws.data_ptr(), bytes,
          b, nq, h, c.Hk, c.num_blocks, static_cast<int>(table->size(1)), c.block, max_seqlen, c.d, scale, causal,
          stream_of(dev));
    }
    if (st == FA_OK) return pair(std::move(o), std::move(lse));
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

// ----------------------------------------------------------------------------
// Rotary positions
// ----------------------------------------------------------------------------
struct Turn {
  const Tensor *turns, *axis;
  int pairs, axes;
  bool interleaved;
};

bool turn_tensors(const Tensor& turns, const Tensor& axis, int axes, int64_t d, int dev, Turn* r) {
  if (turns.dim() != 1) return false;
  const int64_t pairs = turns.size(0);
  r->turns = &turns, r->axis = &axis, r->axes = axes, r->pairs = static_cast<int>(pairs);
  return pairs > 0 && pairs % 8 == 0 && 2 * pairs <= d && axes >= 1 && axes <= pairs &&
         dense(turns, at::kLong, {pairs}, dev) && dense(axis, at::kInt, {pairs}, dev);
}

bool turn_args(PyObject* rotary, int64_t d, int dev, Turn* r) {
  if (!PyTuple_Check(rotary) || PyTuple_GET_SIZE(rotary) != 4) return false;
  const Tensor *turns = tensor(PyTuple_GET_ITEM(rotary, 0)), *axis = tensor(PyTuple_GET_ITEM(rotary, 1));
  int axes = 0;
  const int il = PyObject_IsTrue(PyTuple_GET_ITEM(rotary, 3));
  if (il < 0) PyErr_Clear();
  if (il < 0 || !turns || !axis || !to_int(PyTuple_GET_ITEM(rotary, 2), &axes)) return false;
  r->interleaved = il != 0;
  return turn_tensors(*turns, *axis, axes, d, dev, r);
}

// positions: int32 [axes, T], or [T] with one axis.
bool positions_ok(const Tensor& t, int axes, int64_t T, int dev) {
  return (axes == 1 && t.dim() == 1) ? dense(t, at::kInt, {T}, dev) : dense(t, at::kInt, {axes, T}, dev);
}

struct Rows {
  int dev, T, H, Hk, d;
  int64_t ldq, ldk;
};

bool check_rows(const Tensor& q, const Tensor& k, Rows* r) {
  if (!q.is_cuda() || q.dim() != 3 || k.dim() != 3) return false;
  r->dev = q.get_device();
  const int64_t T = q.size(0), H = q.size(1), d = q.size(2), Hk = k.size(1);
  if (!fits(T) || !fits(H) || !fits(d) || !fits(Hk)) return false;
  r->T = static_cast<int>(T), r->H = static_cast<int>(H), r->d = static_cast<int>(d), r->Hk = static_cast<int>(Hk);
  r->ldq = rows_stride(q, T, H, d, r->dev);
  r->ldk = rows_stride(k, T, Hk, d, r->dev);
  return r->ldq > 0 && r->ldk > 0;
}

const uint64_t* turns_ptr(const Turn& t) { return static_cast<const uint64_t*>(t.turns->data_ptr()); }
const int* ints(const Tensor& t) { return static_cast<const int*>(t.data_ptr()); }

fa_status turn(const Rows& r, const Turn& t, const Tensor& q, const Tensor& k, const Tensor& positions, bool inverse,
               Tensor* q_out, Tensor* k_out) {
  const auto opt = q.options().requires_grad(false);
  *q_out = at::empty({r.T, r.H, r.d}, opt);
  *k_out = at::empty({r.T, r.Hk, r.d}, opt);
  return fa_rotary(q.data_ptr(), k.data_ptr(), q_out->data_ptr(), k_out->data_ptr(), ints(positions), turns_ptr(t),
                   ints(*t.axis), r.T, r.H, r.Hk, r.d, t.pairs, t.axes, t.interleaved, inverse, r.ldq, r.ldk,
                   stream_of(r.dev));
}

// (q, k, positions, rotary) of `args`.
bool rotary_args(PyObject* const* args, const Tensor* (&t)[3], Rows* r, Turn* turn) {
  if (recording()) return false;
  for (int i = 0; i < 3; ++i)
    if (!(t[i] = tensor(args[i]))) return false;
  return check_rows(*t[0], *t[1], r) && turn_args(args[3], r->d, r->dev, turn) &&
         positions_ok(*t[2], turn->axes, r->T, r->dev);
}

// (q, k, positions, rotary, inverse) -> (q', k')
PyObject* py_rotary(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    const Tensor* t[3];
    Rows r;
    Turn plan;
    if (n == 5 && rotary_args(args, t, &r, &plan)) {
      const bool inverse = args[4] == Py_True;
      Tensor q, k;
      fa_status st;
      {
        WithoutLock unlocked;
        st = turn(r, plan, *t[0], *t[1], *t[2], inverse, &q, &k);
      }
      if (st == FA_OK) return pair(std::move(q), std::move(k));
    }
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

// The autograd function; differentiable once, like its Python counterpart.
struct RotaryEmbedding : torch::autograd::Function<RotaryEmbedding> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& q, const Tensor& k,
                                                const Tensor& positions, const Tensor& turns, const Tensor& axis,
                                                int64_t axes, bool interleaved) {
    Rows r;
    Turn t;
    t.interleaved = interleaved;
    TORCH_CHECK(check_rows(q, k, &r) && turn_tensors(turns, axis, static_cast<int>(axes), r.d, r.dev, &t) &&
                    positions_ok(positions, t.axes, r.T, r.dev),
                "rotary_embedding: arguments out of order");
    torch::autograd::variable_list out(2);
    const fa_status st = turn(r, t, q, k, positions, false, &out[0], &out[1]);
    TORCH_CHECK(st == FA_OK, "fa_rotary failed: ", fa_status_string(st), " ", fa_last_error_detail());
    ctx->save_for_backward({positions, turns, axis});
    ctx->saved_data["axes"] = axes;
    ctx->saved_data["interleaved"] = interleaved;
    return out;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto s = ctx->get_saved_variables();
    const Tensor dq = grads[0].contiguous(), dk = grads[1].contiguous();
    Rows r;
    Turn t;
    t.interleaved = ctx->saved_data["interleaved"].toBool();
    // (what was saved comes back through hooks that the user may have set)
    TORCH_CHECK(check_rows(dq, dk, &r), "rotary_embedding: gradients must be bfloat16 tensors of q's and k's shapes on their device");
    TORCH_CHECK(turn_tensors(s[1], s[2], static_cast<int>(ctx->saved_data["axes"].toInt()), r.d, r.dev, &t) &&
                    positions_ok(s[0], t.axes, r.T, r.dev),
                "rotary_embedding: saved tensors out of order");
    const bool again = at::GradMode::is_enabled();
    torch::autograd::variable_list out(7);
    {
      at::AutoGradMode no_grad(false);
      const fa_status st = turn(r, t, dq, dk, s[0], true, &out[0], &out[1]);
      TORCH_CHECK(st == FA_OK, "fa_rotary failed: ", fa_status_string(st), " ", fa_last_error_detail());
    }
    if (again) {  // the gradients are wanted for differentiation: that, not this, is the error
      torch::autograd::variable_list two(out.begin(), out.begin() + 2);
      for (auto& x : two) x = x.requires_grad_(true);
      auto err = std::make_shared<torch::autograd::DelayedError>("rotary_embedding is differentiable once", 2);
      two = (*err)(std::move(two));
      for (int i = 0; i < 2; ++i) out[i] = two[i];
    }
    return out;
  }
};

PyObject* py_rotary_embedding(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    const Tensor* t[3];
    Rows r;
    Turn plan;
    if (n == 4 && rotary_args(args, t, &r, &plan)) {
      torch::autograd::variable_list out;
      {
        WithoutLock unlocked;
        out = RotaryEmbedding::apply(*t[0], *t[1], *t[2], *plan.turns, *plan.axis, static_cast<int64_t>(plan.axes),
                                     plan.interleaved);
      }
      return pair(std::move(out[0]), std::move(out[1]));
    }
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

// (q, k, v, cache, block_table, cu_seqlens, start, max_new, rotary, positions) -> q'
PyObject* py_cache8_store_rotary(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != 10 || recording()) Py_RETURN_NONE;
    const Tensor *q = tensor(args[0]), *k = tensor(args[1]), *v = tensor(args[2]), *table = tensor(args[4]),
                 *cu = tensor(args[5]), *start = tensor(args[6]);
    const Tensor* positions = args[9] == Py_None ? nullptr : tensor(args[9]);
    Cache c;
    Rows r;
    Turn t;
    int max_new = 0;
    if (!q || !k || !v || !table || !cu || !start || (args[9] != Py_None && !positions) || !check_rows(*q, *k, &r) ||
        !cache_args(args[3], r.dev, &c) || c.Hk != r.Hk || c.d != r.d || !to_int(args[7], &max_new) ||
        !turn_args(args[8], r.d, r.dev, &t) || (positions && !positions_ok(*positions, t.axes, r.T, r.dev)))
      Py_RETURN_NONE;
    const int64_t B = start->numel(), ldv = rows_stride(*v, r.T, r.Hk, r.d, r.dev);
    if (ldv < 0 || !fits(B) || table->dim() != 2 || !fits(table->size(1)) ||
        !dense(*table, at::kInt, {B, table->size(1)}, r.dev) || !dense(*cu, at::kInt, {B + 1}, r.dev) ||
        !dense(*start, at::kInt, {B}, r.dev))
      Py_RETURN_NONE;
    Tensor out;
    fa_status st;
    {
      WithoutLock unlocked;
      out = at::empty({r.T, r.H, r.d}, q->options().requires_grad(false));
      st = fa_cache8_store_rotary(
          q->data_ptr(), k->data_ptr(), v->data_ptr(), out.data_ptr(), c.t[0]->data_ptr(), c.t[1]->data_ptr(),
          static_cast<float*>(c.t[2]->data_ptr()), static_cast<float*>(c.t[3]->data_ptr()), ints(*table), ints(*cu),
          ints(*start), positions ? ints(*positions) : nullptr, turns_ptr(t), ints(*t.axis), static_cast<int>(B), max_new,
          r.T, c.num_blocks, static_cast<int>(table->size(1)), r.H, r.Hk, c.block, r.d, t.pairs, t.axes, t.interleaved,
          r.ldq, r.ldk, ldv, 1, stream_of(r.dev));
    }
    if (st == FA_OK) return THPVariable_Wrap(std::move(out));
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

// (q, cache, block_table, cu_seqlens, seqlens, max_new, max_seqlen, causal, scale) -> (o, lse)
PyObject* py_chunk_cache8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != 9 || recording()) Py_RETURN_NONE;
    const Tensor *q = tensor(args[0]), *table = tensor(args[2]), *cu = tensor(args[3]), *lens = tensor(args[4]);
    Cache c;
    int max_new = 0, max_seqlen = 0;
    float scale = 0.f;
    if (!q || !table || !cu || !lens || !q->is_cuda() || q->dim() != 3) Py_RETURN_NONE;
    const int dev = q->get_device();
    const int64_t T = q->size(0), H = q->size(1), d = q->size(2), B = lens->numel();
    const int64_t ldq = rows_stride(*q, T, H, d, dev);
    const int causal = PyObject_IsTrue(args[7]);
    if (causal < 0) PyErr_Clear();
    if (causal < 0 || ldq <= 0 || !cache_args(args[1], dev, &c) || !to_int(args[5], &max_new) ||
        !to_int(args[6], &max_seqlen) || !to_scale(args[8], d, &scale))
      Py_RETURN_NONE;
    if (!fits(T) || !fits(H) || !fits(B) || d != c.d || table->dim() != 2 || !fits(table->size(1)) ||
        !dense(*table, at::kInt, {B, table->size(1)}, dev) || !dense(*cu, at::kInt, {B + 1}, dev) ||
        !dense(*lens, at::kInt, {B}, dev))
      Py_RETURN_NONE;
    const int b = static_cast<int>(B), t = static_cast<int>(T), h = static_cast<int>(H);
    const size_t bytes = fa_chunk_cache8_workspace_bytes(b, max_new, t, h, c.Hk, max_seqlen, c.d);
    if (bytes == 0) Py_RETURN_NONE;
    Tensor o, lse;
    fa_status st;
    {
      WithoutLock unlocked;
      const auto opt = q->options().requires_grad(false);
      o = at::empty({T, H, d}, opt);
      lse = at::empty({H, T}, opt.dtype(at::kFloat));
      Tensor ws = at::empty({static_cast<int64_t>(bytes)}, opt.dtype(at::kByte));
      st = fa_fwd_chunk_cache8(
          q->data_ptr(), c.t[0]->data_ptr(), c.t[1]->data_ptr(), static_cast<const float*>(c.t[2]->data_ptr()),
          static_cast<const float*>(c.t[3]->data_ptr()), ints(*table), ints(*cu), ints(*lens), o.data_ptr(),
          static_cast<float*>(lse.data_ptr()), ws.data_ptr(), bytes, b, max_new, t, h, c.Hk, c.num_blocks,
          static_cast<int>(table->size(1)), c.block, max_seqlen, c.d, ldq, scale, causal, 1, stream_of(dev));
    }
    if (st == FA_OK) return pair(std::move(o), std::move(lse));
  } catch (...) {
    PyErr_Clear();  // an exception that came out of Python
  }
  Py_RETURN_NONE;
}

#define FA_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FA_METHOD(forward_grouped), FA_METHOD(backward_grouped), FA_METHOD(flash_attention_grouped),
                         FA_METHOD(cache8_store), FA_METHOD(decode_cache8), FA_METHOD(rotary), FA_METHOD(rotary_embedding),
                         FA_METHOD(cache8_store_rotary), FA_METHOD(chunk_cache8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
