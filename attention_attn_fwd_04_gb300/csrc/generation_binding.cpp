// generation_binding.cpp -- CPython side of the generation calls
// (generation.py): reads the tensors, makes the outputs, calls the C ABI.
//
// A decode step is a handful of calls whose kernels take a few microseconds;
// marshalled through ctypes each of them cost 12 to 26 us of host time, most
// of it attribute reads and small allocations from Python.  Nothing is
// computed here.  Every function returns its tensors, or the status of the
// library as an int where the library refused.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn.h"

namespace {

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* fmt, const char* name) {
  PyErr_Format(PyExc_ValueError, fmt, name);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

int64_t integer(PyObject* o, const char* name, int64_t lo, int64_t hi) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < lo || v > hi) refuse("%s is out of range", name);
  return v;
}
int32_t int32(PyObject* o, const char* name) {
  return static_cast<int32_t>(integer(o, name, INT32_MIN, INT32_MAX));
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();  // such as a tensor of several elements
  return v != 0;
}

// dim-dimensional, of this type, on this device, last dimension contiguous
void rows(const at::Tensor& t, const char* name, at::ScalarType dt, int64_t dim, at::Device dev) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  if (t.layout() != at::kStrided || t.scalar_type() != dt || t.dim() != dim || t.device() != dev) {
    PyErr_Format(PyExc_ValueError, "%s must be a %d-dimensional %s tensor on %s", name, (int)dim,
                 c10::toString(dt), dev.str().c_str());
    throw Refused();
  }
  if (t.stride(dim - 1) != 1 && t.size(dim - 1) != 1)
    refuse("%s must be contiguous in its last dimension", name);
}

// contiguous, of this type and shape, on this device
void flat(const at::Tensor& t, const char* name, at::ScalarType dt, at::IntArrayRef shape,
          at::Device dev) {
  if (!t.is_cuda() || t.layout() != at::kStrided || t.scalar_type() != dt || t.device() != dev ||
      t.sizes() != shape || !t.is_contiguous()) {
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s %s] tensor on %s", name,
                 c10::toString(dt), s.c_str(), dev.str().c_str());
    throw Refused();
  }
}

int32_t narrow(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse("%s is too large", name);
  return static_cast<int32_t>(v);
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dt, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(dt).device(dev));
}

// Part of a buffer from a byte on, as a tensor of its own (a view without the
// dispatcher's cost, and one allocation for several small outputs).
at::Tensor piece(const at::Tensor& buf, int64_t byte, at::IntArrayRef shape, at::ScalarType dt) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(buf.storage()), buf.key_set(), c10::scalarTypeToTypeMeta(dt));
  t.unsafeGetTensorImpl()->set_storage_offset(byte / (int64_t)c10::elementSize(dt));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

attn_stream_t stream_of(at::Device dev) {
  return reinterpret_cast<attn_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// A tensor's strides outside its last dimension.
const int64_t* strides(const at::Tensor& t) { return t.strides().data(); }

template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// After a call that writes into a caller's tensor: its next version, so that
// autograd's check of the tensors it saved sees the write.  Tensors of inference
// mode have no version.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

const attn_rope_plan* plan_at(PyObject* o) {
  const unsigned long long a = PyLong_AsUnsignedLongLong(o);
  if (a == (unsigned long long)-1 && PyErr_Occurred()) throw Refused();
  return reinterpret_cast<const attn_rope_plan*>(static_cast<uintptr_t>(a));
}

template <typename F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// rope(back, x, plan, positions, offset, out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const bool back = truth(a[0]);
    const char* name = back ? "dout" : "x";
    const at::Tensor& x = tensor(a[1], name);
    const at::Device dev = x.device();
    rows(x, name, at::kBFloat16, 4, dev);
    const attn_rope_plan* plan = plan_at(a[2]);
    const int64_t B = x.size(0), H = x.size(1), S = x.size(2), D = x.size(3);
    const int32_t* pos = nullptr;
    int64_t pos_stride = 0;
    if (given(a[3])) {
      const at::Tensor& p = tensor(a[3], "positions");
      rows(p, "positions", at::kInt, p.dim() == 1 ? 1 : 2, dev);
      const int64_t nr = p.dim() == 1 ? 1 : p.size(0);
      if (p.size(-1) != S || (nr != 1 && nr != B))
        refuse("%s must be [S], [1, S] or [B, S]", "positions");
      pos = data<int32_t>(p);
      if (nr > 1) pos_stride = p.stride(0);
    }
    const int32_t offset = int32(a[4], "offset");
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor y;
    if (given(a[5])) {
      y = tensor(a[5], "out");
      rows(y, "out", at::kBFloat16, 4, dev);
      if (y.sizes() != x.sizes()) refuse("%s must have the shape of the input", "out");
    } else {
      y = at::empty_like(x);
      if (y.stride(3) != 1) y = fresh(x.sizes(), at::kBFloat16, dev);
    }
    if (x.numel() > 0) {
      const attn_status st = (back ? attn_rope_bwd : attn_rope)(
          x.data_ptr(), strides(x), y.data_ptr(), strides(y), narrow(B, "B"), narrow(H, "H"),
          narrow(S, "S"), narrow(D, "D"), pos, pos_stride, offset, plan, stream_of(dev));
      if (st != ATTN_OK) return PyLong_FromLong(st);
      if (given(a[5])) written(y);
    }
    return THPVariable_Wrap(std::move(y));
  });
}

// slots(ctx, new, table, free, n_free, page_size, num_pages, max_tokens, out)
PyObject* slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& table = tensor(a[2], "block_table");
    const at::Device dev = table.device();
    rows(table, "block_table", at::kInt, 2, dev);
    const int64_t B = table.size(0);
    const at::Tensor &ctx = tensor(a[0], "ctx_lens"), &add = tensor(a[1], "new_lens");
    flat(ctx, "ctx_lens", at::kInt, {B}, dev);
    flat(add, "new_lens", at::kInt, {B}, dev);
    if (given(a[3]) != given(a[4])) refuse("%s and n_free come together", "free_pages");
    const bool pool = given(a[3]);
    const int32_t *free_pages = nullptr, *n_free = nullptr;
    int64_t cap = 0;
    if (pool) {
      const at::Tensor &f = tensor(a[3], "free_pages"), &l = tensor(a[4], "n_free");
      cap = f.numel();
      if (cap == 0) refuse("%s must hold at least one entry", "free_pages");
      flat(f, "free_pages", at::kInt, {cap}, dev);
      flat(l, "n_free", at::kInt, {1}, dev);
      free_pages = data<int32_t>(f);
      n_free = data<int32_t>(l);
    }
    const int32_t page = int32(a[5], "page_size"), pages = int32(a[6], "num_pages");
    const int32_t T = int32(a[7], "max_tokens");
    if (T <= 0 || B <= 0) refuse("%s and the number of requests must be > 0", "max_tokens");
    const c10::cuda::CUDAGuard guard(dev);
    static const char* const names[6] = {"out.seq_lens", "out.cu_new", "out.token_req",
                                         "out.positions", "out.slots", "out.n_free"};
    const int64_t sizes[6] = {B, B + 1, T, T, T, 1};
    at::Tensor out[6], buf;
    int64_t at_byte = 0;
    if (!given(a[8])) {  // the 8-byte slots first
      buf = fresh({8 * (int64_t)T + 4 * (2 * (int64_t)T + 2 * B + 2)}, at::kByte, dev);
      out[4] = piece(buf, 0, {T}, at::kLong);
      at_byte = 8 * (int64_t)T;
    }
    for (int i = 0; i < 6; ++i) {
      const at::ScalarType dt = i == 4 ? at::kLong : at::kInt;
      if (!given(a[8])) {
        if (i == 4 || (i == 5 && !pool)) continue;
        out[i] = piece(buf, at_byte, {sizes[i]}, dt);
        at_byte += 4 * sizes[i];
        continue;
      }
      if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 6)
        refuse("%s must be what an earlier call returned", "out");
      PyObject* o = PyTuple_GET_ITEM(a[8], i);
      if (i == 5 && given(o) != pool) refuse("%s and n_free come together", names[i]);
      if (i == 5 && !pool) continue;
      out[i] = tensor(o, names[i]);
      flat(out[i], names[i], dt, {sizes[i]}, dev);
    }
    const attn_status st = attn_cache_slots(
        data<int32_t>(ctx), data<int32_t>(add), narrow(B, "B"), page, pages, data<int32_t>(table),
        table.stride(0), narrow(table.size(1), "max_pages"), free_pages, narrow(cap, "free_pages"),
        n_free, data<int32_t>(out[0]), data<int32_t>(out[1]), data<int32_t>(out[2]),
        data<int32_t>(out[3]), data<int64_t>(out[4]), pool ? data<int32_t>(out[5]) : nullptr, T,
        stream_of(dev));
    if (st != ATTN_OK) return PyLong_FromLong(st);
    if (pool) written(table);
    if (given(a[8])) {
      for (int i = 0; i < (pool ? 6 : 5); ++i) written(out[i]);
      Py_INCREF(a[8]);
      return a[8];
    }
    PyObject* t = PyTuple_New(6);
    if (t == nullptr) return nullptr;
    for (int i = 0; i < 6; ++i) {
      PyObject* o = i < 5 || pool ? THPVariable_Wrap(std::move(out[i])) : Py_NewRef(Py_None);
      if (o == nullptr) {
        Py_DECREF(t);
        return nullptr;
      }
      PyTuple_SET_ITEM(t, i, o);
    }
    return t;
  });
}

// The cache of a call.
attn_cache_desc cache_of(PyObject* k, PyObject* v, PyObject* ks, PyObject* vs, at::Device dev) {
  const at::Tensor &kc = tensor(k, "k_cache"), &vc = tensor(v, "v_cache");
  const at::ScalarType dt = kc.scalar_type();
  if (dt != at::kBFloat16 && dt != at::kFloat8_e4m3fn)
    refuse("%s must be bfloat16 or float8_e4m3fn", "caches");
  rows(kc, "k_cache", dt, 4, dev);
  rows(vc, "v_cache", dt, 4, dev);
  if (kc.sizes() != vc.sizes()) refuse("%s and v_cache must have one shape", "k_cache");
  attn_cache_desc d;
  std::memset(&d, 0, sizeof(d));
  d.version = 1;
  d.dtype = dt == at::kBFloat16 ? ATTN_CACHE_BF16 : ATTN_CACHE_E4M3;
  d.num_pages = narrow(kc.size(0), "num_pages");
  d.H_kv = narrow(kc.size(1), "H_kv");
  d.page_size = narrow(kc.size(2), "page_size");
  d.D = narrow(kc.size(3), "D");
  d.k = kc.data_ptr();
  d.v = vc.data_ptr();
  for (int i = 0; i < 3; ++i) {
    d.k_strides[i] = kc.stride(i);
    d.v_strides[i] = vc.stride(i);
  }
  if (given(ks) || given(vs)) {
    if (dt == at::kBFloat16) refuse("%s and v_scale go with float8_e4m3fn caches", "k_scale");
    if (given(ks)) {
      const at::Tensor& s = tensor(ks, "k_scale");
      flat(s, "k_scale", at::kFloat, {kc.size(1)}, dev);
      d.k_scale = data<float>(s);
    }
    if (given(vs)) {
      const at::Tensor& s = tensor(vs, "v_scale");
      flat(s, "v_scale", at::kFloat, {kc.size(1)}, dev);
      d.v_scale = data<float>(s);
    }
  }
  return d;
}

// append(k, v, k_cache, v_cache, slots, q, q_out, plan, positions, k_scale, v_scale)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const at::Device dev = k.device();
    rows(k, "k", at::kBFloat16, 3, dev);
    rows(v, "v", at::kBFloat16, 3, dev);
    const attn_cache_desc d = cache_of(a[2], a[3], a[9], a[10], dev);
    const int64_t T = k.size(0);
    if (v.sizes() != k.sizes() || k.size(1) != d.H_kv || k.size(2) != d.D)
      refuse("%s and v must be [T, H_kv, D] of the caches", "k");
    const at::Tensor& sl = tensor(a[4], "slots");
    flat(sl, "slots", at::kLong, {T}, dev);
    if (given(a[7]) != given(a[8])) refuse("%s and positions come together", "plan");
    const attn_rope_plan* plan = nullptr;
    const int32_t* pos = nullptr;
    if (given(a[7])) {
      plan = plan_at(a[7]);
      const at::Tensor& p = tensor(a[8], "positions");
      flat(p, "positions", at::kInt, {T}, dev);
      pos = data<int32_t>(p);
    }
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor y;
    const at::Tensor* q = nullptr;
    if (given(a[5])) {
      q = &tensor(a[5], "q");
      rows(*q, "q", at::kBFloat16, 3, dev);
      if (q->size(0) != T || q->size(2) != d.D) refuse("%s must be [T, H, D]", "q");
      if (given(a[6])) {
        y = tensor(a[6], "q_out");
        rows(y, "q_out", at::kBFloat16, 3, dev);
        if (y.sizes() != q->sizes()) refuse("%s must have the shape of q", "q_out");
      } else {
        y = fresh(q->sizes(), at::kBFloat16, dev);
      }
    } else if (given(a[6])) {
      refuse("%s without q", "q_out");
    }
    if (T > 0) {
      const attn_status st = attn_cache_append(
          q ? q->data_ptr() : nullptr, q ? strides(*q) : nullptr, k.data_ptr(), strides(k),
          v.data_ptr(), strides(v), q ? y.data_ptr() : nullptr, q ? strides(y) : nullptr,
          narrow(T, "T"), q ? narrow(q->size(1), "H") : 0, pos, data<int64_t>(sl), plan, &d,
          stream_of(dev));
      if (st != ATTN_OK) return PyLong_FromLong(st);
      written(tensor(a[2], "k_cache"));
      written(tensor(a[3], "v_cache"));
      if (given(a[6])) written(y);
    }
    if (q == nullptr) return Py_NewRef(Py_None);
    return THPVariable_Wrap(std::move(y));
  });
}

// decode(q, k_cache, v_cache, table, lens, scale, window, alibi, alibi_slopes, softcap, rel_bias,
//        k_scale, v_scale, out, lse, return_lse, workspace)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 17)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const at::Device dev = q.device();
    rows(q, "q", at::kBFloat16, 3, dev);
    const attn_cache_desc d = cache_of(a[1], a[2], a[11], a[12], dev);
    const int64_t B = q.size(0), H = q.size(1), D = q.size(2);
    if (D != d.D) refuse("%s must be [B, H, D] of the caches", "q");
    const at::Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
    rows(table, "block_table", at::kInt, 2, dev);
    if (table.size(0) != B) refuse("%s must be [B, max_pages]", "block_table");
    flat(lens, "seq_lens", at::kInt, {B}, dev);
    const float scale =
        given(a[5]) ? (float)real(a[5]) : (float)(1.0 / std::sqrt((double)(D > 0 ? D : 1)));
    attn_mod_desc m;
    std::memset(&m, 0, sizeof(m));
    m.version = ATTN_MOD_DESC_VERSION;
    if (given(a[6])) {  // window <= 0 is rejected by the library
      m.mask_flags |= ATTN_MASK_WINDOW;
      m.window = int32(a[6], "window");
    }
    if (given(a[8])) {
      const at::Tensor& s = tensor(a[8], "alibi_slopes");
      flat(s, "alibi_slopes", at::kFloat, {H}, dev);
      m.alibi_slopes = data<float>(s);
    }
    if (truth(a[7]) || given(a[8])) m.score_flags |= ATTN_SCORE_ALIBI;
    if (given(a[9])) {
      m.softcap = (float)real(a[9]);
      if (m.softcap != 0.0f) m.score_flags |= ATTN_SCORE_SOFTCAP;
    }
    if (given(a[10])) {
      const at::Tensor& r = tensor(a[10], "rel_bias");
      if (r.dim() != 2 || r.size(1) % 2 != 1) refuse("%s must be [H, 2R+1]", "rel_bias");
      flat(r, "rel_bias", at::kFloat, {H, r.size(1)}, dev);
      m.score_flags |= ATTN_SCORE_RELBIAS;
      m.rel_bias = data<float>(r);
      m.rel_max = narrow((r.size(1) - 1) / 2, "rel_bias");
    }
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out, lse, ws;
    const bool want_lse = truth(a[15]);
    if (given(a[13])) {
      out = tensor(a[13], "out");
      flat(out, "out", at::kBFloat16, {B, H, D}, dev);
    }
    if (given(a[14])) {
      lse = tensor(a[14], "lse");
      flat(lse, "lse", at::kFloat, {B, H}, dev);
    }
    if (!out.defined() && !lse.defined() && want_lse) {  // one allocation for both
      const int64_t o_bytes = (2 * B * H * D + 15) / 16 * 16;
      const at::Tensor buf = fresh({o_bytes + 4 * B * H}, at::kByte, dev);
      out = piece(buf, 0, {B, H, D}, at::kBFloat16);
      lse = piece(buf, o_bytes, {B, H}, at::kFloat);
    }
    if (!out.defined()) out = fresh({B, H, D}, at::kBFloat16, dev);
    if (!lse.defined() && want_lse) lse = fresh({B, H}, at::kFloat, dev);
    if (B > 0) {
      if (given(a[16])) {
        ws = tensor(a[16], "workspace");
        flat(ws, "workspace", at::kByte, {ws.numel()}, dev);
      } else {
        const size_t need = attn_decode_workspace_bytes(narrow(H, "H"), d.H_kv, d.D);
        // sizes that need no workspace are refused below: any buffer will do
        ws = fresh({(int64_t)(need > 0 ? need : 16)}, at::kByte, dev);
      }
      const attn_status st = attn_decode(
          q.data_ptr(), strides(q), &d, data<int32_t>(table), table.stride(0),
          narrow(table.size(1), "max_pages"), data<int32_t>(lens), out.data_ptr(),
          lse.defined() ? data<float>(lse) : nullptr, narrow(B, "B"), narrow(H, "H"), scale,
          (m.mask_flags | m.score_flags) != 0 ? &m : nullptr, ws.data_ptr(), (size_t)ws.numel(),
          stream_of(dev));
      if (st != ATTN_OK) return PyLong_FromLong(st);
      if (given(a[13])) written(out);
      if (given(a[14])) written(lse);
      if (given(a[16])) written(ws);
    }
    PyObject* o = THPVariable_Wrap(std::move(out));
    if (!want_lse || o == nullptr) return o;
    PyObject* l = THPVariable_Wrap(std::move(lse));
    PyObject* t = l != nullptr ? PyTuple_New(2) : nullptr;
    if (t == nullptr) {
      Py_DECREF(o);
      Py_XDECREF(l);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, o);
    PyTuple_SET_ITEM(t, 1, l);
    return t;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

}  // namespace

extern "C" PyObject* PyInit__generation() {
  static PyMethodDef methods[] = {method<rope>("rope"), method<slots>("slots"),
                                  method<append>("append"), method<decode>("decode"),
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_generation", nullptr, -1, methods,
                            nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&def);
}
