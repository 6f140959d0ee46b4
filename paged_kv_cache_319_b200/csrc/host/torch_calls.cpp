// _torch_calls: the block-sparse entry points for torch tensors, as a Python
// extension. A call looks at 6 to 12 tensors and passes 14 to 27 arguments; asking
// the tensors through Python attributes and passing the arguments through ctypes
// takes 8 to 12 us, more than the kernels of a small step. Here the tensors are
// read through DLPack's C exchange table (torch.Tensor.__dlpack_c_exchange_api__),
// so neither torch's C++ interface nor its ABI is needed.
//
// Each function checks devices, types, shapes and contiguity (ValueError,
// TypeError), launches on the device's current stream with that device current,
// and returns the library's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvp.h"

namespace {

const DLPackExchangeAPI* g_api = nullptr;
PyTypeObject* g_tensor = nullptr;

enum Type { F16 = KVP_F16, BF16 = KVP_BF16, CODES = KVP_FP8_E4M3, F32, I32, I64, OTHER };

struct View {
  PyObject* obj;
  const char* name;
  void* data;
  Type type;
  int device;
  int ndim;
  const int64_t* shape;
  const int64_t* stride;
};

bool error(PyObject* kind, const char* fmt, const char* name) {
  PyErr_Format(kind, fmt, name);
  return false;
}

bool contiguous(const View& v) {
  int64_t expect = 1;
  for (int i = 0; i < v.ndim; ++i)
    if (v.shape[i] == 0) return true;
  for (int i = v.ndim - 1; i >= 0; --i) {
    if (v.shape[i] != 1 && v.stride[i] != expect) return false;
    expect *= v.shape[i];
  }
  return true;
}

// A tensor of `ndim` dimensions on a CUDA device.
bool look(PyObject* o, const char* name, int ndim, View* v) {
  if (!PyObject_TypeCheck(o, g_tensor)) return error(PyExc_TypeError, "%s must be a torch tensor", name);
  DLTensor t;
  if (g_api->dltensor_from_py_object_no_sync(o, &t)) return false;
  if (t.device.device_type != kDLCUDA)
    return error(PyExc_ValueError, "%s: all tensors must be on the same CUDA device", name);
  if (t.ndim != ndim) {
    PyErr_Format(PyExc_ValueError, "%s must have %d dimensions", name, ndim);
    return false;
  }
  *v = View{o,     name,   static_cast<char*>(t.data) + t.byte_offset, OTHER, t.device.device_id,
            ndim, t.shape, t.strides};
  if (t.dtype.lanes == 1) {
    const int code = t.dtype.code, bits = t.dtype.bits;
    if (code == kDLFloat && bits == 16) v->type = F16;
    if (code == kDLBfloat && bits == 16) v->type = BF16;
    if ((code == kDLFloat8_e4m3fn || code == kDLUInt) && bits == 8) v->type = CODES;
    if (code == kDLFloat && bits == 32) v->type = F32;
    if (code == kDLInt && bits == 32) v->type = I32;
    if (code == kDLInt && bits == 64) v->type = I64;
  }
  return true;
}

// The same, contiguous, on the device of `first`.
bool dense(PyObject* o, const char* name, int ndim, int device, View* v) {
  if (!look(o, name, ndim, v)) return false;
  if (v->device != device)
    return error(PyExc_ValueError, "%s: all tensors must be on the same CUDA device", name);
  if (!contiguous(*v)) return error(PyExc_ValueError, "%s must be contiguous", name);
  return true;
}

bool shaped(const View& v, int64_t a, int64_t b = -1, int64_t c = -1, int64_t d = -1) {
  const int64_t want[4] = {a, b, c, d};
  for (int i = 0; i < v.ndim; ++i)
    if (v.shape[i] != want[i]) return error(PyExc_ValueError, "%s: shape mismatch", v.name);
  return true;
}

bool typed(const View& v, Type t, const char* what) {
  if (v.type == t) return true;
  PyErr_Format(PyExc_TypeError, "%s must be %s", v.name, what);
  return false;
}

bool rows16(const View& v) {
  if (v.type == F16 || v.type == BF16) return true;
  return error(PyExc_TypeError, "%s must be float16 or bfloat16", v.name);
}

// Pools beside 16-bit rows of type `t`: of that type, or E4M3.
bool pools(const View& k, const View& v, Type t) {
  if (k.type != v.type || (k.type != t && k.type != CODES))
    return error(PyExc_TypeError, "%s: the caches must have the dtype of the rows, or be E4M3", k.name);
  return shaped(v, k.shape[0], k.shape[1], k.shape[2], k.shape[3]);
}

// The scales of an E4M3 cache (a 16-bit cache has none).
bool scales(PyObject* ks, PyObject* vs, const View& k, const float** kp, const float** vp) {
  *kp = *vp = nullptr;
  if (k.type != CODES) {
    if (ks == Py_None && vs == Py_None) return true;
    return error(PyExc_ValueError, "%s: k_scale / v_scale belong to E4M3 caches", k.name);
  }
  if (ks == Py_None || vs == Py_None)
    return error(PyExc_ValueError, "%s: an E4M3 cache needs k_scale and v_scale", k.name);
  View a, b;
  if (!dense(ks, "k_scale", 1, k.device, &a) || !dense(vs, "v_scale", 1, k.device, &b)) return false;
  if (a.type != F32 || b.type != F32 || a.shape[0] != k.shape[1] || b.shape[0] != k.shape[1])
    return error(PyExc_ValueError, "%s: k_scale / v_scale must be float32 [num_kv_heads]", k.name);
  *kp = static_cast<const float*>(a.data);
  *vp = static_cast<const float*>(b.data);
  return true;
}

bool int32_of(int64_t x, const char* name, int32_t* out) {
  *out = int32_t(x);
  if (x == *out) return true;
  return error(PyExc_ValueError, "%s does not fit 32 bits", name);
}

// An int argument; None stands for `none`.
bool int32_arg(PyObject* o, const char* name, int64_t none, int32_t* out) {
  int64_t x = none;
  if (o != Py_None) {
    x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) return false;
  }
  return int32_of(x, name, out);
}

// Block tables and lengths of S sequences.
struct Batch {
  const int32_t* tables;
  const int32_t* lens;
  int32_t S, max_blocks, max_context_len;
};
bool batch(PyObject* tables, PyObject* lens, PyObject* max_len, int device, int64_t S, int64_t bs,
           Batch* out) {
  View t, l;
  if (!dense(tables, "block_tables", 2, device, &t) || !dense(lens, "context_lens", 1, device, &l) ||
      !typed(t, I32, "int32") || !typed(l, I32, "int32"))
    return false;
  if (S < 0) S = t.shape[0];
  if (t.shape[0] != S || l.shape[0] != S)
    return error(PyExc_ValueError, "%s: batch metadata mismatch", t.name);
  const int64_t room = bs > 0 && t.shape[1] > INT32_MAX / bs ? INT32_MAX : t.shape[1] * bs;
  out->tables = static_cast<const int32_t*>(t.data);
  out->lens = static_cast<const int32_t*>(l.data);
  return int32_of(S, "the batch", &out->S) &&
         int32_of(t.shape[1] ? t.shape[1] : 1, "the table's width", &out->max_blocks) &&
         int32_arg(max_len, "max_context_len", room, &out->max_context_len);
}

// 32-bit sizes of a pool [NB, Hkv, bs, D].
struct Pool {
  int32_t NB, Hkv, bs, D;
};
bool pool_sizes(const View& k, Pool* p) {
  return int32_of(k.shape[0], k.name, &p->NB) && int32_of(k.shape[1], k.name, &p->Hkv) &&
         int32_of(k.shape[2], k.name, &p->bs) && int32_of(k.shape[3], k.name, &p->D);
}

// f(stream)'s status, with `device` current.
template <typename F>
PyObject* launch(int device, F f) {
  void* stream = nullptr;
  if (g_api->current_work_stream(kDLCUDA, device, &stream)) return nullptr;
  int rc = 0, now = device;
  Py_BEGIN_ALLOW_THREADS;
  cudaGetDevice(&now);
  if (now != device) cudaSetDevice(device);
  rc = f(stream);
  if (now != device) cudaSetDevice(now);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (!g_api) {
    PyErr_SetString(PyExc_RuntimeError, "init() has not been called");
    return false;
  }
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
  return false;
}

// Rows [T, H, D] of type t, strided by token; the stride in elements.
bool token_rows(PyObject* o, const char* name, int device, int64_t T, int64_t H, int64_t D, Type t,
                View* v, int64_t* stride) {
  if (!look(o, name, 3, v)) return false;
  if (v->device != device)
    return error(PyExc_ValueError, "%s: all tensors must be on the same CUDA device", name);
  if (v->type != t) return error(PyExc_TypeError, "%s: dtype mismatch", name);
  if (!shaped(*v, T, H, D)) return false;
  if (T && ((v->stride[2] != 1 && D > 1) || (v->stride[1] != D && H > 1)))
    return error(PyExc_ValueError, "%s: the heads of a token must be contiguous", name);
  *stride = T > 1 ? v->stride[0] : H * D;
  return true;
}

// (q, k_new, v_new, cos_sin, positions, k_cache, v_cache, slot_mapping, q_out,
//  interleaved, k_scale, v_scale)
PyObject* call_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  View q, k, v, cs, pos, kc, vc, slots, qo;
  Pool p;
  if (!look(a[5], "k_cache", 4, &kc)) return nullptr;
  const int dev = kc.device;
  if (!dense(a[5], "k_cache", 4, dev, &kc) || !dense(a[6], "v_cache", 4, dev, &vc) ||
      !dense(a[3], "cos_sin", 2, dev, &cs) || !dense(a[4], "positions", 1, dev, &pos) ||
      !dense(a[7], "slot_mapping", 1, dev, &slots) || !look(a[0], "q", 3, &q) || !rows16(q) ||
      !pools(kc, vc, q.type) || !typed(pos, I64, "int64") || !typed(slots, I64, "int64") ||
      !typed(cs, F32, "float32 [max_positions, rot_dim]") || !pool_sizes(kc, &p))
    return nullptr;
  const int64_t T = q.shape[0], Hq = q.shape[1];
  int64_t sq, sk, sv, so;
  const float *ks, *vs;
  int32_t T32, Hq32, rot;
  if (!token_rows(a[0], "q", dev, T, Hq, p.D, q.type, &q, &sq) ||
      !token_rows(a[1], "k_new", dev, T, p.Hkv, p.D, q.type, &k, &sk) ||
      !token_rows(a[2], "v_new", dev, T, p.Hkv, p.D, q.type, &v, &sv) ||
      !token_rows(a[8], "q_out", dev, T, Hq, p.D, q.type, &qo, &so) || !shaped(pos, T) ||
      !shaped(slots, T) || !scales(a[10], a[11], kc, &ks, &vs) ||
      !int32_of(T, "the number of tokens", &T32) || !int32_of(Hq, "the number of heads", &Hq32) ||
      !int32_of(cs.shape[1], "rot_dim", &rot))
    return nullptr;
  const int interleaved = PyObject_IsTrue(a[9]);
  if (interleaved < 0) return nullptr;
  return launch(dev, [&](void* stream) {
    return rope_reshape_and_cache(
        q.data, k.data, v.data, qo.data, sq, sk, sv, so, static_cast<const float*>(cs.data),
        static_cast<const int64_t*>(pos.data), cs.shape[0], rot, interleaved, kc.data, vc.data,
        static_cast<const int64_t*>(slots.data), ks, vs, T32, Hq32, p.Hkv, p.D, p.bs, p.NB, q.type,
        kc.type, stream);
  });
}

// (k_cache, key_bounds, block_tables, context_lens, new_tokens, max_new_tokens,
//  max_context_len); None for a missing one of the last three
PyObject* call_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 7)) return nullptr;
  View kc, b, fresh;
  Pool p;
  Batch s;
  if (!look(a[0], "k_cache", 4, &kc)) return nullptr;
  const int dev = kc.device;
  if (!dense(a[0], "k_cache", 4, dev, &kc) || !dense(a[1], "key_bounds", 4, dev, &b) ||
      !pool_sizes(kc, &p) || !shaped(b, p.NB, p.Hkv, 2, p.D) ||
      !batch(a[2], a[3], a[6], dev, -1, p.bs, &s))
    return nullptr;
  if (kc.type != CODES && !rows16(kc)) return nullptr;
  if (b.type != (kc.type == CODES ? F16 : kc.type)) {
    error(PyExc_TypeError, "%s must have the cache's dtype (float16 over an E4M3 cache)", b.name);
    return nullptr;
  }
  const int32_t* fp = nullptr;
  if (a[4] != Py_None) {
    if (!dense(a[4], "new_tokens", 1, dev, &fresh)) return nullptr;
    if (fresh.type != I32 || fresh.shape[0] != s.S) {
      error(PyExc_ValueError, "%s must be int32 [S]", fresh.name);
      return nullptr;
    }
    fp = static_cast<const int32_t*>(fresh.data);
  }
  int32_t most;
  if (!int32_arg(a[5], "max_new_tokens", s.max_context_len, &most)) return nullptr;
  return launch(dev, [&](void* stream) {
    return update_key_bounds(kc.data, b.data, s.tables, s.lens, fp, s.S, p.Hkv, p.D, p.bs, p.NB,
                             s.max_blocks, s.max_context_len, most, kc.type, stream);
  });
}

// (q, key_bounds, block_tables, context_lens, out, block_size, num_selected, num_sink,
//  num_recent, max_context_len or None)
PyObject* call_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 10)) return nullptr;
  View q, b, out;
  Batch s;
  int32_t bs, keep, sink, recent, NB, Hkv, Hq, D;
  if (!look(a[0], "q", 3, &q)) return nullptr;
  const int dev = q.device;
  if (!dense(a[0], "q", 3, dev, &q) || !rows16(q) || !dense(a[1], "key_bounds", 4, dev, &b) ||
      !dense(a[4], "out", 3, dev, &out) || !int32_arg(a[5], "block_size", 0, &bs) ||
      !int32_arg(a[6], "num_selected", 0, &keep) || !int32_arg(a[7], "num_sink", 0, &sink) ||
      !int32_arg(a[8], "num_recent", 0, &recent) ||
      !batch(a[2], a[3], a[9], dev, q.shape[0], bs, &s) || !int32_of(b.shape[0], b.name, &NB) ||
      !int32_of(b.shape[1], b.name, &Hkv) || !int32_of(q.shape[1], q.name, &Hq) ||
      !int32_of(q.shape[2], q.name, &D) || !shaped(b, NB, Hkv, 2, D))
    return nullptr;
  if (b.type != q.type && b.type != F16) {
    error(PyExc_TypeError, "%s must have q's dtype, or float16 (bounds of an E4M3 cache)", b.name);
    return nullptr;
  }
  if (!typed(out, I32, "int32") || !shaped(out, s.S, Hkv, keep < 0 ? 0 : keep)) return nullptr;
  return launch(dev, [&](void* stream) {
    return select_blocks(q.data, b.data, s.tables, s.lens, static_cast<int32_t*>(out.data), s.S, Hq,
                         Hkv, D, bs, NB, s.max_blocks, s.max_context_len, keep, sink, recent, q.type,
                         b.type == q.type ? int32_t(b.type) : KVP_FP8_E4M3, stream);
  });
}

// (q, k_cache, v_cache, block_tables, context_lens, selected, scale, out, k_scale,
//  v_scale, max_context_len or None)
PyObject* call_sparse(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  View q, kc, vc, sel, out;
  Pool p;
  Batch s;
  const float *ks, *vs;
  int32_t Hq, keep;
  if (!look(a[0], "q", 3, &q)) return nullptr;
  const int dev = q.device;
  if (!dense(a[0], "q", 3, dev, &q) || !rows16(q) || !dense(a[1], "k_cache", 4, dev, &kc) ||
      !dense(a[2], "v_cache", 4, dev, &vc) || !pools(kc, vc, q.type) || !pool_sizes(kc, &p) ||
      !shaped(q, q.shape[0], q.shape[1], p.D) ||
      !batch(a[3], a[4], a[10], dev, q.shape[0], p.bs, &s) ||
      !dense(a[5], "selected", 3, dev, &sel) || !dense(a[7], "out", 3, dev, &out) ||
      !scales(a[8], a[9], kc, &ks, &vs) || !int32_of(q.shape[1], q.name, &Hq) ||
      !int32_of(sel.shape[2], sel.name, &keep))
    return nullptr;
  if (sel.type != I32 || sel.shape[0] != s.S || sel.shape[1] != p.Hkv) {
    error(PyExc_ValueError, "%s must be int32 [S, Hkv, n]", sel.name);
    return nullptr;
  }
  if (out.type != q.type || !shaped(out, s.S, Hq, p.D)) {
    if (!PyErr_Occurred()) error(PyExc_ValueError, "%s must have q's dtype", out.name);
    return nullptr;
  }
  const double scale = PyFloat_AsDouble(a[6]);
  if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  return launch(dev, [&](void* stream) {
    return paged_attention_decode_sparse(
        q.data, kc.data, vc.data, ks, vs, s.tables, s.lens, static_cast<const int32_t*>(sel.data),
        s.S, Hq, p.Hkv, p.D, p.bs, p.NB, s.max_blocks, s.max_context_len, keep, float(scale),
        out.data, q.type, kc.type, stream);
  });
}

// init(torch.Tensor): reads the tensors' exchange table.
PyObject* call_init(PyObject*, PyObject* type) {
  if (!PyType_Check(type)) {
    PyErr_SetString(PyExc_TypeError, "init() takes torch.Tensor");
    return nullptr;
  }
  PyObject* capsule = PyObject_GetAttrString(type, "__dlpack_c_exchange_api__");
  if (!capsule) return nullptr;
  auto* api = static_cast<const DLPackExchangeAPI*>(PyCapsule_GetPointer(capsule, "dlpack_exchange_api"));
  Py_DECREF(capsule);  // the table is static
  if (!api) return nullptr;
  if (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync ||
      !api->current_work_stream) {
    PyErr_SetString(PyExc_RuntimeError, "torch's DLPack exchange table has another version");
    return nullptr;
  }
  Py_INCREF(type);
  g_tensor = reinterpret_cast<PyTypeObject*>(type);
  g_api = api;
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() {
  static PyMethodDef methods[] = {
      {"init", call_init, METH_O, nullptr},
      {"rope_reshape_and_cache", fast(call_rope), METH_FASTCALL, nullptr},
      {"update_key_bounds", fast(call_bounds), METH_FASTCALL, nullptr},
      {"select_blocks", fast(call_select), METH_FASTCALL, nullptr},
      {"paged_attention_decode_sparse", fast(call_sparse), METH_FASTCALL, nullptr},
      {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                               nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&module);
}
