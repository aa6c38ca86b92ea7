// marshal.cpp -- the binding's arguments in one step.
//
// A call of a few microseconds on the GPU is bound by the host: in Python, reading
// the pointer, type, shape and strides of a dozen tensors and checking them takes
// longer than the launch.  pack(format, device, ...) does that for a whole call and
// returns the C entry point's arguments as a tuple, or None when anything is not
// plainly as the format says; the Python code then goes through its own checks,
// which word the refusal (or take the rarer form).  Nothing is kept between calls.
//
// Format letters (sizes B, H, T, D are those of the first x / y):
//   x  tensor, bf16 or f32, 4-D          -> attn_tensor as bytes
//   y  the same, or 3-D [B, H, D] rows read as [B, H, 1, D]; all y's alike
//   X, Y  as x, y, of the first's sizes (Y: and type)
//   o  as x, or None                     -> bytes or None
//   c  two tensors: a K and a V cache    -> attn_kv_cache as bytes
//   b  block table, >= B rows            -> pointer, row stride, columns
//   V  int32 vector that sets B          -> pointer
//   v  int32 vector of B                 -> pointer
//   n  int32 vector of B, or None        -> pointer or None
//   R  int32 [B, T] rows (y's 3-D: [B])  -> pointer, row stride
//   r  int32 [B, n] rows                 -> pointer, row stride, n
//   q  int32 [B, T] rows                 -> pointer, row stride
//   f  int64 frequencies, 1 .. D / 2     -> pointer, twice their number
//   l  f32, contiguous, B H T elements, or None -> pointer or None
//   A  f32 [blocks, Hkv, 16] of the cache -> pointer
//   K  int32, contiguous [B, Hkv, n]     -> pointer
//   =  any object                        -> itself
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>

#include "libattn.h"

namespace {

struct Sizes {
  int64_t B = -1, H = 0, T = 0, D = 0;
  int64_t blocks = 0, kv_heads = 0, slots = 0;  // of the cache
  int64_t table_rows = -1;  // least of the block tables seen
  at::ScalarType type = at::kBFloat16;
  bool one_token = false;
};

bool on(const at::Tensor& t, int64_t device) { return t.is_cuda() && t.get_device() == device; }

bool describe(const at::Tensor& t, int64_t device, bool insert, attn_tensor* d) {
  if (!on(t, device)) return false;
  const auto type = t.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) return false;
  const int64_t n = t.dim();
  if (n != (insert ? 3 : 4)) return false;
  std::memset(d, 0, sizeof(*d));
  d->data = t.data_ptr();
  d->dtype = type == at::kBFloat16 ? ATTN_BF16 : ATTN_F32;
  d->ndim = 4;
  for (int i = 0, k = 0; i < 4; ++i) {
    if (insert && i == 2) {
      d->shape[2] = 1;
      d->stride[2] = t.size(2) * t.stride(2);
      continue;
    }
    d->shape[i] = t.size(k);
    d->stride[i] = t.stride(k);
    ++k;
  }
  return true;
}

bool int32_rows(const at::Tensor& t, int64_t device) {
  return on(t, device) && t.scalar_type() == at::kInt && t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1);
}

PyObject* address(const at::Tensor& t) { return PyLong_FromVoidPtr(t.data_ptr()); }

PyObject* pack(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs < 2 || !PyUnicode_Check(args[0]) || !PyLong_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "pack(format, device, ...)");
    return nullptr;
  }
  const char* f = PyUnicode_AsUTF8(args[0]);
  const int64_t device = PyLong_AsLongLong(args[1]);
  if (f == nullptr || (device == -1 && PyErr_Occurred())) return nullptr;
  PyObject* out[64];
  int n = 0;
  Py_ssize_t a = 2;
  Sizes s;
  bool ok = true, error = false;
  auto put = [&](PyObject* o) {
    if (o == nullptr || n == 64) {
      error = true;
      Py_XDECREF(o);
    } else {
      out[n++] = o;
    }
  };
  auto none = [&] { Py_INCREF(Py_None); put(Py_None); };
  try {
    for (; ok && !error && *f != 0; ++f) {
      if (a >= nargs) {
        ok = false;
        break;
      }
      PyObject* o = args[a++];
      if (*f == '=') {
        Py_INCREF(o);
        put(o);
        continue;
      }
      if (o == Py_None && (*f == 'o' || *f == 'n' || *f == 'l')) {
        none();
        continue;
      }
      if (!THPVariable_Check(o)) {
        ok = false;
        break;
      }
      const at::Tensor& t = THPVariable_Unpack(o);
      switch (*f) {
        case 'x':
        case 'y':
        case 'X':
        case 'Y':
        case 'o': {
          attn_tensor d;
          const bool first = s.B < 0;
          const bool insert = (*f == 'y' || *f == 'Y') && (first ? t.dim() == 3 : s.one_token);
          ok = describe(t, device, insert, &d);
          if (*f == 'X' || *f == 'Y')
            ok = ok && d.shape[0] == s.B && d.shape[1] == s.H && d.shape[2] == s.T && d.shape[3] == s.D &&
                 (*f == 'X' || t.scalar_type() == s.type);
          if (!ok) break;
          if (first) {
            s.B = d.shape[0], s.H = d.shape[1], s.T = d.shape[2], s.D = d.shape[3];
            s.type = t.scalar_type();
            s.one_token = insert;
          }
          put(PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&d), sizeof(d)));
          break;
        }
        case 'c': {
          if (a >= nargs || !THPVariable_Check(args[a])) {
            ok = false;
            break;
          }
          const at::Tensor& v = THPVariable_Unpack(args[a++]);
          ok = on(t, device) && on(v, device) && t.dim() == 4 && t.sizes() == v.sizes() &&
               t.scalar_type() == v.scalar_type() && t.is_contiguous() && v.is_contiguous() &&
               (t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat);
          if (!ok) break;
          attn_kv_cache c;
          std::memset(&c, 0, sizeof(c));
          c.k = t.data_ptr();
          c.v = v.data_ptr();
          c.dtype = t.scalar_type() == at::kBFloat16 ? ATTN_BF16 : ATTN_F32;
          c.num_blocks = s.blocks = t.size(0);
          c.num_kv_heads = static_cast<int32_t>(s.kv_heads = t.size(1));
          c.block_size = static_cast<int32_t>(s.slots = t.size(2));
          c.head_dim = static_cast<int32_t>(t.size(3));
          put(PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&c), sizeof(c)));
          break;
        }
        case 'b':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) >= s.B && t.stride(1) == 1 &&
               t.stride(0) >= t.size(1);
          if (!ok) break;
          s.table_rows = s.table_rows < 0 ? t.size(0) : std::min(s.table_rows, t.size(0));
          put(address(t));
          put(PyLong_FromLongLong(t.stride(0)));
          put(PyLong_FromLongLong(t.size(1)));
          break;
        case 'V':
        case 'v':
        case 'n':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 1 && t.is_contiguous() &&
               (*f == 'V' || t.size(0) == s.B);
          if (!ok) break;
          if (*f == 'V') {
            s.B = t.size(0);
            ok = s.table_rows < 0 || s.table_rows >= s.B;
            if (!ok) break;
          }
          put(address(t));
          break;
        case 'R':
          if (s.one_token) {  // [B]: a row of one
            ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == s.B;
            if (!ok) break;
            put(address(t));
            put(PyLong_FromLongLong(t.stride(0)));
            break;
          }
          [[fallthrough]];
        case 'q':
          ok = int32_rows(t, device) && t.size(0) == s.B && t.size(1) == s.T;
          if (!ok) break;
          put(address(t));
          put(PyLong_FromLongLong(t.stride(0)));
          break;
        case 'r':
          ok = int32_rows(t, device) && t.size(0) == s.B;
          if (!ok) break;
          put(address(t));
          put(PyLong_FromLongLong(t.stride(0)));
          put(PyLong_FromLongLong(t.size(1)));
          break;
        case 'f':
          ok = on(t, device) && t.scalar_type() == at::kLong && t.dim() == 1 && t.is_contiguous() && t.size(0) >= 1 &&
               t.size(0) <= s.D / 2;
          if (!ok) break;
          put(address(t));
          put(PyLong_FromLongLong(2 * t.size(0)));
          break;
        case 'l':
          ok = on(t, device) && t.scalar_type() == at::kFloat && t.is_contiguous() && t.numel() == s.B * s.H * s.T;
          if (!ok) break;
          put(address(t));
          break;
        case 'A':
          ok = on(t, device) && t.scalar_type() == at::kFloat && t.is_contiguous() && t.dim() == 3 &&
               t.size(0) == s.blocks && t.size(1) == s.kv_heads && t.size(2) == s.slots;
          if (!ok) break;
          put(address(t));
          break;
        case 'K':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.is_contiguous() && t.dim() == 3 && t.size(0) == s.B &&
               t.size(1) == s.kv_heads;
          if (!ok) break;
          put(address(t));
          break;
        default:
          PyErr_Format(PyExc_ValueError, "pack: no format letter %c", *f);
          error = true;
      }
    }
  } catch (...) {  // a tensor without storage and the like: not plainly what the format says
    ok = false;
  }
  if (!error && ok && a != nargs) ok = false;
  if (error || !ok) {
    for (int i = 0; i < n; ++i) Py_DECREF(out[i]);
    if (error) {
      if (!PyErr_Occurred()) PyErr_NoMemory();
      return nullptr;
    }
    Py_RETURN_NONE;
  }
  PyObject* tuple = PyTuple_New(n);
  if (tuple == nullptr) {
    for (int i = 0; i < n; ++i) Py_DECREF(out[i]);
    return nullptr;
  }
  for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(tuple, i, out[i]);
  return tuple;
}

PyMethodDef kMethods[] = {
    {"pack", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(pack)), METH_FASTCALL,
     "pack(format, device, ...): a C entry point's arguments, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "The binding's arguments in one step.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__marshal(void) { return PyModule_Create(&kModule); }
