// marshal.cpp -- a call of the binding in one step.
//
// A call of a few microseconds on the GPU is bound by the host: in Python, reading
// the pointer, type, shape and strides of a dozen tensors, checking them and
// converting them for the C entry takes longer than the launch.  call(address,
// name, format, ...) does that for a whole call on the current device and returns
// the entry's status, or None (and calls nothing) when anything is not plainly as the format
// says; the Python code then goes through its own checks, which word the refusal
// (or take the rarer form).  Nothing is kept between calls.
//
// Format letters (sizes B, H, T, D are those of the first x / y):
//   x  tensor, bf16 or f32, 4-D          -> attn_tensor
//   y  the same, or 3-D [B, H, D] rows read as [B, H, 1, D]; all y's alike
//   X, Y  as x, y, of the first's sizes (Y: and type)
//   o  as x, or None                     -> attn_tensor or null
//   c  two tensors: a K and a V cache    -> attn_kv_cache
//   b  block table, >= B rows            -> pointer, row stride, columns
//   V  int32 vector that sets B          -> pointer
//   v  int32 vector of B                 -> pointer
//   n  int32 vector of B, or None        -> pointer or null
//   R  int32 [B, T] rows (y's 3-D: [B])  -> pointer, row stride
//   r  int32 [B, n] rows                 -> pointer, row stride, n
//   q  int32 [B, T] rows                 -> pointer, row stride
//   f  int64 frequencies, 1 .. D / 2     -> pointer, twice their number
//   l  f32, contiguous, B H T elements, or None -> pointer or null
//   A  f32 [blocks, Hkv, 16] of the cache -> pointer
//   K  int32, contiguous [B, Hkv, n]     -> pointer
//   W  a workspace's bytes               -> pointer, their number
//   S  a stream handle, or None          -> itself, or the current stream
//   =  an int or a float                 -> itself
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <type_traits>
#include <utility>

#include "libattn.h"

namespace {

// One argument of a C entry: a pointer or an integer, or a float.
struct Value {
  int64_t i = 0;
  double d = 0.0;
};

template <typename T>
T as(const Value& v) {
  if constexpr (std::is_pointer_v<T>)
    return reinterpret_cast<T>(static_cast<intptr_t>(v.i));
  else if constexpr (std::is_floating_point_v<T>)
    return static_cast<T>(v.d);
  else
    return static_cast<T>(v.i);
}

template <typename... A, size_t... I>
int invoke(attn_status (*fn)(A...), const Value* v, std::index_sequence<I...>) {
  return static_cast<int>(fn(as<A>(v[I])...));
}
// fn: an entry of this declaration, at `address`; -1 if it takes another number of arguments
template <typename... A>
int invoke(attn_status (*)(A...), intptr_t address, const Value* v, size_t n) {
  if (n != sizeof...(A)) return -1;
  return invoke(reinterpret_cast<attn_status (*)(A...)>(address), v, std::index_sequence_for<A...>());
}

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

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs < 3 || !PyLong_Check(args[0]) || !PyUnicode_Check(args[1]) || !PyUnicode_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "call(address, name, format, ...)");
    return nullptr;
  }
  const intptr_t entry = static_cast<intptr_t>(PyLong_AsLongLong(args[0]));
  const char* name = PyUnicode_AsUTF8(args[1]);
  const char* f = PyUnicode_AsUTF8(args[2]);
  if (name == nullptr || f == nullptr || PyErr_Occurred()) return nullptr;
  constexpr int kMost = 32;
  Value out[kMost];
  attn_tensor tensors[8];
  attn_kv_cache cache;
  int n = 0, n_tensors = 0;
  Py_ssize_t a = 3;
  Sizes s;
  bool ok = true, error = false;
  auto put = [&](int64_t i) {
    if (n == kMost)
      ok = false;
    else
      out[n++].i = i;
  };
  auto address = [](const void* p) { return static_cast<int64_t>(reinterpret_cast<intptr_t>(p)); };
  try {
    const int64_t device = c10::cuda::current_device();
    for (; ok && !error && *f != 0; ++f) {
      if (a >= nargs) {
        ok = false;
        break;
      }
      PyObject* o = args[a++];
      if (o == Py_None && *f == 'S') {
        put(address(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream()));
        continue;
      }
      if (o == Py_None && (*f == 'o' || *f == 'n' || *f == 'l')) {
        put(0);
        continue;
      }
      if (*f == '=' || *f == 'S') {
        if (*f == '=' && PyFloat_Check(o) && n < kMost) {
          out[n++].d = PyFloat_AS_DOUBLE(o);
        } else if (PyLong_Check(o)) {
          int past = 0;
          put(PyLong_AsLongLongAndOverflow(o, &past));
          ok = ok && past == 0;
        } else {
          ok = false;
        }
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
          if (n_tensors == 8) {
            ok = false;
            break;
          }
          attn_tensor& d = tensors[n_tensors];
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
          ++n_tensors;
          put(address(&d));
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
          attn_kv_cache& c = cache;
          std::memset(&c, 0, sizeof(c));
          c.k = t.data_ptr();
          c.v = v.data_ptr();
          c.dtype = t.scalar_type() == at::kBFloat16 ? ATTN_BF16 : ATTN_F32;
          c.num_blocks = s.blocks = t.size(0);
          c.num_kv_heads = static_cast<int32_t>(s.kv_heads = t.size(1));
          c.block_size = static_cast<int32_t>(s.slots = t.size(2));
          c.head_dim = static_cast<int32_t>(t.size(3));
          put(address(&c));
          break;
        }
        case 'b':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) >= s.B && t.stride(1) == 1 &&
               t.stride(0) >= t.size(1);
          if (!ok) break;
          s.table_rows = s.table_rows < 0 ? t.size(0) : std::min(s.table_rows, t.size(0));
          put(address(t.data_ptr()));
          put(t.stride(0));
          put(t.size(1));
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
          put(address(t.data_ptr()));
          break;
        case 'R':
          if (s.one_token) {  // [B]: a row of one
            ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == s.B;
            if (!ok) break;
            put(address(t.data_ptr()));
            put(t.stride(0));
            break;
          }
          [[fallthrough]];
        case 'q':
          ok = int32_rows(t, device) && t.size(0) == s.B && t.size(1) == s.T;
          if (!ok) break;
          put(address(t.data_ptr()));
          put(t.stride(0));
          break;
        case 'r':
          ok = int32_rows(t, device) && t.size(0) == s.B;
          if (!ok) break;
          put(address(t.data_ptr()));
          put(t.stride(0));
          put(t.size(1));
          break;
        case 'f':
          ok = on(t, device) && t.scalar_type() == at::kLong && t.dim() == 1 && t.is_contiguous() && t.size(0) >= 1 &&
               t.size(0) <= s.D / 2;
          if (!ok) break;
          put(address(t.data_ptr()));
          put(2 * t.size(0));
          break;
        case 'l':
          ok = on(t, device) && t.scalar_type() == at::kFloat && t.is_contiguous() && t.numel() == s.B * s.H * s.T;
          if (!ok) break;
          put(address(t.data_ptr()));
          break;
        case 'A':
          ok = on(t, device) && t.scalar_type() == at::kFloat && t.is_contiguous() && t.dim() == 3 &&
               t.size(0) == s.blocks && t.size(1) == s.kv_heads && t.size(2) == s.slots;
          if (!ok) break;
          put(address(t.data_ptr()));
          break;
        case 'W':
          ok = on(t, device) && t.scalar_type() == at::kByte && t.dim() == 1 && t.is_contiguous();
          if (!ok) break;
          put(address(t.data_ptr()));
          put(t.numel());
          break;
        case 'K':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.is_contiguous() && t.dim() == 3 && t.size(0) == s.B &&
               t.size(1) == s.kv_heads;
          if (!ok) break;
          put(address(t.data_ptr()));
          break;
        default:
          PyErr_Format(PyExc_ValueError, "call: no format letter %c", *f);
          error = true;
      }
    }
  } catch (...) {  // a tensor without storage and the like: not plainly what the format says
    ok = false;
  }
  if (error) return nullptr;
  if (!ok || a != nargs) Py_RETURN_NONE;
  int st = -1;
  const size_t count = static_cast<size_t>(n);
  Py_BEGIN_ALLOW_THREADS;
  if (std::strcmp(name, "rope_kv_append") == 0)
    st = invoke(&rope_kv_append, entry, out, count);
  else if (std::strcmp(name, "rope_apply") == 0)
    st = invoke(&rope_apply, entry, out, count);
  else if (std::strcmp(name, "paged_tree_attn") == 0)
    st = invoke(&paged_tree_attn, entry, out, count);
  else if (std::strcmp(name, "kv_tree_accept") == 0)
    st = invoke(&kv_tree_accept, entry, out, count);
  else if (std::strcmp(name, "paged_attn_weights") == 0)
    st = invoke(&paged_attn_weights, entry, out, count);
  else if (std::strcmp(name, "kv_evict") == 0)
    st = invoke(&kv_evict, entry, out, count);
  Py_END_ALLOW_THREADS;
  if (st < 0) return PyErr_Format(PyExc_ValueError, "call: %s with %d arguments", name, n);
  return PyLong_FromLong(st);
}

PyMethodDef kMethods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(call)), METH_FASTCALL,
     "call(address, name, format, ...): a C entry point's status, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "A call of the binding in one step.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__marshal(void) { return PyModule_Create(&kModule); }
