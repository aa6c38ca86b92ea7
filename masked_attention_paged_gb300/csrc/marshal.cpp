// marshal.cpp -- a call of the binding in one step.
//
// A call of a few microseconds on the GPU is bound by the host: in Python, reading
// the pointer, type, shape and strides of a dozen tensors, checking them and
// converting them for the C entry takes longer than the launch.  call(address,
// name, format, ...) does that for a whole call on the current device and returns
// the entry's status, or None (and calls nothing) when anything is not plainly as the format
// says; the Python code then goes through its own checks, which word the refusal
// (or take the rarer form).  Results that the caller has no tensor for are made here, of the
// current stream's memory, and returned behind the status, (status, result, ...).  Nothing is
// kept between calls.
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
//   E  as l, or True: a result of y's rows -> pointer or null
//   A  f32 [blocks, Hkv, 16] of the cache -> pointer
//   K  int32, contiguous [B, Hkv, n]     -> pointer
//   O  as Y, of any type, or None: a result like y, contiguous -> attn_tensor
//   p  tensor, bf16 or f32, 3-D          -> attn_tensor; B, T and D are its sizes
//   P  as p, of its sizes and type, or None -> attn_tensor or null
//   u  f32 [B, T] rows                   -> pointer, row stride
//   k  int32, contiguous [B, T], or None: a result -> pointer
//   i  int32 vector of B, or None: a result -> pointer
//   e  four tensors: an e4m3 cache and its scales -> attn_kv_cache_f8
//   L  a list of tensors with as many blocks as Z says -> their number, attn_pool_tensor[]
//   Z  int32 vector of a pool's blocks   -> pointer, their number
//   t  table, rows apart, that sets B or has B rows -> pointer, row stride, columns
//   U  int32, one element, or None: a result -> pointer
//   W  a workspace's bytes               -> pointer, their number
//   S  a stream handle, or None          -> itself, or the current stream
//   =  an int or a float                 -> itself
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <type_traits>
#include <vector>
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
  int64_t pool = -1;        // blocks of the pool
  at::ScalarType type = at::kBFloat16;
  bool one_token = false;
};

bool on(const at::Tensor& t, int64_t device) { return t.is_cuda() && t.get_device() == device; }

// a 4-D tensor, or (insert) 3-D rows with a dimension of one before the last; or (three) 3-D as it is
bool describe(const at::Tensor& t, int64_t device, bool insert, attn_tensor* d, bool three = false) {
  if (!on(t, device)) return false;
  const auto type = t.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) return false;
  const int64_t n = t.dim();
  if (n != (insert || three ? 3 : 4)) return false;
  std::memset(d, 0, sizeof(*d));
  d->data = t.data_ptr();
  d->dtype = type == at::kBFloat16 ? ATTN_BF16 : ATTN_F32;
  d->ndim = three ? 3 : 4;
  for (int i = 0, k = 0; i < d->ndim; ++i) {
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
  attn_kv_cache_f8 cache_f8;
  std::vector<attn_pool_tensor> pool;
  int n = 0, n_tensors = 0;
  Py_ssize_t a = 3;
  Sizes s;
  constexpr int kMostMade = 4;
  at::Tensor made[kMostMade];
  int n_made = 0;
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
      if (o == Py_None && (*f == 'o' || *f == 'n' || *f == 'l' || *f == 'E' || *f == 'P')) {
        put(0);
        continue;
      }
      const bool makes = (o == Py_None && (*f == 'k' || *f == 'i' || *f == 'U' || *f == 'O')) ||
                         (o == Py_True && *f == 'E');
      if (makes) {
        if (n_made == kMostMade || n_tensors == 8 || (*f != 'U' && s.B < 0)) {
          ok = false;
          break;
        }
        const int64_t sizes[4] = {s.B, *f == 'k' ? s.T : s.H, s.one_token ? s.D : s.T, s.D};
        const int64_t one = 1;
        const int dims = *f == 'k' ? 2 : (*f == 'i' || *f == 'U' ? 1 : (*f == 'E' ? 3 : 4) - (s.one_token ? 1 : 0));
        const at::ScalarType type = *f == 'O' ? s.type : (*f == 'E' ? at::kFloat : at::kInt);
        at::Tensor& x = made[n_made++];
        x = at::empty(*f == 'U' ? at::IntArrayRef(&one, 1) : at::IntArrayRef(sizes, dims),
                      at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
        if (*f == 'O') {
          ok = describe(x, device, s.one_token, &tensors[n_tensors]);
          put(address(&tensors[n_tensors++]));
        } else {
          put(address(x.data_ptr()));
        }
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
      if (*f == 'L') {
        const bool list = PyList_Check(o);
        const Py_ssize_t count = list ? PyList_GET_SIZE(o) : (PyTuple_Check(o) ? PyTuple_GET_SIZE(o) : -1);
        ok = count >= 0 && count <= 4096;
        pool.resize(ok ? static_cast<size_t>(count) : 0);
        for (Py_ssize_t i = 0; ok && i < count; ++i) {
          PyObject* x = list ? PyList_GET_ITEM(o, i) : PyTuple_GET_ITEM(o, i);
          ok = THPVariable_Check(x);
          if (!ok) break;
          const at::Tensor& c = THPVariable_Unpack(x);
          ok = on(c, device) && c.dim() >= 1 && c.size(0) > 0 && c.is_contiguous() &&
               (s.pool < 0 || s.pool == c.size(0));
          if (!ok) break;
          s.pool = c.size(0);
          pool[i].data = c.data_ptr();
          pool[i].block_bytes = c.numel() / c.size(0) * static_cast<int64_t>(c.element_size());
        }
        put(count);
        put(address(pool.data()));
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
        case 'O':
        case 'o': {
          if (n_tensors == 8) {
            ok = false;
            break;
          }
          attn_tensor& d = tensors[n_tensors];
          const bool first = n_tensors == 0;
          const bool insert = (*f == 'y' || *f == 'Y' || *f == 'O') && (first ? t.dim() == 3 : s.one_token);
          ok = describe(t, device, insert, &d);
          if (*f == 'X' || *f == 'Y' || *f == 'O')
            ok = ok && d.shape[0] == s.B && d.shape[1] == s.H && d.shape[2] == s.T && d.shape[3] == s.D &&
                 (*f != 'Y' || t.scalar_type() == s.type);
          if (!ok) break;
          if (first) {
            ok = s.B < 0 || s.B == d.shape[0];  // (a vector before it may have said)
            if (!ok) break;
            s.B = d.shape[0], s.H = d.shape[1], s.T = d.shape[2], s.D = d.shape[3];
            s.type = t.scalar_type();
            s.one_token = insert;
          }
          ++n_tensors;
          put(address(&d));
          break;
        }
        case 'p':
        case 'P': {
          if (n_tensors == 8) {
            ok = false;
            break;
          }
          attn_tensor& d = tensors[n_tensors];
          ok = describe(t, device, false, &d, true);
          if (!ok) break;
          if (*f == 'p') {
            s.B = d.shape[0], s.T = d.shape[1], s.D = d.shape[2];
            s.type = t.scalar_type();
          }
          ok = d.shape[0] == s.B && d.shape[1] == s.T && d.shape[2] == s.D && t.scalar_type() == s.type;
          ++n_tensors;
          put(address(&d));
          break;
        }
        case 'u':
          ok = on(t, device) && t.scalar_type() == at::kFloat && t.dim() == 2 && t.size(0) == s.B && t.size(1) == s.T &&
               (s.T <= 1 || t.stride(1) == 1);
          if (!ok) break;
          put(address(t.data_ptr()));
          put(t.stride(0));
          break;
        case 'k':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.is_contiguous() && t.dim() == 2 && t.size(0) == s.B &&
               t.size(1) == s.T;
          if (!ok) break;
          put(address(t.data_ptr()));
          break;
        case 'Z':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 1 && t.is_contiguous() &&
               (s.pool < 0 || s.pool == t.size(0));
          if (!ok) break;
          put(address(t.data_ptr()));
          put(t.size(0));
          break;
        case 't':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 2 && t.stride(1) == 1 &&
               t.stride(0) >= t.size(1) && (s.B < 0 || s.B == t.size(0));
          if (!ok) break;
          s.B = t.size(0);
          put(address(t.data_ptr()));
          put(t.stride(0));
          put(t.size(1));
          break;
        case 'U':
          ok = on(t, device) && t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == 1;
          if (!ok) break;
          put(address(t.data_ptr()));
          break;
        case 'e': {
          const at::Tensor* c[4] = {&t, nullptr, nullptr, nullptr};
          for (int i = 1; ok && i < 4; ++i) {
            ok = a < nargs && THPVariable_Check(args[a]);
            if (ok) c[i] = &THPVariable_Unpack(args[a++]);
          }
          if (!ok) break;
          for (int i = 0; i < 4; ++i) ok = ok && on(*c[i], device) && c[i]->is_contiguous();
          ok = ok && t.dim() == 4 && t.sizes() == c[1]->sizes() && t.scalar_type() == at::kFloat8_e4m3fn &&
               c[1]->scalar_type() == at::kFloat8_e4m3fn;
          for (int i = 2; i < 4; ++i)
            ok = ok && c[i]->scalar_type() == at::kFloat && c[i]->dim() == 2 && c[i]->size(0) == t.size(0) &&
                 c[i]->size(1) == t.size(1);
          if (!ok) break;
          std::memset(&cache_f8, 0, sizeof(cache_f8));
          cache_f8.k = t.data_ptr();
          cache_f8.v = c[1]->data_ptr();
          cache_f8.k_scale = static_cast<float*>(c[2]->data_ptr());
          cache_f8.v_scale = static_cast<float*>(c[3]->data_ptr());
          cache_f8.num_blocks = t.size(0);
          cache_f8.num_kv_heads = static_cast<int32_t>(t.size(1));
          cache_f8.block_size = static_cast<int32_t>(t.size(2));
          cache_f8.head_dim = static_cast<int32_t>(t.size(3));
          put(address(&cache_f8));
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
        case 'i':
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
        case 'E':
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
  else if (std::strcmp(name, "draft_verify") == 0)
    st = invoke(&draft_verify, entry, out, count);
  else if (std::strcmp(name, "kv_free") == 0)
    st = invoke(&kv_free, entry, out, count);
  else if (std::strcmp(name, "kv_reserve") == 0)
    st = invoke(&kv_reserve, entry, out, count);
  else if (std::strcmp(name, "kv_fork") == 0)
    st = invoke(&kv_fork, entry, out, count);
  else if (std::strcmp(name, "kv_compact") == 0)
    st = invoke(&kv_compact, entry, out, count);
  else if (std::strcmp(name, "kv_append_f8") == 0)
    st = invoke(&kv_append_f8, entry, out, count);
  else if (std::strcmp(name, "paged_attn_f8") == 0)
    st = invoke(&paged_attn_f8, entry, out, count);
  Py_END_ALLOW_THREADS;
  if (st < 0) return PyErr_Format(PyExc_ValueError, "call: %s with %d arguments", name, n);
  if (n_made == 0 || st != 0) return PyLong_FromLong(st);
  PyObject* all = PyTuple_New(1 + n_made);
  if (all == nullptr) return nullptr;
  PyTuple_SET_ITEM(all, 0, PyLong_FromLong(st));
  for (int i = 0; i < n_made; ++i) PyTuple_SET_ITEM(all, 1 + i, THPVariable_Wrap(made[i]));
  return all;
}

PyMethodDef kMethods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(call)), METH_FASTCALL,
     "call(address, name, format, ...): a C entry point's status, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "A call of the binding in one step.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__marshal(void) { return PyModule_Create(&kModule); }
