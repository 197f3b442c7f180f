// binding.cpp -- the Python binding of the calls whose host time matters: the
// 8-bit cache's write and read, its decode, and the shared-prefix decode run in
// a few microseconds on small inputs, as long as ctypes and checks written in
// Python take (of 10.2 us a call for the write of one token, 6.3 were checks and
// argument conversion). Each function checks its tensors, as the other
// entry points of the package do in Python, and calls the C entry point of the
// same name. The library is the one that the package has loaded: its handle
// comes with every call, so no second copy is linked here.
#include <Python.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>

#include "attn.h"

namespace {

struct Fns {
  decltype(&attn_cache_write_e4m3) write;
  decltype(&attn_cache_read_e4m3) read;
  decltype(&attn_decode_paged_e4m3) decode;
  decltype(&attn_decode_paged_shared) shared;
};

// Entry points of the library `handle` (guarded by the interpreter lock).
const Fns& entries(PyObject* handle) {
  static void* loaded = nullptr;
  static Fns f;
  void* h = PyLong_AsVoidPtr(handle);
  if (h == nullptr) throw std::runtime_error("no library handle");
  if (h != loaded) {
    auto sym = [&](const char* name) {
      void* p = dlsym(h, name);
      if (p == nullptr) throw std::runtime_error(std::string("library lacks ") + name);
      return p;
    };
    Fns n;
    n.write = reinterpret_cast<decltype(n.write)>(sym("attn_cache_write_e4m3"));
    n.read = reinterpret_cast<decltype(n.read)>(sym("attn_cache_read_e4m3"));
    n.decode = reinterpret_cast<decltype(n.decode)>(sym("attn_decode_paged_e4m3"));
    n.shared = reinterpret_cast<decltype(n.shared)>(sym("attn_decode_paged_shared"));
    f = n;
    loaded = h;
  }
  return f;
}

void need(bool ok, const char* what) {
  if (!ok) throw std::invalid_argument(what);
}
const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o), "tensor expected");
  return THPVariable_Unpack(o);
}
int small(int64_t n) {
  need(n <= INT32_MAX, "size beyond int32");
  return static_cast<int>(n);
}
// Every tensor on the current device (kernels launch there).
void on_device(long dev, std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    need(t->is_cuda() && t->get_device() == dev, "tensors must be on the current CUDA device");
}
void contiguous(std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts) need(t->is_contiguous(), "tensors must be contiguous");
}
void int32(std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    need(t->scalar_type() == at::kInt, "tables, offsets and lengths must be int32");
}
void* ptr(const at::Tensor& t) { return t.data_ptr(); }
const int32_t* iptr(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
uint8_t* bptr(const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

// A checked 8-bit cache: caches [num_blocks, h_kv, page, d], scales without d.
void check_cache8(const at::Tensor& kc, const at::Tensor& vc, const at::Tensor& ks,
                  const at::Tensor& vs) {
  need(kc.scalar_type() == at::kFloat8_e4m3fn && vc.scalar_type() == at::kFloat8_e4m3fn &&
           ks.scalar_type() == at::kByte && vs.scalar_type() == at::kByte,
       "caches must be float8_e4m3fn and scales uint8 exponents");
  need(kc.dim() == 4 && vc.sizes() == kc.sizes() && ks.sizes() == kc.sizes().slice(0, 3) &&
           vs.sizes() == ks.sizes(),
       "caches [num_blocks,h_kv,16,d] and scales [num_blocks,h_kv,16] expected");
  contiguous({&kc, &vc, &ks, &vs});
}

template <class F>
PyObject* guarded(F f) {
  try {
    return PyLong_FromLong(f());
  } catch (const std::invalid_argument& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
void args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw std::runtime_error("wrong number of arguments");
}

// (handle, device, stream, k, v, k_cache, v_cache, k_scale, v_scale,
//  block_table, cu_seqlens, seq_lens, write?) -> status
PyObject* cache_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> long {
    args(n, 13);
    const Fns& f = entries(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    void* stream = PyLong_AsVoidPtr(a[2]);
    const at::Tensor &k = tensor(a[3]), &v = tensor(a[4]), &kc = tensor(a[5]), &vc = tensor(a[6]),
                     &ks = tensor(a[7]), &vs = tensor(a[8]), &table = tensor(a[9]),
                     &cu = tensor(a[10]), &lens = tensor(a[11]);
    on_device(dev, {&k, &v, &kc, &vc, &ks, &vs, &table, &cu, &lens});
    check_cache8(kc, vc, ks, vs);
    const auto dt = k.scalar_type();
    need(v.scalar_type() == dt && (dt == at::kBFloat16 || dt == at::kFloat),
         "k, v must share dtype bf16 or fp32");
    need(k.dim() == 3 && v.sizes() == k.sizes() && k.size(1) == kc.size(1) && k.size(2) == kc.size(3),
         "k, v [total,h_kv,d] expected");
    need(k.stride(2) == 1 && v.stride(2) == 1, "k, v must be contiguous in d");
    int32({&table, &cu, &lens});
    need(lens.dim() == 1 && cu.dim() == 1 && cu.size(0) == lens.size(0) + 1 && table.dim() == 2 &&
             table.size(0) == lens.size(0),
         "block_table [B,max_blocks], cu_seqlens [B+1] and seq_lens [B] expected");
    contiguous({&table, &cu, &lens});
    const attn_dtype_t t = dt == at::kBFloat16 ? ATTN_DTYPE_BF16 : ATTN_DTYPE_F32;
    const int B = small(lens.size(0)), total = small(k.size(0)), h_kv = small(kc.size(1)),
              d = small(kc.size(3)), page = small(kc.size(2)), nb = small(kc.size(0)),
              mb = small(table.size(1));
    if (a[12] == Py_True)
      return f.write(ptr(k), ptr(v), k.stride(0), k.stride(1), v.stride(0), v.stride(1), t, iptr(table),
                     iptr(cu), iptr(lens), B, total, h_kv, d, page, nb, mb, ptr(kc), ptr(vc), bptr(ks),
                     bptr(vs), stream);
    return f.read(ptr(kc), ptr(vc), bptr(ks), bptr(vs), iptr(table), iptr(cu), iptr(lens), B, total,
                  h_kv, d, page, nb, mb, ptr(k), ptr(v), k.stride(0), k.stride(1), v.stride(0),
                  v.stride(1), t, stream);
  });
}

// Checks workspace, o and lse (or None) of a decode of q [B, h, d].
float* check_outputs(long dev, const at::Tensor& q, const at::Tensor& ws, const at::Tensor& o,
                     PyObject* lse) {
  on_device(dev, {&ws, &o});
  need(ws.is_contiguous(), "workspace must be contiguous");
  need(o.sizes() == q.sizes() && o.scalar_type() == at::kBFloat16 && o.is_contiguous(),
       "o must be like q");
  if (lse == Py_None) return nullptr;
  const at::Tensor& l = tensor(lse);
  on_device(dev, {&l});
  need(l.dim() == 2 && l.size(0) == q.size(0) && l.size(1) == q.size(1) &&
           l.scalar_type() == at::kFloat && l.is_contiguous(),
       "lse must be contiguous fp32 [B,h]");
  return static_cast<float*>(l.data_ptr());
}
float scale_of(PyObject* scale, int64_t d) {
  if (scale == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  const double s = PyFloat_AsDouble(scale);
  if (s == -1.0 && PyErr_Occurred()) throw std::invalid_argument("scale");
  return static_cast<float>(s);
}
void check_rows(const at::Tensor& q, const at::Tensor& table, const at::Tensor& lens) {
  int32({&table, &lens});
  need(table.dim() == 2 && table.size(0) == q.size(0) && lens.dim() == 1 && lens.size(0) == q.size(0),
       "block_table [B,max_blocks] and seq_lens [B] expected");
  contiguous({&q, &table, &lens});
}

// (handle, device, stream, q, k_cache, v_cache, k_scale, v_scale, block_table,
//  seq_lens, scale, workspace, o, lse) -> status
PyObject* decode_e4m3(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> long {
    args(n, 14);
    const Fns& f = entries(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    void* stream = PyLong_AsVoidPtr(a[2]);
    const at::Tensor &q = tensor(a[3]), &kc = tensor(a[4]), &vc = tensor(a[5]), &ks = tensor(a[6]),
                     &vs = tensor(a[7]), &table = tensor(a[8]), &lens = tensor(a[9]);
    on_device(dev, {&q, &kc, &vc, &ks, &vs, &table, &lens});
    check_cache8(kc, vc, ks, vs);
    need(q.scalar_type() == at::kBFloat16 && q.dim() == 3 && q.size(2) == kc.size(3),
         "q must be bf16 [B,h,d]");
    check_rows(q, table, lens);
    const at::Tensor &ws = tensor(a[11]), &o = tensor(a[12]);
    float* lse = check_outputs(dev, q, ws, o, a[13]);
    return f.decode(ptr(q), ptr(kc), ptr(vc), bptr(ks), bptr(vs), iptr(table), iptr(lens),
                    small(q.size(0)), small(q.size(1)), small(kc.size(1)), small(q.size(2)),
                    small(kc.size(2)), small(kc.size(0)), small(table.size(1)),
                    scale_of(a[10], q.size(2)), ptr(ws), ws.nbytes(), ptr(o), lse, stream);
  });
}

// (handle, device, stream, q, k_cache, v_cache, prefix_table, prefix_len,
//  block_table, seq_lens, scale, workspace, o, lse) -> status
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> long {
    args(n, 14);
    const Fns& f = entries(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    void* stream = PyLong_AsVoidPtr(a[2]);
    const at::Tensor &q = tensor(a[3]), &kc = tensor(a[4]), &vc = tensor(a[5]), &pt = tensor(a[6]),
                     &pl = tensor(a[7]), &table = tensor(a[8]), &lens = tensor(a[9]);
    on_device(dev, {&q, &kc, &vc, &pt, &pl, &table, &lens});
    need(q.scalar_type() == at::kBFloat16 && kc.scalar_type() == at::kBFloat16 &&
             vc.scalar_type() == at::kBFloat16,
         "q and caches must be bf16");
    need(q.dim() == 3 && kc.dim() == 4 && vc.sizes() == kc.sizes() && kc.size(3) == q.size(2),
         "q [B,h,d] and caches [num_blocks,16,h_kv,d] expected");
    int32({&pt, &pl});
    need(pt.dim() == 1 && pl.dim() == 1 && pl.size(0) == 1,
         "prefix_table [max_prefix_blocks] and prefix_len [1] expected");
    check_rows(q, table, lens);
    contiguous({&kc, &vc, &pt, &pl});
    const at::Tensor &ws = tensor(a[11]), &o = tensor(a[12]);
    float* lse = check_outputs(dev, q, ws, o, a[13]);
    return f.shared(ptr(q), ptr(kc), ptr(vc), iptr(pt), iptr(pl), iptr(table), iptr(lens),
                    small(q.size(0)), small(q.size(1)), small(kc.size(2)), small(q.size(2)),
                    small(kc.size(1)), small(kc.size(0)), small(pt.size(0)), small(table.size(1)),
                    scale_of(a[10], q.size(2)), ptr(ws), ws.nbytes(), ptr(o), lse, stream);
  });
}

PyMethodDef methods[] = {
    {"cache_tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_tokens)),
     METH_FASTCALL, "attn_cache_write_e4m3 and attn_cache_read_e4m3"},
    {"decode_e4m3", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_e4m3)), METH_FASTCALL,
     "attn_decode_paged_e4m3"},
    {"decode_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_shared)),
     METH_FASTCALL, "attn_decode_paged_shared"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr,
                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
