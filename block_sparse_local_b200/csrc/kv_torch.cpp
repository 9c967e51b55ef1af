// kv_torch.cpp - argument marshalling of the paged-cache calls for Python, in
// C++: a decoding step makes two of these calls per layer, with a dozen
// tensors each, and reading their shapes and strides from Python took longer
// (about 20 us a call) than the kernels.  The checks and messages are those that
// a Python binding of the two C entry points would make; nothing else is here.
#include <torch/extension.h>
#include <torch/csrc/autograd/python_variable.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cstdint>

namespace {

// The torch and Python versions whose interface this file was compiled against;
// read from the file before it is loaded.
__attribute__((used)) const char kBuiltFor[] = KV_TORCH_BUILT_FOR;

using AppendFn = int (*)(const void*, const void*, const void*, void*, const int64_t*, void*,
                         void*, float*, float*, const int64_t*, const int*, int, const int*,
                         const int*, const float*, int, int, int, int, int, int, int, int, int,
                         int, void*);
using AttentionFn = int (*)(const void*, void*, float*, const int64_t*, const void*, const void*,
                            const float*, const float*, const int64_t*, const int*, int,
                            const int*, const int*, int, void*, size_t, int, int, int, int, int,
                            int, int, int, void*);
using WorkspaceFn = int64_t (*)(int, int, int, int);

AppendFn g_append = nullptr;
AttentionFn g_attention = nullptr;
WorkspaceFn g_workspace = nullptr;
PyObject* g_error = nullptr;          // StaError(code, where)

struct Refused {};                    // a Python error is set

[[noreturn]] void refuse(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  throw Refused{};
}

struct Range {                        // an NVTX range per public call, as the others have
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw Refused{};
  }
  return THPVariable_Unpack(o);
}

// None: an undefined tensor.
at::Tensor optional(PyObject* o, const char* name) {
  return o == Py_None ? at::Tensor() : tensor(o, name);
}

void* pointer(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

struct Cache {
  int64_t B, S, hkv, d, blocks, block, width;
  int type;
  int64_t strides[4];
};

// A dimension of one element never moves the pointer: its stride is free.
void put_strides(int64_t* to, const at::Tensor& t) {
  for (int i = 0; i < 3; ++i) to[i] = t.size(i) > 1 ? t.stride(i) : 0;
}

int fits(int64_t n) {
  if (n < 0 || n > 0x7fffffff) refuse("a size is beyond 32 bits");
  return static_cast<int>(n);
}

// What the two calls share.  tokens: the call's [B, heads, S, d] tensors.
Cache check(const at::Tensor* const* tokens, int count, int64_t hq, const at::Tensor& kc,
            const at::Tensor& vc, const at::Tensor& table, const at::Tensor& lens,
            const at::Tensor& ks, const at::Tensor& vs, const at::Tensor& new_lens) {
  Cache c;
  const at::Tensor& t0 = *tokens[0];
  c.B = t0.size(0);
  c.S = t0.size(2);
  c.d = t0.size(3);
  const auto dtype = kc.scalar_type();
  if ((dtype != at::kBFloat16 && dtype != at::kFloat8_e4m3fn) || vc.scalar_type() != dtype)
    refuse("caches must both be torch.bfloat16 or torch.float8_e4m3fn");
  c.type = dtype == at::kBFloat16 ? 0 : 1;
  if (kc.dim() != 4 || vc.sizes() != kc.sizes() || kc.size(3) != c.d)
    refuse("caches must be [num_blocks, kv heads, block, d], alike");
  c.blocks = kc.size(0);
  c.hkv = kc.size(1);
  c.block = kc.size(2);
  if (kc.stride(3) != 1 || vc.stride(3) != 1 || kc.stride(2) != c.d || vc.stride(2) != c.d)
    refuse("the rows of a cache block must be contiguous");
  c.strides[0] = kc.stride(0);
  c.strides[1] = kc.stride(1);
  c.strides[2] = vc.stride(0);
  c.strides[3] = vc.stride(1);
  for (int i = 0; i < count; ++i) {
    const at::Tensor& t = *tokens[i];
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 4 || t.size(0) != c.B ||
        t.size(2) != c.S || t.size(3) != c.d || t.stride(3) != 1)
      refuse("token tensors must be bf16 [B, heads, S, d], d contiguous");
  }
  const bool f8 = c.type == 1;
  if (ks.defined() != f8 || vs.defined() != f8)
    refuse("an e4m3 cache has k_scale and v_scale, a bf16 cache none");
  for (const at::Tensor* t : {&ks, &vs})
    if (t->defined() && (t->scalar_type() != at::kFloat || t->dim() != 2 ||
                         t->size(0) != c.blocks || t->size(1) != c.hkv || !t->is_contiguous()))
      refuse("scales must be contiguous fp32 [num_blocks, kv heads]");
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != c.B ||
      !table.is_contiguous())
    refuse("block_table must be contiguous int32 [B, width]");
  c.width = table.size(1);
  for (const at::Tensor* t : {&lens, &new_lens})
    if (t->defined() && (t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != c.B ||
                         !t->is_contiguous()))
      refuse("seq_lens and new_lens must be contiguous int32 [B]");
  if (!kc.is_cuda()) refuse("tensors must be CUDA tensors");
  const auto device = kc.device();
  auto same = [&](const at::Tensor& t) {
    if (t.defined() && t.device() != device) refuse("tensors must be on one CUDA device");
  };
  for (int i = 0; i < count; ++i) same(*tokens[i]);
  for (const at::Tensor* t : {&vc, &ks, &vs, &table, &lens, &new_lens}) same(*t);
  if (c.hkv < 1 || hq % c.hkv) refuse("query heads must be a multiple of the kv heads");
  return c;
}

void check_status(int code, const char* where) {
  if (code == 0) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", code, where);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}

// Positions end below 2^31: a longer window is none.
int as_window(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  if (v < 0) refuse("window must be a number of tokens, or 0 for all");
  return static_cast<int>(std::min<long long>(v, 0x7fffffff));
}

// append(k, v, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale,
//        new_lens, q, rope, interleaved, q_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 13) refuse("13 arguments");
    Range range("sta.kv_cache_append");
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const at::Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
    const at::Tensor &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "seq_lens");
    const at::Tensor ks = optional(a[6], "k_scale"), vs = optional(a[7], "v_scale");
    const at::Tensor new_lens = optional(a[8], "new_lens"), q = optional(a[9], "q");
    const at::Tensor rope = optional(a[10], "rope");
    at::Tensor q_out = optional(a[12], "q_out");
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) throw Refused{};
    if (k.dim() != 4 || v.sizes() != k.sizes())
      refuse("k and v must be [B, kv heads, S, d], alike");
    if (q.defined() && !rope.defined()) refuse("queries are only rotated: q needs rope");
    if (!q.defined() && q_out.defined()) refuse("q_out needs q");
    if (q.defined() && q.dim() != 4) refuse("q must be [B, heads, S, d]");
    if (q.defined() && !q_out.defined()) q_out = at::empty_like(q);
    const at::Tensor* tokens[4] = {&k, &v, &q, &q_out};
    const int64_t hq = q.defined() ? q.size(1) : k.size(1);
    const Cache c = check(tokens, q.defined() ? 4 : 2, hq, kc, vc, table, lens, ks, vs, new_lens);
    if (k.size(1) != c.hkv || (q.defined() && q_out.sizes() != q.sizes()))
      refuse("k, v must have the cache's heads, q_out the shape of q");
    int64_t rows = 0;
    if (rope.defined()) {
      if (rope.scalar_type() != at::kFloat || rope.dim() != 2 || rope.size(1) != c.d ||
          !rope.is_contiguous() || rope.device() != kc.device())
        refuse("rope must be a contiguous fp32 [positions, d] CUDA table");
      rows = rope.size(0);
      if (rows < c.width * c.block)
        refuse("rope must cover block_table's width * block positions");
    }
    if (c.B > 0 && c.S > 0) {
      int64_t st[12] = {};
      put_strides(st, k);
      put_strides(st + 3, v);
      if (q.defined()) {
        put_strides(st + 6, q);
        put_strides(st + 9, q_out);
      }
      const c10::cuda::CUDAGuard guard(kc.device());
      check_status(
          g_append(k.data_ptr(), v.data_ptr(), pointer(q), pointer(q_out), st, kc.data_ptr(),
                   vc.data_ptr(), static_cast<float*>(pointer(ks)),
                   static_cast<float*>(pointer(vs)), c.strides,
                   static_cast<const int*>(table.data_ptr()), fits(c.width),
                   static_cast<const int*>(lens.data_ptr()),
                   static_cast<const int*>(pointer(new_lens)),
                   static_cast<const float*>(pointer(rope)),
                   static_cast<int>(std::min<int64_t>(rows, 0x7fffffff)), interleaved, fits(c.B),
                   fits(c.S), fits(hq), fits(c.hkv), fits(c.d), fits(c.blocks), fits(c.block),
                   c.type, c10::cuda::getCurrentCUDAStream().stream()),
          "sta_kv_append");
    }
    if (!q.defined()) Py_RETURN_NONE;
    if (a[12] != Py_None) return Py_NewRef(a[12]);
    return THPVariable_Wrap(q_out);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// attention(q, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale,
//           new_lens, window, out, return_lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 11) refuse("11 arguments");
    Range range("sta.kv_cache_attention");
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
    const at::Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
    const at::Tensor ks = optional(a[5], "k_scale"), vs = optional(a[6], "v_scale");
    const at::Tensor new_lens = optional(a[7], "new_lens");
    const int window = as_window(a[8]);
    at::Tensor out = optional(a[9], "out");
    const int want_lse = PyObject_IsTrue(a[10]);
    if (want_lse < 0) throw Refused{};
    if (q.dim() != 4) refuse("q must be [B, heads, S, d]");
    if (!out.defined()) out = at::empty(q.sizes(), q.options());
    else if (out.sizes() != q.sizes()) refuse("out must have the shape of q");
    const at::Tensor* tokens[2] = {&q, &out};
    const int64_t hq = q.size(1);
    const Cache c = check(tokens, 2, hq, kc, vc, table, lens, ks, vs, new_lens);
    at::Tensor lse;
    if (want_lse) lse = at::empty({c.B, hq, c.S}, q.options().dtype(at::kFloat));
    if (c.B > 0 && c.S > 0) {
      int64_t st[6];
      put_strides(st, q);
      put_strides(st + 3, out);
      const c10::cuda::CUDAGuard guard(kc.device());
      // the caller's allocator owns the workspace: calls on other streams, and
      // captured graphs, each get their own
      const int64_t bytes =
          std::max<int64_t>(g_workspace(fits(c.S), fits(hq), fits(c.hkv), fits(c.d)), 1);
      const at::Tensor ws = at::empty({bytes}, q.options().dtype(at::kByte));
      check_status(
          g_attention(q.data_ptr(), out.data_ptr(), static_cast<float*>(pointer(lse)), st,
                      kc.data_ptr(), vc.data_ptr(), static_cast<const float*>(pointer(ks)),
                      static_cast<const float*>(pointer(vs)), c.strides,
                      static_cast<const int*>(table.data_ptr()), fits(c.width),
                      static_cast<const int*>(lens.data_ptr()),
                      static_cast<const int*>(pointer(new_lens)), window, ws.data_ptr(),
                      static_cast<size_t>(bytes), fits(c.B), fits(c.S), fits(hq), fits(c.hkv),
                      fits(c.d), fits(c.blocks), fits(c.block), c.type,
                      c10::cuda::getCurrentCUDAStream().stream()),
          "sta_kv_attention");
    }
    PyObject* o = a[9] != Py_None ? Py_NewRef(a[9]) : THPVariable_Wrap(out);
    if (!want_lse || o == nullptr) return o;
    return Py_BuildValue("(NN)", o, THPVariable_Wrap(lse));
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// connect(append, attention, workspace, error): addresses of the C entry points
// of the loaded library, and the exception for their status codes.
PyObject* connect(PyObject*, PyObject* args) {
  unsigned long long f[3];
  PyObject* error;
  if (!PyArg_ParseTuple(args, "KKKO", &f[0], &f[1], &f[2], &error)) return nullptr;
  g_append = reinterpret_cast<AppendFn>(f[0]);
  g_attention = reinterpret_cast<AttentionFn>(f[1]);
  g_workspace = reinterpret_cast<WorkspaceFn>(f[2]);
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL,
     nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)),
     METH_FASTCALL, nullptr},
    {"connect", connect, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kv_torch", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__kv_torch() { return PyModule_Create(&kModule); }
