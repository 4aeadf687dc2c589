// The paged-cache calls' way from Python: checks of the tensors, outputs and
// workspaces, the device and its stream, then the C ABI (bitlinear.h). These
// calls are made for every layer of every step, and their kernels take a few
// microseconds: marshalling in Python took 9 us a call.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "../../include/bitlinear.h"

namespace {

using at::Tensor;

PyObject* g_fail = nullptr;    // _check(rc): raises for rc != 0
PyObject* g_status = nullptr;  // status_buffer(device index)

// The library's functions, from the handle that _lib.py holds (linking to it
// would bind this module's C++ runtime to the copy that it carries).
struct Abi {
  decltype(&::kv_append_3bit) kv_append_3bit;
  decltype(&::kv_pages_copy) kv_pages_copy;
  decltype(&::kv_pages_fork) kv_pages_fork;
  decltype(&::kv_pages_free) kv_pages_free;
  decltype(&::kv_pages_grow) kv_pages_grow;
  decltype(&::kv_pages_compact) kv_pages_compact;
  decltype(&::kv_attention_3bit_paged_workspace) kv_attention_3bit_paged_workspace;
  decltype(&::kv_attention_3bit_paged) kv_attention_3bit_paged;
  decltype(&::kv_page_block_bytes) kv_page_block_bytes;
} g_abi;

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// None: an undefined tensor
const Tensor& maybe(PyObject* o, const char* name) {
  static const Tensor none;
  return o == Py_None ? none : tensor(o, name);
}

template <typename T = void>
T* ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

void need_bf16(const Tensor& t, const char* name, int dim) {
  const auto s = t.scalar_type();
  TORCH_CHECK_VALUE(s == at::kBFloat16 || s == at::kShort || s == at::kUInt16, name, ": dtype ", s, ", expected bf16 or 16-bit patterns of it");
  TORCH_CHECK_VALUE(t.dim() == dim, name, ": ", t.dim(), "-D, expected ", dim, "-D");
}

void need_ints(const Tensor& t, const char* name, int64_t size = -1) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt, name, ": dtype ", t.scalar_type(), ", expected int32");
  TORCH_CHECK_VALUE(t.dim() == 1 && t.is_contiguous(), name, ": must be contiguous and 1-D");
  TORCH_CHECK_VALUE(size < 0 || t.numel() == size, name, ": ", t.numel(), " values, expected ", size);
}

struct Pool {
  int64_t L, n_pages, H, D, block, C4;
  int64_t bytes() const { return H * block; }
  int64_t bytes4() const { return H * C4 * D; }
};

// A pool [L x] n_pages x H x block and its 4-bit rows.
Pool need_pool(const Tensor& pages, const Tensor& codes4, bool layers) {
  const int64_t d = pages.dim();
  TORCH_CHECK_VALUE(pages.scalar_type() == at::kByte && (d == 3 || (layers && d == 4)) && pages.is_contiguous(),
                    "pages: must be a contiguous uint8 tensor [", layers ? "L x " : "", "n_pages x H x block]");
  Pool p{d == 4 ? pages.size(0) : 1, pages.size(d - 3), pages.size(d - 2), 0, pages.size(d - 1), 0};
  for (const int64_t D : {64, 128, 256})
    if (g_abi.kv_page_block_bytes(D) == p.block) p.D = D;
  TORCH_CHECK_VALUE(p.D, "pages: blocks of ", p.block, " bytes, expected kv_page_block_bytes(D)");
  if (!codes4.defined()) return p;
  TORCH_CHECK_VALUE(codes4.scalar_type() == at::kByte && codes4.is_contiguous(), "codes4: must be a contiguous uint8 tensor");
  bool same = codes4.dim() == d + 1 && codes4.size(d) == p.D;
  for (int64_t i = 0; same && i < d - 1; ++i) same = codes4.size(i) == pages.size(i);
  TORCH_CHECK_VALUE(same, "codes4: shape ", codes4.sizes(), ", expected that of pages with (rows4, ", p.D, ") for the block");
  p.C4 = codes4.size(d - 1);
  return p;
}

struct Tables {
  int64_t R, W, ld;
};

Tables need_tables(const Tensor& tables, const Tensor& lens) {
  TORCH_CHECK_VALUE(tables.scalar_type() == at::kInt && tables.dim() == 2 && (tables.size(1) <= 1 || tables.stride(1) == 1),
                    "tables: must be an int32 tensor [R x W] with contiguous rows");
  const int64_t R = tables.size(0), W = tables.size(1);
  need_ints(lens, "lens", R);
  return {R, W, R > 1 ? tables.stride(0) : std::max<int64_t>(W, 1)};
}

// The device of a call's tensors, its status word and its stream. Memory taken
// while this lives belongs to that stream.
class Call {
 public:
  Call(const Tensor& lead, PyObject* status, PyObject* stream, std::initializer_list<std::pair<const char*, const Tensor*>> others) {
    const Tensor& st = maybe(status, "status");
    TORCH_CHECK_VALUE(!st.defined() || (st.scalar_type() == at::kInt && st.numel() > 0), "status: must be an int32 tensor of one value");
    TORCH_CHECK_VALUE(lead.is_cuda(), "expected a CUDA tensor");
    const at::Device dev = lead.device();
    for (const auto& [name, t] : others) on(dev, name, *t);
    on(dev, "status", st);
    if (st.defined()) {
      status_ = ptr<int>(st);
    } else {
      PyObject* own = PyObject_CallFunction(g_status, "i", static_cast<int>(dev.index()));
      if (own == nullptr) throw python_error();
      status_ = ptr<int>(tensor(own, "status"));  // kept by status_buffer()
      Py_DECREF(own);
    }
    if (stream == Py_None) {
      guard_.emplace(dev);
      stream_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    } else {
      const c10::cuda::CUDAStream s = c10::cuda::CUDAStream::unpack3(number(stream, "stream_id"), static_cast<c10::DeviceIndex>(number(stream, "device_index")),
                                                                     static_cast<c10::DeviceType>(number(stream, "device_type")));
      TORCH_CHECK_VALUE(s.device() == dev, "a stream of ", s.device(), " for tensors of ", dev);
      stream_guard_.emplace(s);
      stream_ = s.stream();
    }
  }
  template <typename F, typename... A>
  bool run(F fn, A... args) {  // false: a Python error is set
    int rc;
    {
      NoGil nogil;
      rc = fn(args..., status_, reinterpret_cast<bitlinear_stream_t>(stream_));
    }
    if (rc == BITLINEAR_OK) return true;
    Py_XDECREF(PyObject_CallFunction(g_fail, "i", rc));
    return false;
  }

 private:
  struct NoGil {
    PyThreadState* s = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(s); }
  };
  static void on(const at::Device& dev, const char* name, const Tensor& t) {
    TORCH_CHECK_VALUE(!t.defined() || t.device() == dev, name, ": on ", t.device(), ", expected ", dev);
  }
  static int64_t number(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    if (v == nullptr) throw python_error();
    const int64_t n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) throw python_error();
    return n;
  }
  int* status_;
  cudaStream_t stream_;
  std::optional<c10::cuda::CUDAGuard> guard_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_guard_;
};

void arguments(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

#define BLT_CALL(NAME) PyObject* NAME(PyObject*, PyObject* const* a, Py_ssize_t n_args)

BLT_CALL(append) {
  HANDLE_TH_ERRORS
  arguments(n_args, 8);
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"), &pages = tensor(a[3], "pages");
  const Tensor &row4 = maybe(a[4], "row4"), &codes4 = maybe(a[5], "codes4");
  const Pool p = need_pool(pages, codes4, false);
  for (const auto& [name, t] : {std::pair{"k", &k}, std::pair{"v", &v}}) {
    need_bf16(*t, name, 3);
    TORCH_CHECK_VALUE(t->size(1) == p.H && t->size(2) == p.D && (t->numel() == 0 || (t->stride(2) == 1 && (p.H == 1 || t->stride(1) == p.D))),
                      name, ": shape ", t->sizes(), ", strides ", t->strides(), ", expected [n x ", p.H, " x ", p.D, "] with contiguous heads");
  }
  const int64_t n = k.size(0);
  TORCH_CHECK_VALUE(v.size(0) == n, "v: ", v.size(0), " tokens, k has ", n);
  need_ints(slots, "slots", n);
  if (row4.defined()) need_ints(row4, "row4", n);
  Call call(pages, a[6], a[7], {{"k", &k}, {"v", &v}, {"slots", &slots}, {"row4", &row4}, {"codes4", &codes4}});
  const int64_t row = p.H * p.D;
  if (!call.run(g_abi.kv_append_3bit, ptr<uint16_t>(k), n > 1 ? k.stride(0) : row, ptr<uint16_t>(v), n > 1 ? v.stride(0) : row, n, p.H, p.D,
                ptr<int32_t>(slots), ptr<int32_t>(row4), ptr<uint8_t>(pages), p.n_pages, ptr<uint8_t>(codes4), p.C4))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

BLT_CALL(copy) {
  HANDLE_TH_ERRORS
  arguments(n_args, 6);
  const Tensor &pages = tensor(a[0], "pages"), &src = tensor(a[1], "src"), &dst = tensor(a[2], "dst"), &codes4 = maybe(a[3], "codes4");
  const Pool p = need_pool(pages, codes4, true);
  need_ints(src, "src");
  need_ints(dst, "dst", src.numel());
  Call call(pages, a[4], a[5], {{"src", &src}, {"dst", &dst}, {"codes4", &codes4}});
  if (!call.run(g_abi.kv_pages_copy, ptr<uint8_t>(pages), p.bytes(), ptr<uint8_t>(codes4), p.bytes4(), p.L, p.n_pages, ptr<int32_t>(src),
                ptr<int32_t>(dst), src.numel()))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

BLT_CALL(fork) {
  HANDLE_TH_ERRORS
  arguments(n_args, 7);
  const Tensor &tables = tensor(a[0], "tables"), &lens = tensor(a[1], "lens"), &refs = tensor(a[2], "refs");
  const Tensor &parents = tensor(a[3], "parents"), &children = tensor(a[4], "children");
  const Tables t = need_tables(tables, lens);
  need_ints(refs, "refs");
  need_ints(parents, "parents");
  need_ints(children, "children", parents.numel());
  Call call(tables, a[5], a[6], {{"lens", &lens}, {"refs", &refs}, {"parents", &parents}, {"children", &children}});
  if (!call.run(g_abi.kv_pages_fork, ptr<int32_t>(tables), t.R, t.W, t.ld, ptr<int32_t>(lens), ptr<int32_t>(refs), refs.numel(),
                ptr<int32_t>(parents), ptr<int32_t>(children), parents.numel()))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

BLT_CALL(release) {
  HANDLE_TH_ERRORS
  arguments(n_args, 7);
  const Tensor &tables = tensor(a[0], "tables"), &lens = tensor(a[1], "lens"), &refs = tensor(a[2], "refs");
  const Tensor &rows = tensor(a[3], "rows"), &keep = maybe(a[4], "keep");
  const Tables t = need_tables(tables, lens);
  need_ints(refs, "refs");
  need_ints(rows, "rows");
  if (keep.defined()) need_ints(keep, "keep", rows.numel());
  Call call(tables, a[5], a[6], {{"lens", &lens}, {"refs", &refs}, {"rows", &rows}, {"keep", &keep}});
  if (!call.run(g_abi.kv_pages_free, ptr<int32_t>(tables), t.R, t.W, t.ld, ptr<int32_t>(lens), ptr<int32_t>(refs), refs.numel(), ptr<int32_t>(rows),
                ptr<int32_t>(keep), rows.numel()))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

BLT_CALL(grow) {
  HANDLE_TH_ERRORS
  arguments(n_args, 10);
  const Tensor &pages = tensor(a[0], "pages"), &tables = tensor(a[1], "tables"), &lens = tensor(a[2], "lens"), &refs = tensor(a[3], "refs");
  const Tensor &rows = tensor(a[4], "rows"), &n_new = tensor(a[5], "n_new"), &codes4 = maybe(a[7], "codes4");
  const int64_t max_new = PyLong_AsLongLong(a[6]);
  if (max_new == -1 && PyErr_Occurred()) throw python_error();
  const Pool p = need_pool(pages, codes4, true);
  const Tables t = need_tables(tables, lens);
  need_ints(refs, "refs", p.n_pages);
  need_ints(rows, "rows");
  const int64_t n = rows.numel();
  need_ints(n_new, "n_new", n);
  TORCH_CHECK_VALUE(max_new >= 0, "max_new = ", max_new);
  Call call(pages, a[8], a[9], {{"tables", &tables}, {"lens", &lens}, {"refs", &refs}, {"rows", &rows}, {"n_new", &n_new}, {"codes4", &codes4}});
  const Tensor slots = at::empty({n, max_new}, lens.options()), work = at::empty({2 * n}, lens.options());
  if (!call.run(g_abi.kv_pages_grow, ptr<uint8_t>(pages), p.bytes(), ptr<uint8_t>(codes4), p.bytes4(), p.L, p.n_pages, ptr<int32_t>(tables), t.R,
                t.W, t.ld, ptr<int32_t>(lens), ptr<int32_t>(refs), ptr<int32_t>(rows), ptr<int32_t>(n_new), n, max_new, ptr<int32_t>(slots),
                ptr<int32_t>(work)))
    return nullptr;
  return THPVariable_Wrap(slots);
  END_HANDLE_TH_ERRORS
}

BLT_CALL(compact) {
  HANDLE_TH_ERRORS
  arguments(n_args, 7);
  const Tensor &pages = tensor(a[0], "pages"), &tables = tensor(a[1], "tables"), &lens = tensor(a[2], "lens"), &refs = tensor(a[3], "refs");
  const Tensor& codes4 = maybe(a[4], "codes4");
  const Pool p = need_pool(pages, codes4, true);
  const Tables t = need_tables(tables, lens);
  need_ints(refs, "refs", p.n_pages);
  Call call(pages, a[5], a[6], {{"tables", &tables}, {"lens", &lens}, {"refs", &refs}, {"codes4", &codes4}});
  const Tensor n_live = at::empty({1}, lens.options()), work = at::empty({2 * p.n_pages + 3}, lens.options());
  if (!call.run(g_abi.kv_pages_compact, ptr<uint8_t>(pages), p.bytes(), ptr<uint8_t>(codes4), p.bytes4(), p.L, p.n_pages, ptr<int32_t>(tables), t.R,
                t.W, t.ld, ptr<int32_t>(lens), ptr<int32_t>(refs), ptr<int32_t>(n_live), ptr<int32_t>(work)))
    return nullptr;
  return THPVariable_Wrap(n_live);
  END_HANDLE_TH_ERRORS
}

BLT_CALL(attention) {
  HANDLE_TH_ERRORS
  arguments(n_args, 10);
  const Tensor &q = tensor(a[0], "q"), &pages = tensor(a[1], "pages"), &tables = tensor(a[2], "tables"), &lens = tensor(a[3], "lens");
  const Tensor &shared = maybe(a[4], "shared"), &codes4 = maybe(a[5], "codes4");
  Tensor out = maybe(a[6], "out"), work = maybe(a[7], "workspace");
  const Pool p = need_pool(pages, codes4, false);
  need_bf16(q, "q", 4);
  const int64_t B = q.size(0), Sq = q.size(1), Hq = q.size(2);
  TORCH_CHECK_VALUE(q.size(3) == p.D, "q: head dimension ", q.size(3), ", the pages hold ", p.D);
  const auto st = q.strides();
  TORCH_CHECK_VALUE(q.numel() == 0 || (st[3] == 1 && (Hq == 1 || st[2] == p.D) && (B == 1 || Sq == 1 || st[0] == Sq * st[1])), "q: strides ", st,
                    ", expected contiguous heads and evenly spaced tokens");
  const Tables t = need_tables(tables, lens);
  TORCH_CHECK_VALUE(t.R == B, "tables: ", t.R, " rows for ", B, " sequences");
  if (shared.defined()) need_ints(shared, "shared");
  const int64_t n_shared = shared.defined() ? shared.numel() : 0;
  if (out.defined()) {
    need_bf16(out, "out", 4);
    TORCH_CHECK_VALUE(out.is_contiguous(), "out: must be contiguous");
    TORCH_CHECK_VALUE(out.sizes() == q.sizes(), "out: shape ", out.sizes(), ", expected ", q.sizes());
  }
  TORCH_CHECK_VALUE(!work.defined() || work.is_contiguous(), "workspace: must be contiguous");
  Call call(q, a[8], a[9], {{"pages", &pages}, {"tables", &tables}, {"lens", &lens}, {"shared", &shared}, {"codes4", &codes4}, {"out", &out},
                            {"workspace", &work}});
  if (!out.defined()) out = at::empty(q.sizes(), q.options().dtype(at::kBFloat16));
  if (!work.defined()) {
    const int64_t bytes = g_abi.kv_attention_3bit_paged_workspace(B, Sq, Hq, p.H, p.D, n_shared, t.W);
    if (bytes < 0) {
      Py_XDECREF(PyObject_CallFunction(g_fail, "i", static_cast<int>(bytes)));
      return nullptr;
    }
    work = at::empty({bytes}, pages.options());
  }
  const int64_t ldq = Sq > 1 ? st[1] : B > 1 ? st[0] : Hq * p.D;
  if (!call.run(g_abi.kv_attention_3bit_paged, ptr<uint16_t>(q), ldq, B, Sq, Hq, p.H, p.D, ptr<uint8_t>(pages), p.n_pages, ptr<uint8_t>(codes4), p.C4,
                ptr<int32_t>(shared), n_shared, ptr<int32_t>(tables), t.W, t.ld, ptr<int32_t>(lens), ptr<uint16_t>(out), ptr<>(work),
                static_cast<int64_t>(work.nbytes())))
    return nullptr;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* setup(PyObject*, PyObject* args) {
  PyObject *fail, *status, *addresses;
  if (!PyArg_ParseTuple(args, "OOO!", &fail, &status, &PyDict_Type, &addresses)) return nullptr;
  bool ok = true;
  auto take = [&](const char* name, auto& fn) {
    PyObject* v = PyDict_GetItemString(addresses, name);
    void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
    ok = ok && p;
    fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(p);
  };
  take("kv_append_3bit", g_abi.kv_append_3bit);
  take("kv_pages_copy", g_abi.kv_pages_copy);
  take("kv_pages_fork", g_abi.kv_pages_fork);
  take("kv_pages_free", g_abi.kv_pages_free);
  take("kv_pages_grow", g_abi.kv_pages_grow);
  take("kv_pages_compact", g_abi.kv_pages_compact);
  take("kv_attention_3bit_paged_workspace", g_abi.kv_attention_3bit_paged_workspace);
  take("kv_attention_3bit_paged", g_abi.kv_attention_3bit_paged);
  take("kv_page_block_bytes", g_abi.kv_page_block_bytes);
  if (!ok) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "a function's address is missing");
    return nullptr;
  }
  Py_XSETREF(g_fail, Py_NewRef(fail));
  Py_XSETREF(g_status, Py_NewRef(status));
  Py_RETURN_NONE;
}

#define BLT_ENTRY(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {BLT_ENTRY(append), BLT_ENTRY(copy),    BLT_ENTRY(fork),      BLT_ENTRY(release),
                           BLT_ENTRY(grow),   BLT_ENTRY(compact), BLT_ENTRY(attention), {"setup", setup, METH_VARARGS, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&g_module); }
