// Argument marshalling of the entry points that take HOST arrays of pointers
// (the AdamW steps, the microscaled 4-bit and the 8-bit code and products) and of
// the experts' balance: checks lists of
// torch tensors, makes the outputs and calls the C ABI of libmuon.so, whose
// functions binding.py hands over once (so the library that MUON_LIBRARY names
// is the one that runs).  A call costs the host about as much as its launch; in
// Python a list of 114 parameters took 140 us to check, ten times its kernel.
//
// Bad arguments raise ValueError before anything is enqueued; the library's
// status is returned for binding.py to check.  Calls go to the current stream of
// the tensors' device, which is made the current device for them.
#include <torch/extension.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <vector>

#include "../../include/muon.h"

namespace {

struct Functions {
  decltype(&muon_adamw_step) adamw = nullptr;
  decltype(&muon_adamw8_step) adamw8 = nullptr;
  decltype(&muon_mx4_quantize) quantize = nullptr;
  decltype(&muon_mx4_dequantize) dequantize = nullptr;
  decltype(&muon_mx4_workspace_size) workspace_size = nullptr;
  decltype(&muon_mx4_matmul) matmul = nullptr;
  decltype(&muon_fp8_quantize) fp8_quantize = nullptr;
  decltype(&muon_fp8_dequantize) fp8_dequantize = nullptr;
  decltype(&muon_fp8_workspace_size) fp8_workspace_size = nullptr;
  decltype(&muon_fp8_matmul) fp8_matmul = nullptr;
  decltype(&muon_fp8_grouped_matmul) fp8_grouped_matmul = nullptr;
  decltype(&muon_fp8_grouped_weight_grad) fp8_grouped_weight_grad = nullptr;
  decltype(&muon_expert_balance_workspace_size) balance_workspace_size = nullptr;
  decltype(&muon_expert_balance) balance = nullptr;
} fn;

PyObject* raw_stream_fn = nullptr;  // torch._C._cuda_getCurrentRawStream

template <class F>
void take(F& f, const py::dict& addresses, const char* name) {
  f = reinterpret_cast<F>(addresses[name].cast<uintptr_t>());
}

void bind_library(const py::dict& addresses, const py::object& raw_stream) {
  take(fn.adamw, addresses, "muon_adamw_step");
  take(fn.adamw8, addresses, "muon_adamw8_step");
  take(fn.quantize, addresses, "muon_mx4_quantize");
  take(fn.dequantize, addresses, "muon_mx4_dequantize");
  take(fn.workspace_size, addresses, "muon_mx4_workspace_size");
  take(fn.matmul, addresses, "muon_mx4_matmul");
  Py_XDECREF(raw_stream_fn);
  raw_stream_fn = py::object(raw_stream).release().ptr();
}

// The 8-bit calls and the experts' balance, which an older library may lack.
void bind_fp8(const py::dict& addresses) {
  take(fn.fp8_quantize, addresses, "muon_fp8_quantize");
  take(fn.fp8_dequantize, addresses, "muon_fp8_dequantize");
  take(fn.fp8_workspace_size, addresses, "muon_fp8_workspace_size");
  take(fn.fp8_matmul, addresses, "muon_fp8_matmul");
  take(fn.fp8_grouped_matmul, addresses, "muon_fp8_grouped_matmul");
  take(fn.fp8_grouped_weight_grad, addresses, "muon_fp8_grouped_weight_grad");
  take(fn.balance_workspace_size, addresses, "muon_expert_balance_workspace_size");
  take(fn.balance, addresses, "muon_expert_balance");
}

void* current_stream(const at::Device& device) {
  py::object handle = py::reinterpret_steal<py::object>(PyObject_CallFunction(raw_stream_fn, "i", device.index()));
  if (!handle) throw py::error_already_set();
  return reinterpret_cast<void*>(handle.cast<uintptr_t>());
}

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

// The tensors of a list or tuple (which keeps them alive during the call).
std::vector<const at::Tensor*> tensors_of(const py::object& seq, const char* name) {
  if (!PyList_Check(seq.ptr()) && !PyTuple_Check(seq.ptr())) refuse(std::string(name) + ": a list of tensors is needed");
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq.ptr());
  std::vector<const at::Tensor*> out(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* item = PySequence_Fast_GET_ITEM(seq.ptr(), i);
    if (!THPVariable_Check(item)) refuse(std::string(name) + ": a list of tensors is needed");
    out[i] = &THPVariable_Unpack(item);
  }
  return out;
}

// The buffers that a call reads and writes.
class Buffers {
 public:
  void reserve(size_t n) {
    ranges_.reserve(n);
    written_.reserve(n);
  }

  // The tensor's memory, which is noted.
  void* add(const at::Tensor& t, bool written) {
    void* const memory = t.data_ptr();
    const uintptr_t p = reinterpret_cast<uintptr_t>(memory);
    const size_t bytes = t.nbytes();
    if (bytes > 0) ranges_.push_back({p, p + bytes, written});
    if (written) written_.push_back(&t);
    return memory;
  }

  // `bytes` bytes from p on that are read.
  void add_read(const void* p, size_t bytes) {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(p);
    if (bytes > 0) ranges_.push_back({begin, begin + bytes, false});
  }

  // No written buffer may overlap another one.
  void check() {
    sort();
    uintptr_t end = 0, written_end = 0;  // of what begins earlier
    for (const Range& r : ranges_) {
      if (r.begin < (r.written ? end : written_end))
        refuse("a buffer that is written overlaps another one of the call (is a tensor in the lists twice?)");
      end = std::max(end, r.end);
      if (r.written) written_end = std::max(written_end, r.end);
    }
  }

  // The status of a call that wrote the written buffers, unless it was refused: their
  // tensors' versions go up, as with any operation in place, so that autograd sees the
  // change (inference tensors have no version).
  int called(muon_status status) const {
    if (status == MUON_OK || status == MUON_ERR_HIP)
      for (const at::Tensor* t : written_)
        if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
    return status;
  }

 private:
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Range> ranges_;
  std::vector<const at::Tensor*> written_;

  // By begin.  The tensors of a list mostly lie in the order of the list, so there are
  // a few ascending runs, which are merged (114 tensors in 4 lists, a step with the
  // sort of all of them 18.4 us, so 17.6).
  void sort() {
    const auto before = [](const Range& a, const Range& b) { return a.begin < b.begin; };
    constexpr size_t kRuns = 16;
    size_t runs[kRuns + 1] = {0}, n = 1;  // where they start, then the end
    for (size_t i = 1; i < ranges_.size(); ++i) {
      if (!before(ranges_[i], ranges_[i - 1])) continue;
      if (n == kRuns) {
        std::sort(ranges_.begin(), ranges_.end(), before);
        return;
      }
      runs[n++] = i;
    }
    runs[n] = ranges_.size();
    for (; n > 1; n = (n + 1) / 2) {  // runs 2 r and 2 r + 1 become run r
      for (size_t r = 0; 2 * r < n; ++r) {
        if (2 * r + 1 < n)
          std::inplace_merge(ranges_.begin() + runs[2 * r], ranges_.begin() + runs[2 * r + 1],
                             ranges_.begin() + runs[2 * r + 2], before);
        runs[r] = runs[2 * r];
      }
      runs[(n + 1) / 2] = ranges_.size();
    }
  }
};

muon_dtype dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return MUON_F32;
    case at::kBFloat16: return MUON_BF16;
    case at::kHalf: return MUON_F16;
    default: refuse(std::string(name) + ": dtype must be float32, bfloat16 or float16");
  }
}

// Contiguous device tensors of one dtype, with the given sizes, on `device`.
std::vector<void*> list_pointers(const std::vector<const at::Tensor*>& list, const char* name,
                                 const std::vector<int64_t>& sizes, const at::Device& device, at::ScalarType dtype,
                                 Buffers& buffers, bool written) {
  if (list.size() != sizes.size()) refuse(std::string(name) + ": one tensor per tensor of W is needed");
  std::vector<void*> out(list.size());
  for (size_t i = 0; i < list.size(); ++i) {
    const at::Tensor& t = *list[i];
    if (t.scalar_type() != dtype)
      refuse(std::string(name) + ": dtype of all tensors must be " + c10::toString(dtype));
    if (t.device() != device) refuse(std::string(name) + ": all tensors must be on the device of W");
    if (t.numel() != sizes[i]) refuse(std::string(name) + ": wrong number of elements");
    if (!t.is_contiguous()) refuse(std::string(name) + ": tensors must be contiguous");
    out[i] = buffers.add(t, written);
  }
  return out;
}

const void* scalar_pointer(const py::object& o, const char* name, at::ScalarType dtype, const at::Device& device,
                           Buffers& buffers) {
  if (!THPVariable_Check(o.ptr())) refuse(std::string(name) + ": a device tensor is needed");
  const at::Tensor& t = THPVariable_Unpack(o.ptr());
  if (t.numel() != 1 || t.scalar_type() != dtype || t.device() != device)
    refuse(std::string(name) + ": a tensor must be one " + c10::toString(dtype) + " on the device of W");
  return buffers.add(t, false);  // every block reads it while others write
}

// A step number on the host.
int64_t host_step(const py::object& o) {
  int overflow = 0;
  const py::object number = py::reinterpret_steal<py::object>(PyNumber_Index(o.ptr()));
  if (!number) PyErr_Clear();
  const int64_t step = number ? PyLong_AsLongLongAndOverflow(number.ptr(), &overflow) : 0;
  if (!number || overflow != 0) refuse("step: an integer of at most 63 bits or a one-element int64 device tensor is needed");
  return step;
}

struct Adamw {
  std::vector<const at::Tensor*> W, G;
  std::vector<int64_t> sizes;
  at::Device device{at::kCPU};
  muon_dtype w_dtype, g_dtype;
  std::vector<void*> w, g;
  Buffers buffers;
  muon_adamw_config cfg;

  Adamw(const py::object& w_list, const py::object& g_list, const py::object& step, double lr, double beta1,
        double beta2, double eps, double weight_decay, const py::object& grad_scale, uint32_t seed) {
    W = tensors_of(w_list, "W");
    if (W.empty()) refuse("W: empty list");
    device = W[0]->device();
    if (!device.is_cuda()) refuse("W: tensors must be device tensors");
    sizes.reserve(W.size());
    for (const at::Tensor* t : W) sizes.push_back(t->numel());
    buffers.reserve(6 * W.size() + 2);
    w_dtype = dtype_of(*W[0], "W");
    if (w_dtype == MUON_F16) refuse("W: dtype must be float32 or bfloat16");
    w = list_pointers(W, "W", sizes, device, W[0]->scalar_type(), buffers, true);
    G = tensors_of(g_list, "G");
    if (G.size() != W.size()) refuse("G: one tensor per tensor of W is needed");
    g_dtype = dtype_of(*G[0], "G");
    g = list_pointers(G, "G", sizes, device, G[0]->scalar_type(), buffers, false);
    cfg = {lr, beta1, beta2, eps, weight_decay, 0, nullptr, nullptr, seed};
    if (THPVariable_Check(step.ptr())) {
      cfg.step_dev = static_cast<const int64_t*>(scalar_pointer(step, "step", at::kLong, device, buffers));
    } else {
      cfg.step = host_step(step);
    }
    if (!grad_scale.is_none())
      cfg.grad_scale =
          static_cast<const float*>(scalar_pointer(grad_scale, "grad_scale", at::kFloat, device, buffers));
  }

  std::vector<void*> state(const py::object& list, const char* name, const std::vector<int64_t>& n, at::ScalarType dtype) {
    return list_pointers(tensors_of(list, name), name, n, device, dtype, buffers, true);
  }
};

int adamw_step(const py::object& W, const py::object& M, const py::object& V, const py::object& G,
               const py::object& step, double lr, double beta1, double beta2, double eps, double weight_decay,
               const py::object& grad_scale) {
  Adamw a(W, G, step, lr, beta1, beta2, eps, weight_decay, grad_scale, 0);
  const std::vector<void*> m = a.state(M, "M", a.sizes, at::kFloat), v = a.state(V, "V", a.sizes, at::kFloat);
  a.buffers.check();
  const c10::DeviceGuard guard(a.device);
  const muon_status st =
      fn.adamw(static_cast<int>(a.sizes.size()), a.sizes.data(), a.w.data(), a.w_dtype, m.data(), v.data(),
               const_cast<const void* const*>(a.g.data()), a.g_dtype, &a.cfg, current_stream(a.device));
  return a.buffers.called(st);
}

int adamw8_step(const py::object& W, const py::object& m_codes, const py::object& m_scales, const py::object& r_codes,
                const py::object& r_scales, const py::object& G, const py::object& step, double lr, double beta1,
                double beta2, double eps, double weight_decay, const py::object& grad_scale, uint32_t seed) {
  Adamw a(W, G, step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed);
  std::vector<int64_t> groups(a.sizes.size());
  for (size_t i = 0; i < groups.size(); ++i) groups[i] = (a.sizes[i] + 127) / 128;
  const std::vector<void*> mc = a.state(m_codes, "m_codes", a.sizes, at::kFloat8_e4m3fn),
                           ms = a.state(m_scales, "m_scales", groups, at::kFloat),
                           rc = a.state(r_codes, "r_codes", a.sizes, at::kFloat8_e4m3fn),
                           rs = a.state(r_scales, "r_scales", groups, at::kFloat);
  a.buffers.check();
  const muon_adamw8_state state{mc.data(), ms.data(), rc.data(), rs.data()};
  const c10::DeviceGuard guard(a.device);
  const muon_status st =
      fn.adamw8(static_cast<int>(a.sizes.size()), a.sizes.data(), a.w.data(), a.w_dtype, &state,
                const_cast<const void* const*>(a.g.data()), a.g_dtype, &a.cfg, current_stream(a.device));
  return a.buffers.called(st);
}

// ---------------------------------------------------------------------------
// microscaled 4-bit code
// ---------------------------------------------------------------------------
int64_t units_of(int64_t k) { return (k + 127) / 128; }

// A batch of same-shape contiguous device matrices.
struct Matrices {
  std::vector<void*> ptr;
  int64_t rows = 0, cols = 0;
  muon_dtype dtype = MUON_F32;
  at::Device device{at::kCPU};

  Matrices(const py::object& seq, const char* name, Buffers* buffers, bool written) {
    const std::vector<const at::Tensor*> list = tensors_of(seq, name);
    if (list.empty()) refuse(std::string(name) + ": empty batch");
    const at::Tensor& t0 = *list[0];
    if (t0.dim() != 2) refuse(std::string(name) + ": matrices must be 2-D");
    rows = t0.size(0);
    cols = t0.size(1);
    dtype = dtype_of(t0, name);
    device = t0.device();
    ptr.reserve(list.size());
    for (const at::Tensor* t : list) {
      if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || t->scalar_type() != t0.scalar_type() ||
          t->device() != device)
        refuse(std::string(name) + ": all matrices must share shape, dtype and device");
      if (!t->is_contiguous()) refuse(std::string(name) + ": matrices must be contiguous");
      if (!device.is_cuda()) refuse(std::string(name) + ": matrices must be device tensors");
      ptr.push_back(t->data_ptr());
      if (buffers != nullptr) buffers->add(*t, written);
    }
  }
  int batch() const { return static_cast<int>(ptr.size()); }
  const void* const* in() const { return const_cast<const void* const*>(ptr.data()); }
};

// A batch of codes: (codes, scales) lists and the length of a row.
struct Codes {
  std::vector<void*> codes, scales;
  int64_t rows = 0, cols = 0;
  at::Device device{at::kCPU};

  Codes() = default;
  Codes(const py::object& code_list, const py::object& scale_list, int64_t k, const char* name,
        Buffers* buffers, bool written) {
    const auto c = tensors_of(code_list, name), s = tensors_of(scale_list, name);
    if (c.empty() || c.size() != s.size())
      refuse(std::string(name) + ": codes and scales must hold one tensor per matrix");
    cols = k;
    if (k < 1 || c[0]->dim() != 3 || c[0]->size(0) != units_of(k) || c[0]->size(1) < 1 || c[0]->size(2) != 64)
      refuse(std::string(name) + ": codes must be (ceil(cols / 128), rows, 64)");
    rows = c[0]->size(1);
    device = c[0]->device();
    if (!device.is_cuda()) refuse(std::string(name) + ": codes must be device tensors");
    read(c, 64, 16, codes, name, buffers, written);
    read(s, 4, 4, scales, name, buffers, written);
  }
  // New buffers for `batch` matrices, appended to the given lists.
  Codes(int batch, int64_t r, int64_t k, const at::Device& d, py::list code_list, py::list scale_list)
      : rows(r), cols(k), device(d) {
    const int64_t lines = units_of(k) * r, split = batch * lines * 64;  // all codes first: 16-byte aligned
    const at::Tensor flat = at::empty({batch * lines * 68}, at::TensorOptions().dtype(at::kByte).device(d));
    for (int b = 0; b < batch; ++b) {
      const at::Tensor c = flat.as_strided({units_of(k), r, 64}, {r * 64, 64, 1}, b * lines * 64);
      const at::Tensor s = flat.as_strided({units_of(k), r, 4}, {r * 4, 4, 1}, split + b * lines * 4);
      codes.push_back(c.data_ptr());
      scales.push_back(s.data_ptr());
      code_list.append(c);
      scale_list.append(s);
    }
  }
  int batch() const { return static_cast<int>(codes.size()); }
  const void* const* c() const { return const_cast<const void* const*>(codes.data()); }
  const void* const* s() const { return const_cast<const void* const*>(scales.data()); }

 private:
  void read(const std::vector<const at::Tensor*>& list, int64_t last, uintptr_t align, std::vector<void*>& to,
            const char* name, Buffers* buffers, bool written) {
    for (const at::Tensor* t : list) {
      if (t->scalar_type() != at::kByte || t->device() != device || t->dim() != 3 || t->size(0) != units_of(cols) ||
          t->size(1) != rows || t->size(2) != last)
        refuse(std::string(name) + ": all codes and scales must be uint8 of one shape and device");
      if (!t->is_contiguous() || reinterpret_cast<uintptr_t>(t->data_ptr()) % align != 0)
        refuse(std::string(name) + ": codes and scales must be contiguous, codes 16-byte and scales 4-byte aligned");
      to.push_back(t->data_ptr());
      if (buffers != nullptr) buffers->add(*t, written);
    }
  }
};

int as_int(int64_t x) { return x > INT32_MAX ? INT32_MAX : static_cast<int>(x); }  // out of the library's range

// out: None, or per orientation (codes, scales, cols).  Returns (status, codes
// and scales lists of each orientation).
py::tuple mx4_quantize(const py::object& X, bool along, bool across, const py::object& out) {
  Buffers buffers;
  const Matrices x(X, "X", out.is_none() ? nullptr : &buffers, false);
  const c10::DeviceGuard guard(x.device);
  Codes q[2];
  py::list made;
  int given = 0;
  for (int o = 0; o < 2; ++o) {
    if (!(o == 0 ? along : across)) continue;
    const int64_t r = o == 0 ? x.rows : x.cols, k = o == 0 ? x.cols : x.rows;
    if (out.is_none()) {
      if (r < 1 || k < 1) refuse("X: matrices must not be empty");
      py::list c, s;
      q[o] = Codes(x.batch(), r, k, x.device, c, s);
      made.append(py::make_tuple(c, s));
    } else {
      const py::tuple t = out.cast<py::sequence>()[given++].cast<py::tuple>();
      q[o] = Codes(t[0], t[1], t[2].cast<int64_t>(), "out", &buffers, true);
      if (q[o].batch() != x.batch() || q[o].rows != r || q[o].cols != k || q[o].device != x.device)
        refuse("out must have the shape, batch and device of the result");
    }
  }
  buffers.check();
  const muon_status st = fn.quantize(x.batch(), as_int(x.rows), as_int(x.cols), x.in(), x.dtype,
                                     along ? q[0].codes.data() : nullptr, along ? q[0].scales.data() : nullptr,
                                     across ? q[1].codes.data() : nullptr, across ? q[1].scales.data() : nullptr,
                                     current_stream(x.device));
  return py::make_tuple(buffers.called(st), made);
}

// New matrices, as a list.
py::list new_matrices(int batch, int64_t rows, int64_t cols, at::ScalarType dtype, const at::Device& device) {
  py::list out;
  const at::Tensor all = at::empty({batch, rows, cols}, at::TensorOptions().dtype(dtype).device(device));
  for (int b = 0; b < batch; ++b) out.append(all.select(0, b));
  return out;
}

at::ScalarType value_type(const py::object& dtype) {
  if (!THPDtype_Check(dtype.ptr())) refuse("dtype must be float32 or bfloat16");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
  if (t != at::kFloat && t != at::kBFloat16 && t != at::kHalf) refuse("dtype must be float32 or bfloat16");
  return t;
}

py::tuple mx4_dequantize(const py::object& codes, const py::object& scales, int64_t cols, const py::object& dtype,
                         const py::object& out) {
  Buffers buffers;
  const Codes q(codes, scales, cols, "q", &buffers, false);
  const at::ScalarType t = value_type(dtype);
  const c10::DeviceGuard guard(q.device);
  const py::object Y = out.is_none() ? py::object(new_matrices(q.batch(), q.rows, cols, t, q.device)) : out;
  const Matrices y(Y, "out", &buffers, true);
  if (y.batch() != q.batch() || y.rows != q.rows || y.cols != cols || y.device != q.device)
    refuse("out must have the shape, batch and device of the result");
  buffers.check();
  const muon_status st = fn.dequantize(q.batch(), as_int(q.rows), as_int(cols), q.c(), q.s(), y.ptr.data(), y.dtype,
                                       current_stream(q.device));
  return py::make_tuple(buffers.called(st), Y);
}

// Returns (status, C).
py::tuple mx4_matmul(const py::object& a_codes, const py::object& a_scales, const py::object& b_codes,
                     const py::object& b_scales, int64_t k, int64_t kb, const py::object& dtype, const py::object& out,
                     bool accumulate, const py::object& workspace) {
  Buffers buffers;
  const Codes a(a_codes, a_scales, k, "A", &buffers, false), b(b_codes, b_scales, kb, "B", &buffers, false);
  if (a.batch() != b.batch() || k != kb || a.device != b.device)
    refuse("A and B must share the batch, the row length and the device");
  if (accumulate && out.is_none()) refuse("accumulate needs out");
  const c10::DeviceGuard guard(a.device);
  const size_t need = fn.workspace_size(a.batch(), as_int(a.rows), as_int(b.rows), as_int(k));
  if (need == 0) return py::make_tuple(static_cast<int>(MUON_ERR_INVALID_ARG), py::none());
  const py::object C =
      out.is_none() ? py::object(new_matrices(a.batch(), a.rows, b.rows, value_type(dtype), a.device)) : out;
  const Matrices c(C, "out", &buffers, true);
  if (c.batch() != a.batch() || c.rows != a.rows || c.cols != b.rows || c.device != a.device)
    refuse("out must have one m x n matrix per pair, on the same device");
  // from the allocator at every call: its memory is reused in the stream's order,
  // and under capture it belongs to the graph, so two graphs never share it
  at::Tensor ws;
  if (workspace.is_none()) {
    ws = at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(a.device));
  } else {
    if (!THPVariable_Check(workspace.ptr())) refuse("workspace must be a device tensor");
    ws = THPVariable_Unpack(workspace.ptr());
    if (ws.device() != a.device || !ws.is_contiguous()) refuse("workspace must be a contiguous tensor on the device of A");
    buffers.add(ws, true);
  }
  buffers.check();
  const muon_status st = fn.matmul(a.batch(), as_int(a.rows), as_int(b.rows), as_int(k), a.c(), a.s(), b.c(), b.s(),
                                   c.ptr.data(), c.dtype, accumulate ? 1 : 0, ws.data_ptr(), ws.nbytes(),
                                   current_stream(a.device));
  return py::make_tuple(buffers.called(st), C);
}

// A call's scratch, from the allocator at every call: its memory is reused in the
// stream's order, and under capture it belongs to the graph, so two graphs never
// share it.  Or the caller's.
at::Tensor scratch(const py::object& workspace, size_t need, const at::Device& device, Buffers& buffers) {
  if (workspace.is_none())
    return at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(device));
  if (!THPVariable_Check(workspace.ptr())) refuse("workspace must be a device tensor");
  const at::Tensor& ws = THPVariable_Unpack(workspace.ptr());  // the Python object's, which outlives the call
  if (ws.device() != device || !ws.is_contiguous()) refuse("workspace must be a contiguous tensor on the device of the operands");
  buffers.add(ws, true);
  return ws;
}

// ---------------------------------------------------------------------------
// 8-bit code with a scale for each block of 128
// ---------------------------------------------------------------------------
// A batch of codes: (codes, scales) lists, the length of a row and, if its rows were
// coded in groups, their number.
struct Fp8Codes {
  std::vector<void*> codes, scales;
  int64_t rows = 0, cols = 0, groups = 0;
  muon_fp8_format format = MUON_E4M3;
  at::Device device{at::kCPU};

  static int64_t units(int64_t k, int64_t groups) { return groups > 0 ? (k + 127 * groups) / 128 : units_of(k); }
  static int64_t pitch(int64_t rows) { return (rows + 15) / 16 * 16; }

  Fp8Codes() = default;
  Fp8Codes(const py::object& code_list, const py::object& scale_list, int64_t k, int64_t g, const char* name,
           Buffers* buffers, bool written)
      : cols(k), groups(g) {
    const auto c = tensors_of(code_list, name), s = tensors_of(scale_list, name);
    if (c.empty() || c.size() != s.size())
      refuse(std::string(name) + ": codes and scales must hold one tensor per matrix");
    const at::ScalarType type = c[0]->scalar_type();
    if (type != at::kFloat8_e4m3fn && type != at::kFloat8_e5m2)
      refuse(std::string(name) + ": codes must be float8_e4m3fn or float8_e5m2");
    format = type == at::kFloat8_e4m3fn ? MUON_E4M3 : MUON_E5M2;
    if (k < 1 || k > INT32_MAX || g < 0 || g > INT32_MAX || c[0]->dim() != 3 || c[0]->size(0) != 2 * units(k, g) ||
        c[0]->size(1) < 1 || c[0]->size(2) != 64)
      refuse(std::string(name) + ": codes must be (2 * units, rows, 64), units = ceil(cols / 128), or with groups "
                                 "(cols + 127 * groups) // 128");
    rows = c[0]->size(1);
    device = c[0]->device();
    if (!device.is_cuda()) refuse(std::string(name) + ": codes must be device tensors");
    codes.reserve(c.size());
    scales.reserve(c.size());
    for (size_t i = 0; i < c.size(); ++i) {
      if (c[i]->scalar_type() != type || c[i]->device() != device || c[i]->sizes() != c[0]->sizes())
        refuse(std::string(name) + ": all codes must share type, shape and device");
      if (s[i]->scalar_type() != at::kByte || s[i]->device() != device || s[i]->dim() != 2 ||
          s[i]->size(0) != units(k, g) || s[i]->size(1) != pitch(rows))
        refuse(std::string(name) + ": scales must be uint8 (units, rows rounded up to 16) on the codes' device");
      for (const at::Tensor* t : {c[i], s[i]}) {
        void* const p = t->data_ptr();
        if (!t->is_contiguous() || reinterpret_cast<uintptr_t>(p) % 16 != 0)
          refuse(std::string(name) + ": codes and scales must be contiguous and 16-byte aligned");
        (t == c[i] ? codes : scales).push_back(p);
        if (buffers != nullptr) buffers->add(*t, written);
      }
    }
  }
  // New buffers for `batch` matrices, appended to the given lists.
  Fp8Codes(int batch, int64_t r, int64_t k, int64_t g, muon_fp8_format f, const at::Device& d, py::list code_list,
           py::list scale_list)
      : rows(r), cols(k), groups(g), format(f), device(d) {
    const int64_t u = units(k, g), code_bytes = u * r * 128, scale_bytes = u * pitch(r);  // multiples of 16
    const at::Tensor flat = at::empty({batch * (code_bytes + scale_bytes)}, at::TensorOptions().dtype(at::kByte).device(d));
    const at::ScalarType type = f == MUON_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2;
    const at::Tensor all = flat.view(type);
    for (int b = 0; b < batch; ++b) {
      const at::Tensor c = all.as_strided({2 * u, r, 64}, {r * 64, 64, 1}, b * code_bytes);
      const at::Tensor s = flat.as_strided({u, pitch(r)}, {pitch(r), 1}, batch * code_bytes + b * scale_bytes);
      codes.push_back(c.data_ptr());
      scales.push_back(s.data_ptr());
      code_list.append(c);
      scale_list.append(s);
    }
  }
  int batch() const { return static_cast<int>(codes.size()); }
  const void* const* c() const { return const_cast<const void* const*>(codes.data()); }
  const void* const* s() const { return const_cast<const void* const*>(scales.data()); }
};

// Row counts of groups: a contiguous int32 device tensor.
const int32_t* counts_pointer(const py::object& o, const at::Device& device, int64_t* groups, Buffers& buffers) {
  if (!THPVariable_Check(o.ptr())) refuse("counts: a device tensor is needed");
  const at::Tensor& t = THPVariable_Unpack(o.ptr());
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.numel() < 1 || !t.is_contiguous() || t.device() != device)
    refuse("counts must be a contiguous 1-D int32 tensor on the device of the operands");
  *groups = t.numel();
  return static_cast<const int32_t*>(buffers.add(t, false));
}

// out: None, or per orientation (codes, scales, cols, groups).  Returns (status, codes
// and scales lists of each orientation).
py::tuple fp8_quantize(const py::object& X, bool along, bool across, bool tile, bool e5m2, const py::object& counts,
                       const py::object& out) {
  Buffers buffers;
  const Matrices x(X, "X", &buffers, false);
  const c10::DeviceGuard guard(x.device);
  const muon_fp8_format format = e5m2 ? MUON_E5M2 : MUON_E4M3;
  int64_t groups = 0;
  const int32_t* const n = counts.is_none() ? nullptr : counts_pointer(counts, x.device, &groups, buffers);
  if (n != nullptr && (!across || tile || x.batch() != 1))
    refuse("counts: one matrix, coded in blocks of a row, with its transposed code");
  Fp8Codes q[2];
  py::list made;
  int given = 0;
  for (int o = 0; o < 2; ++o) {
    if (!(o == 0 ? along : across)) continue;
    const int64_t r = o == 0 ? x.rows : x.cols, k = o == 0 ? x.cols : x.rows, g = o == 0 ? 0 : groups;
    if (out.is_none()) {
      if (r < 1 || k < 1) refuse("X: matrices must not be empty");
      py::list c, s;
      q[o] = Fp8Codes(x.batch(), r, k, g, format, x.device, c, s);
      made.append(py::make_tuple(c, s));
    } else {
      const py::tuple t = out.cast<py::sequence>()[given++].cast<py::tuple>();
      q[o] = Fp8Codes(t[0], t[1], t[2].cast<int64_t>(), t[3].cast<int64_t>(), "out", &buffers, true);
      if (q[o].batch() != x.batch() || q[o].rows != r || q[o].cols != k || q[o].groups != g || q[o].device != x.device ||
          q[o].format != format)
        refuse("out must have the shape, batch, groups, format and device of the result");
    }
  }
  buffers.check();
  const muon_status st = fn.fp8_quantize(x.batch(), as_int(x.rows), as_int(x.cols), x.in(), x.dtype, tile ? 1 : 0, format, n,
                                         as_int(groups), along ? q[0].codes.data() : nullptr,
                                         along ? q[0].scales.data() : nullptr, across ? q[1].codes.data() : nullptr,
                                         across ? q[1].scales.data() : nullptr, current_stream(x.device));
  return py::make_tuple(static_cast<int>(buffers.called(st)), made);
}

py::tuple fp8_dequantize(const py::object& codes, const py::object& scales, int64_t cols, int64_t groups,
                         const py::object& dtype, const py::object& out) {
  Buffers buffers;
  const Fp8Codes q(codes, scales, cols, groups, "q", &buffers, false);
  if (groups != 0) refuse("q: a code in groups has no values of its own");
  const at::ScalarType t = value_type(dtype);
  const c10::DeviceGuard guard(q.device);
  const py::object Y = out.is_none() ? py::object(new_matrices(q.batch(), q.rows, cols, t, q.device)) : out;
  const Matrices y(Y, "out", &buffers, true);
  if (y.batch() != q.batch() || y.rows != q.rows || y.cols != cols || y.device != q.device)
    refuse("out must have the shape, batch and device of the result");
  buffers.check();
  const muon_status st = fn.fp8_dequantize(q.batch(), as_int(q.rows), as_int(cols), q.c(), q.s(), q.format, y.ptr.data(),
                                           y.dtype, current_stream(q.device));
  return py::make_tuple(static_cast<int>(buffers.called(st)), Y);
}

void check_operands(const Fp8Codes& a, const Fp8Codes& b) {
  if (a.cols != b.cols || a.device != b.device) refuse("A and B must share the row length and the device");
  if (b.format != MUON_E4M3) refuse("B must be coded in e4m3 (A may be e5m2)");
}

// Returns (status, C), as the two calls below.
py::tuple fp8_matmul(const py::tuple& A, const py::tuple& B, const py::object& dtype, const py::object& out, bool accumulate,
                     const py::object& workspace) {
  Buffers buffers;
  const Fp8Codes a(A[0], A[1], A[2].cast<int64_t>(), A[3].cast<int64_t>(), "A", &buffers, false);
  const Fp8Codes b(B[0], B[1], B[2].cast<int64_t>(), B[3].cast<int64_t>(), "B", &buffers, false);
  check_operands(a, b);
  if (a.groups != 0 || b.groups != 0) refuse("a code in groups takes part in fp8_grouped_weight_grad only");
  if (a.batch() != b.batch()) refuse("A and B must share the batch");
  if (accumulate && out.is_none()) refuse("accumulate needs out");
  const c10::DeviceGuard guard(a.device);
  const size_t need = fn.fp8_workspace_size(a.batch(), as_int(a.rows), as_int(b.rows), as_int(a.cols));
  if (need == 0) return py::make_tuple(static_cast<int>(MUON_ERR_INVALID_ARG), py::none());
  const py::object C =
      out.is_none() ? py::object(new_matrices(a.batch(), a.rows, b.rows, value_type(dtype), a.device)) : out;
  const Matrices c(C, "out", &buffers, true);
  if (c.batch() != a.batch() || c.rows != a.rows || c.cols != b.rows || c.device != a.device)
    refuse("out must have one m x n matrix per pair, on the same device");
  const at::Tensor ws = scratch(workspace, need, a.device, buffers);
  buffers.check();
  const muon_status st = fn.fp8_matmul(a.batch(), as_int(a.rows), as_int(b.rows), as_int(a.cols), a.c(), a.s(), a.format,
                                       b.c(), b.s(), c.ptr.data(), c.dtype, accumulate ? 1 : 0, ws.data_ptr(), ws.nbytes(),
                                       current_stream(a.device));
  return py::make_tuple(static_cast<int>(buffers.called(st)), C);
}

py::tuple fp8_grouped_matmul(const py::tuple& A, const py::tuple& B, const py::object& counts, const py::object& dtype,
                             const py::object& out, bool accumulate) {
  Buffers buffers;
  const Fp8Codes a(A[0], A[1], A[2].cast<int64_t>(), A[3].cast<int64_t>(), "A", &buffers, false);
  const Fp8Codes b(B[0], B[1], B[2].cast<int64_t>(), B[3].cast<int64_t>(), "B", &buffers, false);
  check_operands(a, b);
  if (a.groups != 0 || b.groups != 0) refuse("a code in groups takes part in fp8_grouped_weight_grad only");
  int64_t groups = 0;
  const int32_t* const n = counts_pointer(counts, a.device, &groups, buffers);
  if (a.batch() != 1 || b.batch() != groups) refuse("A must be one matrix, and B one for each of the counts");
  if (accumulate && out.is_none()) refuse("accumulate needs out");
  const c10::DeviceGuard guard(a.device);
  const py::object C = out.is_none() ? py::object(new_matrices(1, a.rows, b.rows, value_type(dtype), a.device)) : out;
  const Matrices c(C, "out", &buffers, true);
  if (c.batch() != 1 || c.rows != a.rows || c.cols != b.rows || c.device != a.device)
    refuse("out must be one m x n matrix on the same device");
  buffers.check();
  const muon_status st = fn.fp8_grouped_matmul(as_int(groups), as_int(a.rows), as_int(b.rows), as_int(a.cols), n, a.codes[0],
                                               a.scales[0], a.format, b.c(), b.s(), c.ptr[0], c.dtype, accumulate ? 1 : 0,
                                               out.is_none() ? 1 : 0, current_stream(a.device));
  return py::make_tuple(static_cast<int>(buffers.called(st)), C);
}

py::tuple fp8_grouped_weight_grad(const py::tuple& A, const py::tuple& B, const py::object& counts, const py::object& dtype,
                                  const py::object& out, bool accumulate) {
  Buffers buffers;
  const Fp8Codes a(A[0], A[1], A[2].cast<int64_t>(), A[3].cast<int64_t>(), "A", &buffers, false);
  const Fp8Codes b(B[0], B[1], B[2].cast<int64_t>(), B[3].cast<int64_t>(), "B", &buffers, false);
  check_operands(a, b);
  int64_t groups = 0;
  const int32_t* const n = counts_pointer(counts, a.device, &groups, buffers);
  if (a.batch() != 1 || b.batch() != 1 || a.groups != groups || b.groups != groups)
    refuse("A and B must be one matrix each, coded along columns with as many counts");
  if (accumulate && out.is_none()) refuse("accumulate needs out");
  const c10::DeviceGuard guard(a.device);
  const py::object C =
      out.is_none() ? py::object(new_matrices(as_int(groups), a.rows, b.rows, value_type(dtype), a.device)) : out;
  const Matrices c(C, "out", &buffers, true);
  if (c.batch() != groups || c.rows != a.rows || c.cols != b.rows || c.device != a.device)
    refuse("out must have one m x n matrix per group, on the same device");
  buffers.check();
  const muon_status st = fn.fp8_grouped_weight_grad(as_int(groups), as_int(a.cols), as_int(a.rows), as_int(b.rows), n,
                                                    a.codes[0], a.scales[0], a.format, b.codes[0], b.scales[0], c.ptr.data(),
                                                    c.dtype, accumulate ? 1 : 0, current_stream(a.device));
  return py::make_tuple(static_cast<int>(buffers.called(st)), C);
}

// ---------------------------------------------------------------------------
// experts' balance
// ---------------------------------------------------------------------------
const at::Tensor& one_tensor(const py::object& o, const char* name) {
  if (!THPVariable_Check(o.ptr())) refuse(std::string(name) + ": a device tensor is needed");
  return THPVariable_Unpack(o.ptr());
}

// grad: None (no gradient), True (a new one) or a tensor.  Returns (status, loss, counts, gradient).
py::tuple expert_balance(const py::object& logits, const py::object& index, double coefficient, bool sigmoid,
                         const py::object& mask, const py::object& grad, bool accumulate, const py::object& grad_scale,
                         const py::object& workspace) {
  Buffers buffers;
  const at::Tensor &z = one_tensor(logits, "logits"), &choice = one_tensor(index, "index");
  const at::Device device = z.device();
  if (!device.is_cuda()) refuse("logits must be a device tensor");
  const muon_dtype type = dtype_of(z, "logits");
  const int64_t dim = z.dim();
  if (dim != 2 && dim != 3) refuse("logits must be (tokens, experts) or (sequences, tokens, experts)");
  const int64_t S = dim == 3 ? z.size(0) : 1, T = z.size(dim - 2), E = z.size(dim - 1);
  if (z.numel() == 0) refuse("logits must not be empty");
  const int64_t stride = z.stride(dim - 2);
  if ((E > 1 && z.stride(dim - 1) != 1) || stride < 0 || (S > 1 && T > 1 && z.stride(0) != T * stride))
    refuse("logits: the experts of a token must lie behind one another, and all tokens one stride apart");
  const int64_t step = T > 1 ? stride : (dim == 3 ? z.stride(0) : stride);
  if (choice.dim() != dim || choice.size(dim - 1) < 1 || choice.device() != device ||
      (choice.scalar_type() != at::kInt && choice.scalar_type() != at::kLong) || !choice.is_contiguous())
    refuse("index must be a contiguous int32 or int64 tensor on the device of the logits, with one row a token");
  for (int64_t d = 0; d + 1 < dim; ++d)
    if (choice.size(d) != z.size(d)) refuse("index must have one row for each row of the logits");
  const int64_t K = choice.size(dim - 1);
  buffers.add_read(z.data_ptr(), ((S * T - 1) * step + E) * z.element_size());  // with what lies between the rows
  buffers.add(choice, false);
  const uint8_t* m = nullptr;
  if (!mask.is_none()) {
    const at::Tensor& t = one_tensor(mask, "mask");
    if ((t.scalar_type() != at::kBool && t.scalar_type() != at::kByte) || !t.is_contiguous() || t.device() != device ||
        t.dim() != dim - 1 || t.size(0) != z.size(0) || (dim == 3 && t.size(1) != T))
      refuse("mask must be a contiguous bool or uint8 tensor on the device of the logits, one element a token");
    m = static_cast<const uint8_t*>(buffers.add(t, false));
  }
  const float* scale = nullptr;
  if (!grad_scale.is_none())
    scale = static_cast<const float*>(scalar_pointer(grad_scale, "grad_scale", at::kFloat, device, buffers));
  const c10::DeviceGuard guard(device);
  const size_t need = fn.balance_workspace_size(as_int(S), as_int(T), as_int(E), as_int(K));
  if (need == 0)
    return py::make_tuple(static_cast<int>(MUON_ERR_INVALID_ARG), py::none(), py::none(), py::none());
  const auto options = at::TensorOptions().device(device);
  at::Tensor g;
  if (grad.ptr() == Py_True) {
    if (accumulate) refuse("accumulate needs a gradient to add to");
    g = at::empty(z.sizes(), options.dtype(z.scalar_type()));
  } else if (!grad.is_none()) {
    g = one_tensor(grad, "grad");
    if (g.scalar_type() != z.scalar_type() || g.sizes() != z.sizes() || g.device() != device || !g.is_contiguous())
      refuse("grad must be contiguous, of the shape, dtype and device of the logits");
    buffers.add(g, true);
  } else if (accumulate) {
    refuse("accumulate needs a gradient to add to");
  }
  const at::Tensor loss = at::empty({}, options.dtype(at::kFloat)), counts = at::empty({E}, options.dtype(at::kInt));
  const at::Tensor ws = scratch(workspace, need, device, buffers);
  buffers.check();
  const muon_status st =
      fn.balance(as_int(S), as_int(T), as_int(E), as_int(K), z.data_ptr(), type, step, choice.data_ptr(),
                 choice.scalar_type() == at::kLong ? 64 : 32, m, sigmoid ? MUON_SIGMOID : MUON_SOFTMAX, coefficient, scale,
                 static_cast<float*>(loss.data_ptr()), static_cast<int32_t*>(counts.data_ptr()),
                 g.defined() ? g.data_ptr() : nullptr, accumulate ? 1 : 0, ws.data_ptr(), ws.nbytes(), current_stream(device));
  return py::make_tuple(static_cast<int>(buffers.called(st)), loss, counts, g.defined() ? py::cast(g) : py::none());
}

}  // namespace

PYBIND11_MODULE(_native, m) {
  m.def("bind_library", &bind_library);
  m.def("adamw_step", &adamw_step);
  m.def("adamw8_step", &adamw8_step);
  m.def("mx4_quantize", &mx4_quantize);
  m.def("mx4_dequantize", &mx4_dequantize);
  m.def("mx4_matmul", &mx4_matmul);
  m.def("bind_fp8", &bind_fp8);
  m.def("fp8_quantize", &fp8_quantize);
  m.def("fp8_dequantize", &fp8_dequantize);
  m.def("fp8_matmul", &fp8_matmul);
  m.def("fp8_grouped_matmul", &fp8_grouped_matmul);
  m.def("fp8_grouped_weight_grad", &fp8_grouped_weight_grad);
  m.def("expert_balance", &expert_balance);
}
