// The serving operators' calls from Python, without its per-argument cost.
//
// A generated token's step has kernels of a few microseconds, and marshalling
// its tensors in Python took more than twenty.  The functions here do for the
// ordinary call what serving.py does for every call: check the tensors,
// allocate the outputs and the workspace, and pass raw pointers and the
// current stream to the C entry point.  Whatever is not plainly an ordinary
// call (another device, an unusual stride, a wrong type, pages or a table over
// what the call reads) returns None, and serving.py takes it from there, with its
// own checks and messages.
//
// Each returns a tuple of tensors (the last one is the workspace), a negative
// pa_status as an int, or None.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <initializer_list>
#include <utility>

#include "../../include/pulsar_serving.h"

namespace {

using at::Tensor;

constexpr int64_t kMaxInt = 2147483647;

// An ordinary call's tensors: on the current CUDA device.
struct Args {
  PyObject* const* v;
  Py_ssize_t n;
  int dev = -1;   // the current device, asked for once there is a CUDA tensor
  bool ok;

  Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t want) : v(args), n(count), ok(count == want) {}
  const Tensor* tensor(int i) {
    if (!ok || !THPVariable_Check(v[i])) {
      ok = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(v[i]);
    if (t.is_cuda() && dev < 0) dev = c10::cuda::current_device();
    if (!t.is_cuda() || t.get_device() != dev) {
      ok = false;
      return nullptr;
    }
    return &t;
  }
  // dense int32 with at least n elements
  const Tensor* ints(int i, int64_t count) {
    const Tensor* t = tensor(i);
    if (t && (t->scalar_type() != at::kInt || !t->is_contiguous() || t->numel() < count)) ok = false;
    return t;
  }
  // packed [N][heads][d] rows, N >= 1, dense inside a token
  const Tensor* rows(int i, int64_t* ld) {
    const Tensor* t = tensor(i);
    if (!t) return nullptr;
    if (t->dim() != 3 || t->size(0) < 1 || t->size(1) < 1 || t->size(2) < 2 || t->stride(2) != 1 ||
        (t->size(1) > 1 && t->stride(1) != t->size(2))) {
      ok = false;
      return nullptr;
    }
    *ld = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
    if (*ld < t->size(1) * t->size(2)) ok = false;
    return t;
  }
  const Tensor* table(int i, int64_t B, int64_t* stride) {
    const Tensor* t = tensor(i);
    if (!t) return nullptr;
    if (t->dim() != 2 || t->scalar_type() != at::kInt || t->size(0) < B || t->size(1) < 1 || t->size(1) > kMaxInt ||
        (t->size(1) > 1 && t->stride(1) != 1) || (t->size(0) > 1 && t->stride(0) < t->size(1))) {
      ok = false;
      return nullptr;
    }
    *stride = t->size(0) > 1 ? t->stride(0) : t->size(1);
    return t;
  }
  int64_t integer(int i) {
    if (!ok || !PyLong_Check(v[i])) {
      ok = false;
      return 0;
    }
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(v[i], &over);
    if (over != 0 || x < -kMaxInt || x > kMaxInt) ok = false;
    return x;
  }
  Tensor make(at::IntArrayRef size, at::ScalarType type) const {
    const c10::Device device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev));
    return at::detail::empty_cuda(size, type, device, std::nullopt);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }
};

// Whether a tensor's elements share an address with another's: what a kernel
// writes must not be read or written by another of its blocks.  (The spans of
// serving.py, which refuses such a call with a message.)
bool overlap(const Tensor& a, std::initializer_list<const Tensor*> others) {
  auto span = [](const Tensor& t) {
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    const char* first = static_cast<const char*>(t.const_data_ptr());
    return std::make_pair(first, first + (last + 1) * static_cast<int64_t>(t.element_size()));
  };
  if (a.numel() == 0) return false;
  const auto x = span(a);
  for (const Tensor* t : others) {
    if (t->numel() == 0) continue;
    const auto y = span(*t);
    if (x.first < y.second && y.first < x.second) return true;
  }
  return false;
}

int dtype_of(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? PA_BF16 : t.scalar_type() == at::kFloat ? PA_F32 : -1;
}

PyObject* to_slow() { Py_RETURN_NONE; }

template <typename... T>
PyObject* result(int rc, T&&... tensors) {
  if (rc != PA_OK) return PyLong_FromLong(rc);
  PyObject* out = PyTuple_New(sizeof...(T));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  auto put = [&](const Tensor& t) {
    if (t.defined()) {
      PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(out, i++, Py_None);
    }
  };
  (put(tensors), ...);
  return out;
}

// C++ exceptions become the Python ones that torch's own functions raise for
// them (an allocation that fails: torch.OutOfMemoryError).
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// The C entry point without the interpreter's lock: where the queue of launches
// is full a launch waits for the GPU, and other threads go on meanwhile.  (The
// caller holds its tensors.)
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename... P, typename... A>
int launch(int (*entry)(P...), A... args) {
  const Unlocked unlocked;
  return entry(args...);
}

// (q_len, kv_len, block_table, free_pages, page_size, n_tokens)
PyObject* paged_schedule(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 6);
    if (!a.ok) return to_slow();
    const Tensor* q = a.ints(0, 0);
    const Tensor* kv = a.ints(1, q ? q->numel() : 0);
    int64_t stride = 0;
    const Tensor* table = a.table(2, q ? q->numel() : 0, &stride);
    const Tensor* pool = a.ints(3, 0);
    const int64_t page = a.integer(4), tokens = a.integer(5);
    if (!a.ok || tokens < 0 || pool->numel() > kMaxInt || q->numel() > 8192 || overlap(*table, {q, kv, pool}))
      return to_slow();
    const int64_t B = q->numel();
    // one allocation, in the order of the results
    Tensor all = a.make({2 * B + 2 * tokens + 2}, at::kInt), ws = a.make({256}, at::kByte);
    int32_t* p = all.data_ptr<int32_t>();
    const int rc = launch(pa_paged_schedule, q->data_ptr<int32_t>(), kv->data_ptr<int32_t>(), static_cast<int32_t>(B),
                          table->data_ptr<int32_t>(), stride, static_cast<int32_t>(table->size(1)),
                          pool->data_ptr<int32_t>(), static_cast<int32_t>(pool->numel()), static_cast<int32_t>(page),
                          tokens, p, p + B + 1, p + 2 * B + 1, p + 2 * B + 1 + tokens, p + 2 * B + 1 + 2 * tokens,
                          ws.data_ptr(), 256, a.stream());
    if (rc != PA_OK) return PyLong_FromLong(rc);
    // (tensors over its storage, put together here: five dispatched views took as long as the launch)
    auto part = [&](int64_t from, int64_t count) {
      Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
      t.unsafeGetTensorImpl()->set_storage_offset(from);
      t.unsafeGetTensorImpl()->set_sizes_contiguous({count});
      return t;
    };
    return result(rc, part(0, B + 1), part(B + 1, B), part(2 * B + 1, tokens), part(2 * B + 1 + tokens, tokens),
                  part(2 * B + 1 + 2 * tokens, 1), ws);
  });
}

// the cache of `type`, [n_pages][page_size][hkv][d]
bool cache_ok(const Tensor* k, const Tensor* v, at::ScalarType type, int64_t d) {
  return k && v && k->dim() == 4 && k->scalar_type() == type && v->scalar_type() == type && k->sizes() == v->sizes() &&
         k->is_contiguous() && v->is_contiguous() && k->size(3) == d && k->size(0) <= kMaxInt &&
         k->size(1) <= kMaxInt && k->size(0) * k->size(1) <= kMaxInt;
}

// (q, k_new, v_new, positions, slots, k_pages, v_pages, rope_theta, want_k)
PyObject* paged_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 9);
    if (!a.ok || !PyFloat_Check(args[7])) return to_slow();
    const double theta = PyFloat_AS_DOUBLE(args[7]);
    int64_t ldq = 0, ldk = 0, ldv = 0;
    const Tensor* q = a.rows(0, &ldq);
    const Tensor* k = a.rows(1, &ldk);
    const Tensor* v = a.rows(2, &ldv);
    if (!a.ok) return to_slow();
    const int64_t N = k->size(0), hq = q->size(1), hkv = k->size(1), d = k->size(2);
    const Tensor* pos = a.ints(3, N);
    const Tensor* slots = a.ints(4, N);
    const Tensor* kp = a.tensor(5);
    const Tensor* vp = a.tensor(6);
    const int type = dtype_of(*k);
    if (!a.ok || type < 0 || q->scalar_type() != k->scalar_type() || v->scalar_type() != k->scalar_type() ||
        v->sizes() != k->sizes() || q->size(0) != N || q->size(2) != d || N > kMaxInt || hq > kMaxInt ||
        !cache_ok(kp, vp, k->scalar_type(), d) || kp->size(2) != hkv || overlap(*kp, {vp, q, k, v, pos, slots}) ||
        overlap(*vp, {q, k, v, pos, slots}))
      return to_slow();
    Tensor q_out = a.make({N, hq, d}, q->scalar_type()), k_out, ws = a.make({256}, at::kByte);
    const int want_k = PyObject_IsTrue(args[8]);
    if (want_k < 0) return nullptr;   // (its error is set)
    if (want_k) k_out = a.make({N, hkv, d}, k->scalar_type());
    const int rc = launch(pa_paged_append, q->data_ptr(), k->data_ptr(), v->data_ptr(), type, N, ldq, ldk, ldv,
                          static_cast<int32_t>(hq), static_cast<int32_t>(hkv), static_cast<int32_t>(d), theta,
                          pos->data_ptr<int32_t>(), slots->data_ptr<int32_t>(), kp->data_ptr(), vp->data_ptr(),
                          kp->size(0) * kp->size(1), q_out.data_ptr(), k_out.defined() ? k_out.data_ptr() : nullptr,
                          ws.data_ptr(), 256, a.stream());
    return result(rc, q_out, k_out, ws);
  });
}

// (q, k, v, cu_q, want_lse)
PyObject* prompt_attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 5);
    int64_t ldq = 0, ldk = 0, ldv = 0;
    if (!a.ok) return to_slow();
    const Tensor* q = a.rows(0, &ldq);
    const Tensor* k = a.rows(1, &ldk);
    const Tensor* v = a.rows(2, &ldv);
    const Tensor* cu = a.ints(3, 1);
    if (!a.ok) return to_slow();
    const int64_t N = q->size(0), hq = q->size(1), hkv = k->size(1), d = q->size(2), B = cu->numel() - 1;
    const int type = dtype_of(*q);
    if (type < 0 || k->scalar_type() != q->scalar_type() || v->scalar_type() != q->scalar_type() ||
        k->sizes() != v->sizes() || k->size(0) != N || k->size(2) != d || N > kMaxInt || hq > kMaxInt || B > kMaxInt)
      return to_slow();
    const size_t need = pa_prompt_attend_workspace_size(static_cast<int32_t>(B), N, static_cast<int32_t>(hq),
                                                        static_cast<int32_t>(hkv), static_cast<int32_t>(d), type);
    if (need == 0) return to_slow();
    Tensor o = a.make({N, hq, d}, q->scalar_type()), lse, ws = a.make({static_cast<int64_t>(need)}, at::kByte);
    const int want_lse = PyObject_IsTrue(args[4]);
    if (want_lse < 0) return nullptr;
    if (want_lse) lse = a.make({N, hq}, at::kFloat);
    const int rc = launch(pa_prompt_attend, q->data_ptr(), k->data_ptr(), v->data_ptr(), type, N, ldq, ldk, ldv,
                          cu->data_ptr<int32_t>(), static_cast<int32_t>(B), static_cast<int32_t>(hq),
                          static_cast<int32_t>(hkv), static_cast<int32_t>(d), o.data_ptr(),
                          lse.defined() ? lse.data_ptr<float>() : nullptr, ws.data_ptr(), need, a.stream());
    return result(rc, o, lse, ws);
  });
}

// (q, cu_q, kv_len, block_table, k_pages, v_pages, max_q, want_lse)
PyObject* paged_attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 8);
    if (!a.ok) return to_slow();
    int64_t ldq = 0, stride = 0;
    const Tensor* q = a.rows(0, &ldq);
    const Tensor* cu = a.ints(1, 1);
    if (!a.ok) return to_slow();
    const int64_t N = q->size(0), hq = q->size(1), d = q->size(2), B = cu->numel() - 1;
    const Tensor* kv = a.ints(2, B);
    const Tensor* table = a.table(3, B, &stride);
    const Tensor* kp = a.tensor(4);
    const Tensor* vp = a.tensor(5);
    const int64_t max_q = a.integer(6);
    const int type = dtype_of(*q);
    if (!a.ok || type < 0 || !cache_ok(kp, vp, q->scalar_type(), d) || N > kMaxInt || hq > kMaxInt || B > kMaxInt ||
        kp->size(2) > kMaxInt)
      return to_slow();
    const int32_t b = static_cast<int32_t>(B), width = static_cast<int32_t>(table->size(1)),
                  page = static_cast<int32_t>(kp->size(1)), hkv = static_cast<int32_t>(kp->size(2)),
                  mq = static_cast<int32_t>(max_q);
    const size_t need = pa_paged_attend_workspace_size(b, N, mq, width, page, static_cast<int32_t>(hq), hkv,
                                                       static_cast<int32_t>(d), type);
    if (need == 0) return to_slow();
    Tensor o = a.make({N, hq, d}, q->scalar_type()), lse, ws = a.make({static_cast<int64_t>(need)}, at::kByte);
    const int want_lse = PyObject_IsTrue(args[7]);
    if (want_lse < 0) return nullptr;
    if (want_lse) lse = a.make({N, hq}, at::kFloat);
    const int rc = launch(pa_paged_attend, q->data_ptr(), type, N, ldq, cu->data_ptr<int32_t>(),
                          kv->data_ptr<int32_t>(), b, mq, table->data_ptr<int32_t>(), stride, width, page,
                          kp->data_ptr(), vp->data_ptr(), static_cast<int32_t>(kp->size(0)), static_cast<int32_t>(hq),
                          hkv, static_cast<int32_t>(d), o.data_ptr(), lse.defined() ? lse.data_ptr<float>() : nullptr,
                          ws.data_ptr(), need, a.stream());
    return result(rc, o, lse, ws);
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(paged_schedule), FAST(paged_append), FAST(prompt_attend), FAST(paged_attend),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__serving_call() { return PyModule_Create(&module); }
