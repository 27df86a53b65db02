// The usual call of the serving step's operators from Python, natively: tensors are checked and
// turned into the C ABI's pointers, sizes and strides here, which the binding's own checks (ctypes
// calls, one attribute after the other) take two to four times the launch for.  A function answers
// None where anything is unusual or wrong, and has then called nothing: the binding looks again in
// Python, which calls the library too or says what is wrong.  The library's functions come as
// addresses from the binding, so that there is one library.
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "gdn.h"

namespace {

decltype(&gdn_qk_norm_rope) p_qk_norm_rope;
decltype(&gdn_page_plan) p_page_plan;
decltype(&gdn_page_release) p_page_release;
decltype(&gdn_verify_tokens) p_verify_tokens;
PyObject* p_raw_stream;                    // device index -> the current stream

struct Unusual {};                         // thrown: the binding is to look itself

inline void need(bool ok) {
  if (!ok) throw Unusual{};
}
inline const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}
inline bool none(PyObject* o) { return o == Py_None; }

inline long long whole(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  need(!PyErr_Occurred());
  return x;
}
inline int32_t small(PyObject* o) {
  const long long x = whole(o);
  need(x >= INT32_MIN && x <= INT32_MAX);
  return (int32_t)x;
}
inline double real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  need(!PyErr_Occurred());
  return x;
}
inline int32_t size32(int64_t n) {
  need(n >= 0 && n <= INT32_MAX);
  return (int32_t)n;
}

inline bool is(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape,
               const at::Device& device) {
  return t.scalar_type() == type && t.device() == device && t.layout() == at::kStrided &&
         t.sizes().equals(at::IntArrayRef(shape.begin(), shape.size()));
}
// the pointer of a contiguous tensor of this type and shape
inline void* dense(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape,
                   const at::Device& device) {
  need(is(t, type, shape, device) && t.is_contiguous());
  return t.data_ptr();
}
inline void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape,
                   const at::Device& device) {
  return dense(tensor(o), type, shape, device);
}
inline void* dense_or_null(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape,
                           const at::Device& device) {
  return none(o) ? nullptr : dense(tensor(o), type, shape, device);
}
inline gdn_dtype dtype_of(const at::Tensor& t) {
  need(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat);
  return t.scalar_type() == at::kBFloat16 ? GDN_BF16 : GDN_F32;
}
// The token stride of t [n, H, D] with dense heads.
inline int64_t token_stride(const at::Tensor& t, at::ScalarType type, int64_t n, int64_t H, int64_t D,
                            const at::Device& device) {
  need(is(t, type, {n, H, D}, device));
  if (t.is_contiguous()) return H * D;
  const auto s = t.strides();
  need((D == 1 || s[2] == 1) && (H == 1 || s[1] == D));
  return n > 1 ? s[0] : H * D;
}
// The row stride of t [B, T, V] with dense rows at one stride.
inline int64_t row_stride(const at::Tensor& t, at::ScalarType type, int64_t B, int64_t T, int64_t V,
                          const at::Device& device) {
  need(is(t, type, {B, T, V}, device));
  if (t.is_contiguous()) return V;
  const auto s = t.strides();
  need(V == 1 || s[2] == 1);
  if (T == 1) return B > 1 ? s[0] : V;
  need(B == 1 || s[0] == T * s[1]);
  return s[1];
}

inline const at::Tensor& on_gpu(const at::Tensor& t) {
  need(t.device().is_cuda() && t.layout() == at::kStrided);
  return t;
}

void* stream_of(PyObject* o, const at::Device& device) {
  if (!none(o)) return reinterpret_cast<void*>(whole(o));
  PyObject* index = PyLong_FromLong(device.index());
  need(index);
  PyObject* raw = PyObject_CallOneArg(p_raw_stream, index);
  Py_DECREF(index);
  need(raw);
  const long long x = PyLong_AsLongLong(raw);
  Py_DECREF(raw);
  need(!PyErr_Occurred());
  return reinterpret_cast<void*>(x);
}

// Calls the library with the interpreter's lock given up: a launch waits where the queue is full, and
// other threads, and what the stream's host functions need of them, go on meanwhile.  (The arguments
// are made before, under the lock; the caller's frame keeps the tensors.)
template <typename F, typename... A>
gdn_status unlocked(F* f, A... args) {
  struct Unlock {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlock() { PyEval_RestoreThread(state); }
  } unlock;
  return f(args...);
}

// (the body's C++ exceptions end here)
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return PyLong_FromLong((long)body());
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// q k positions phase_steps q_out k_out q_weight k_weight eps interleaved amplitude v k_cache
// v_cache slots k_exp v_exp stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* x, Py_ssize_t count) {
  return guarded([&] {
    need(count == 18);
    const at::Tensor &q = on_gpu(tensor(x[0])), &k = tensor(x[1]), &out = tensor(x[4]);
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    need(q.dim() == 3 && k.dim() == 3);
    const gdn_dtype dt = dtype_of(q);
    const int64_t n = q.size(0), Hq = q.size(1), D = q.size(2), H = k.size(1);
    const auto s = q.strides();
    need(D == 1 || s[2] == 1);
    const int64_t head = Hq == 1 ? D : s[1], token = n > 1 ? s[0] : (Hq - 1) * head + D;
    const int interleaved = PyObject_IsTrue(x[9]);
    need(interleaved >= 0);
    gdn_rope rope = {0, interleaved ? GDN_ROPE_INTERLEAVED : GDN_ROPE_HALF, (float)real(x[10]), nullptr};
    const int32_t* positions = nullptr;
    if (!none(x[3])) {
      const at::Tensor& steps = tensor(x[3]);
      need(steps.dim() == 1 && steps.size(0) <= 128);
      rope.rotary_dim = 2 * (int32_t)steps.size(0);
      void* p = dense(steps, at::kLong, {steps.size(0)}, dev);
      void* at_token = dense(x[2], at::kInt, {n}, dev);
      if (rope.rotary_dim > 0) {
        rope.phase_steps = static_cast<const uint64_t*>(p);
        positions = static_cast<const int32_t*>(at_token);
      }
    }
    gdn_kv_cache cache = {};
    const void* v = nullptr;
    int64_t v_stride = 0;
    const int32_t* slots = nullptr;
    const bool cached = !none(x[12]);
    if (cached) {
      const at::Tensor& kc = tensor(x[12]);
      need(kc.dim() == 4);
      const bool f8 = kc.scalar_type() == at::kFloat8_e4m3fn;
      need(f8 || kc.scalar_type() == at::kBFloat16);
      const int64_t pages = kc.size(0), heads = kc.size(1), page = kc.size(2), d = kc.size(3);
      cache.num_pages = size32(pages), cache.page_size = size32(page);
      cache.num_kv_heads = size32(heads), cache.head_dim = size32(d);
      cache.format = f8 ? GDN_KV_E4M3 : GDN_KV_BF16;
      cache.k = dense(kc, kc.scalar_type(), {pages, heads, page, d}, dev);
      cache.v = dense(x[13], kc.scalar_type(), {pages, heads, page, d}, dev);
      need(f8 == !none(x[15]) && f8 == !none(x[16]));
      cache.k_exp = (uint8_t*)dense_or_null(x[15], at::kByte, {pages, heads, page}, dev);
      cache.v_exp = (uint8_t*)dense_or_null(x[16], at::kByte, {pages, heads, page}, dev);
      const at::Tensor& values = tensor(x[11]);
      v_stride = token_stride(values, type, n, H, D, dev);
      v = values.data_ptr();
      slots = (const int32_t*)dense(x[14], at::kInt, {n}, dev);
    } else {
      need(!none(x[5]) && none(x[11]) && none(x[13]) && none(x[14]));
    }
    return unlocked(
        p_qk_norm_rope, size32(n), size32(Hq), size32(H), size32(D), dt, q.data_ptr(), token, head,
        k.data_ptr(), token_stride(k, type, n, H, D, dev), (const float*)dense_or_null(x[6], at::kFloat, {D}, dev),
        (const float*)dense_or_null(x[7], at::kFloat, {D}, dev), (float)real(x[8]), positions, &rope,
        out.data_ptr(), token_stride(out, type, n, Hq, D, dev),
        dense_or_null(x[5], type, {n, H, D}, dev), cached ? &cache : nullptr, v, v_stride, slots,
        stream_of(x[17], dev));
  });
}

// table held free_pages free_count page_size
gdn_page_pool pool_of(PyObject* const* x, at::Device* device) {
  const at::Tensor &table = on_gpu(tensor(x[0])), &free_pages = tensor(x[2]);
  need(table.dim() == 2 && free_pages.dim() == 1);
  const at::Device dev = table.device();
  *device = dev;
  const int64_t rows = table.size(0), columns = table.size(1), pages = free_pages.size(0);
  return gdn_page_pool{size32(pages), small(x[4]), size32(rows), size32(columns),
                       (int32_t*)dense(table, at::kInt, {rows, columns}, dev),
                       (int32_t*)dense(x[1], at::kInt, {rows}, dev),
                       (int32_t*)dense(free_pages, at::kInt, {pages}, dev),
                       (int32_t*)dense(x[3], at::kInt, {1}, dev)};
}

// kv_len new_len slots positions cu_seqlens kv_len_out pages table held free_pages free_count
// page_size rows position_offset stream
PyObject* page_plan(PyObject*, PyObject* const* x, Py_ssize_t count) {
  return guarded([&] {
    need(count == 15);
    at::Device dev(at::kCPU);
    const gdn_page_pool pool = pool_of(x + 7, &dev);
    const at::Tensor& kv = tensor(x[0]);
    need(kv.dim() == 1);
    const int64_t B = kv.size(0);
    need(!none(x[12]) || B <= pool.num_rows);
    int64_t capacity = INT32_MAX;          // (nothing to be written a token)
    for (PyObject* o : {x[3], x[2]})
      if (!none(o)) need(tensor(o).dim() == 1), capacity = tensor(o).size(0);
    return unlocked(p_page_plan, &pool, size32(B),
                    (const int32_t*)dense_or_null(x[12], at::kInt, {B}, dev),
                    (const int32_t*)dense(kv, at::kInt, {B}, dev),
                    (const int32_t*)dense(x[1], at::kInt, {B}, dev), size32(capacity), small(x[13]),
                    (int32_t*)dense_or_null(x[2], at::kInt, {capacity}, dev),
                    (int32_t*)dense_or_null(x[3], at::kInt, {capacity}, dev),
                    (int32_t*)dense_or_null(x[4], at::kInt, {B + 1}, dev),
                    (int32_t*)dense_or_null(x[5], at::kInt, {B}, dev),
                    (int32_t*)dense_or_null(x[6], at::kInt, {B, pool.max_pages}, dev),
                    stream_of(x[14], dev));
  });
}

// keep_len table held free_pages free_count page_size rows stream
PyObject* page_release(PyObject*, PyObject* const* x, Py_ssize_t count) {
  return guarded([&] {
    need(count == 8);
    at::Device dev(at::kCPU);
    const gdn_page_pool pool = pool_of(x + 1, &dev);
    const at::Tensor& keep = tensor(x[0]);
    need(keep.dim() == 1);
    const int64_t B = keep.size(0);
    need(!none(x[6]) || B <= pool.num_rows);
    return unlocked(p_page_release, &pool, size32(B),
                    (const int32_t*)dense_or_null(x[6], at::kInt, {B}, dev),
                    (const int32_t*)dense(keep, at::kInt, {B}, dev), stream_of(x[7], dev));
  });
}

// target_logits tokens accepted clocks draft_ids draft_logits accept_u scale logprobs workspace
// stream
PyObject* verify_tokens(PyObject*, PyObject* const* x, Py_ssize_t count) {
  return guarded([&] {
    need(count == 11);
    const at::Tensor &target = on_gpu(tensor(x[0])), &workspace = tensor(x[9]);
    const at::Device dev = target.device();
    const at::ScalarType type = target.scalar_type();
    need(target.dim() == 3);
    const gdn_dtype dt = dtype_of(target);
    const int64_t B = target.size(0), T = target.size(1) - 1, V = target.size(2);
    need(T >= 0 && workspace.device() == dev && workspace.layout() == at::kStrided &&
         workspace.is_contiguous());
    const void *ids = nullptr, *draft = nullptr, *u = nullptr;
    int64_t draft_stride = 0;
    if (T > 0) {
      ids = dense(x[4], at::kInt, {B, T}, dev);
      u = dense(x[6], at::kFloat, {B, T}, dev);
      if (!none(x[5])) {
        draft_stride = row_stride(tensor(x[5]), type, B, T, V, dev);
        draft = tensor(x[5]).data_ptr();
      }
    } else {
      need(none(x[4]) && none(x[5]) && none(x[6]));
    }
    return unlocked(p_verify_tokens, size32(B), size32(T), size32(V), dt, target.data_ptr(),
                    row_stride(target, type, B, T + 1, V, dev), (const int32_t*)ids, draft,
                    draft_stride, (const float*)u, (const float*)dense(x[3], at::kFloat, {B, V}, dev),
                    (const float*)dense_or_null(x[7], at::kFloat, {B}, dev),
                    (int32_t*)dense(x[1], at::kInt, {B, T + 1}, dev),
                    (int32_t*)dense(x[2], at::kInt, {B}, dev),
                    (float*)dense_or_null(x[8], at::kFloat, {B, T + 1}, dev), workspace.data_ptr(),
                    workspace.nbytes(), stream_of(x[10], dev));
  });
}

// The library's functions, in this order, and what gives a device's current stream.
PyObject* bind(PyObject*, PyObject* const* x, Py_ssize_t count) {
  if (count != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses and a callable");
    return nullptr;
  }
  void* at[4];
  for (int i = 0; i < 4; ++i) {
    at[i] = PyLong_AsVoidPtr(x[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_qk_norm_rope = reinterpret_cast<decltype(p_qk_norm_rope)>(at[0]);
  p_page_plan = reinterpret_cast<decltype(p_page_plan)>(at[1]);
  p_page_release = reinterpret_cast<decltype(p_page_release)>(at[2]);
  p_verify_tokens = reinterpret_cast<decltype(p_verify_tokens)>(at[3]);
  Py_INCREF(x[4]);
  p_raw_stream = x[4];
  Py_RETURN_NONE;
}

#define GDN_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {GDN_FAST(bind),       GDN_FAST(qk_norm_rope), GDN_FAST(page_plan),
                          GDN_FAST(page_release), GDN_FAST(verify_tokens), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr,
                       nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&kModule);
  // (the binding leaves a module of another torch alone)
  if (m && PyModule_AddStringConstant(m, "torch_version", GDN_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
