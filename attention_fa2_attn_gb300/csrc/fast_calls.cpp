// fast_calls.cpp -- the calls of a decode step, from Python objects to the C ABI in one go.
//
// Between the layers of a decode step the host's time is the call's time: the kernels of
// fa_paged_plan or fa_rope_append_paged run for 4 us, and reading twenty attributes of
// tensors, making the outputs and marshalling twenty arguments in Python took 15 to 20.
// Each function here takes the arguments of the Python call of the same name (without its
// outputs, or with those of the rotary calls), tests them, makes the outputs that are not
// given and calls the library. It answers
//   - a tuple of the outputs, or one output,
//   - an int, the library's status, where that is not FA_OK,
//   - None where an argument is not plainly right: the Python call then goes through its
//     own checks, which name the argument, or take what these tests do not know.
// Nothing is decided here that the Python calls would decide otherwise.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/CUDAContextLight.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <climits>
#include <cmath>
#include <utility>

#include "../../include/fa_gb300.h"

namespace {

using at::Tensor;

// The tensor in `o`, or null: exact torch.Tensors only, subclasses may mean something else.
const Tensor* tensor_of(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// The current device, where `t` is on some GPU; else one that no tensor is on.
int device_for(const Tensor& t) { return t.is_cuda() ? c10::cuda::current_device() : -2; }

bool dense(const Tensor& t, at::ScalarType type, int dim, int dev) {
  return t.is_cuda() && t.layout() == at::kStrided && t.scalar_type() == type && t.dim() == dim &&
         t.get_device() == dev && t.is_contiguous();
}

bool fits(int64_t n) { return n >= 0 && n <= INT_MAX; }

// [B][heads][T][d] with dense rows; every size an int
bool rows(const Tensor& t, at::ScalarType type, int dev) {
  return t.is_cuda() && t.layout() == at::kStrided && t.scalar_type() == type && t.dim() == 4 &&
         t.get_device() == dev && t.stride(3) == 1 && fits(t.size(0)) && fits(t.size(1)) && fits(t.size(2)) &&
         fits(t.size(3));
}

bool same_sizes(const Tensor& a, const Tensor& b) { return a.sizes() == b.sizes(); }

Tensor make(at::IntArrayRef sizes, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

// Dense int tensors as parts of one allocation, each at a 16-byte border: an allocation costs
// more than all else that a step call does on the host but the launch.
template <size_t N>
std::array<Tensor, N> make_ints(const std::array<std::array<int64_t, 3>, N>& sizes, const std::array<int, N>& dims,
                                int dev) {
  std::array<int64_t, N> at;
  int64_t total = 0;
  for (size_t i = 0; i < N; ++i) {
    int64_t n = 1;
    for (int k = 0; k < dims[i]; ++k) n *= sizes[i][k];
    at[i] = total;
    total += (n + 3) & ~int64_t(3);
  }
  const Tensor all = make({total}, at::kInt, dev);
  std::array<Tensor, N> out;
  for (size_t i = 0; i < N; ++i) {
    out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
    out[i].unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(sizes[i].data(), dims[i]));
    out[i].unsafeGetTensorImpl()->set_storage_offset(at[i]);
  }
  return out;
}

// The interpreter is released from here to the end of the scope: an allocation may wait for
// the driver, and a launch for room in the stream's queue. Tensors of the arguments are kept by
// the caller's frame.
struct NoInterpreter {
  PyThreadState* state = PyEval_SaveThread();
  ~NoInterpreter() { PyEval_RestoreThread(state); }
};

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

bool int_of(PyObject* o, int* out) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (overflow || v < INT_MIN || v > INT_MAX) return false;
  *out = static_cast<int>(v);
  return true;
}

bool float_of(PyObject* o, float* out) {
  if (!PyFloat_CheckExact(o)) return false;
  *out = static_cast<float>(PyFloat_AS_DOUBLE(o));
  return true;
}

bool flag_of(PyObject* o, bool* out) {
  if (!PyBool_Check(o)) return false;
  *out = o == Py_True;
  return true;
}

PyObject* answer(fa_status st, std::initializer_list<Tensor> outs) {
  if (st != FA_OK) return PyLong_FromLong(st);
  if (outs.size() == 1) return THPVariable_Wrap(*outs.begin());
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : outs) {
    PyObject* w = THPVariable_Wrap(t);
    if (!w) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, w);
  }
  return r;
}

const int* ints(const Tensor& t) { return static_cast<const int*>(t.const_data_ptr()); }
int* ints_out(const Tensor& t) { return static_cast<int*>(t.mutable_data_ptr()); }

// (cached_lens, new_lens, free_pages, block_table, T, align_end)
PyObject* paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int T = 0;
  bool end = false;
  const Tensor *cached, *fresh, *free_pages, *table;
  if (n != 6 || !(cached = tensor_of(a[0])) || !(fresh = tensor_of(a[1])) || !(free_pages = tensor_of(a[2])) ||
      !(table = tensor_of(a[3])) || !int_of(a[4], &T) || T < 1 || !flag_of(a[5], &end))
    Py_RETURN_NONE;
  const int dev = device_for(*table);
  if (!dense(*table, at::kInt, 2, dev) || !dense(*cached, at::kInt, 1, dev) || !dense(*fresh, at::kInt, 1, dev) ||
      !dense(*free_pages, at::kInt, 1, dev))
    Py_RETURN_NONE;
  const int64_t B = table->size(0), pages = table->size(1), F = free_pages->size(0);
  if (cached->size(0) != B || fresh->size(0) != B || !fits(B) || !fits(pages) || !fits(F) || !fits(B * T) ||
      T > FA_PLAN_MAX_T)  // refused before its outputs are made
    Py_RETURN_NONE;
  std::array<Tensor, 4> out;  // seqlens, slots, positions, pages used
  fa_status st;
  {
    NoInterpreter released;
    out = make_ints<4>({{{B, 0, 0}, {B, T, 0}, {B, T, 0}, {1, 0, 0}}}, {1, 2, 2, 1}, dev);
    st = fa_paged_plan(ints(*cached), ints(*fresh), ints(*free_pages), static_cast<int>(F), ints_out(*table),
                       ints_out(out[0]), ints_out(out[1]), ints_out(out[2]), ints_out(out[3]), static_cast<int>(B), T,
                       static_cast<int>(pages), 16, end, stream_of(dev));
  }
  return answer(st, {out[0], out[1], out[2], out[3]});
  END_HANDLE_TH_ERRORS
}

// (parents, seqlens, tree_lens or None)
PyObject* tree_mask(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *parents, *seqlens, *lens = nullptr;
  if (n != 3 || !(parents = tensor_of(a[0])) || !(seqlens = tensor_of(a[1])) ||
      (a[2] != Py_None && !(lens = tensor_of(a[2]))))
    Py_RETURN_NONE;
  const int dev = device_for(*parents);
  if (!dense(*parents, at::kInt, 2, dev) || !dense(*seqlens, at::kInt, 1, dev) ||
      (lens && !dense(*lens, at::kInt, 1, dev)))
    Py_RETURN_NONE;
  const int64_t B = parents->size(0), T = parents->size(1);
  if (seqlens->size(0) != B || (lens && lens->size(0) != B) || B > FA_TREE_MASK_MAX_B || T > FA_TREE_MASK_MAX_T)
    Py_RETURN_NONE;
  std::array<Tensor, 2> out;  // mask, positions
  fa_status st;
  {
    NoInterpreter released;
    out = make_ints<2>({{{B, T, (T + 31) / 32}, {B, T, 0}}}, {3, 2}, dev);
    st = fa_tree_mask(ints(*parents), ints(*seqlens), lens ? ints(*lens) : nullptr, ints_out(out[0]), ints_out(out[1]),
                      static_cast<int>(B), static_cast<int>(T), stream_of(dev));
  }
  return answer(st, {out[0], out[1]});
  END_HANDLE_TH_ERRORS
}

bool angles(const Tensor& positions, const Tensor& inv_freq, int64_t B, int64_t T, int dev, bool* shared) {
  *shared = positions.dim() == 1;
  return dense(positions, at::kInt, *shared ? 1 : 2, dev) && dense(inv_freq, at::kDouble, 1, dev) &&
         (*shared || positions.size(0) == B) && positions.size(positions.dim() - 1) == T &&
         inv_freq.size(0) <= INT_MAX / 2;
}

// A caller's output for rows like `like`, no two of its rows on one another.
bool rows_out(const Tensor& t, const Tensor& like, int dev) {
  if (!rows(t, like.scalar_type(), dev) || !same_sizes(t, like)) return false;
  std::array<std::pair<int64_t, int64_t>, 3> dims;
  for (int i = 0; i < 3; ++i) dims[i] = {t.size(i) > 1 ? t.stride(i) : -1, t.size(i)};
  std::sort(dims.begin(), dims.end());
  int64_t reach = t.size(3);  // values up to the end of the rows of the dimensions so far
  for (const auto& d : dims) {
    if (d.first < 0) continue;  // a dimension of one
    if (d.first < reach) return false;
    reach += d.first * (d.second - 1);
  }
  return true;
}

// (q, k or None, positions, inv_freq, interleaved, mscale, backward, q_out or None, k_out or None)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *q, *k = nullptr, *positions, *inv_freq;
  bool inter = false, back = false, shared = false;
  float mscale = 1.f;
  const Tensor *q_out = nullptr, *k_out = nullptr;
  if (n != 9 || !(q = tensor_of(a[0])) || (a[1] != Py_None && !(k = tensor_of(a[1]))) ||
      (a[7] != Py_None && !(q_out = tensor_of(a[7]))) || (a[8] != Py_None && !(k_out = tensor_of(a[8]))) ||
      !(positions = tensor_of(a[2])) || !(inv_freq = tensor_of(a[3])) || !flag_of(a[4], &inter) ||
      !float_of(a[5], &mscale) || !flag_of(a[6], &back))
    Py_RETURN_NONE;
  const int dev = device_for(*q);
  const at::ScalarType type = q->scalar_type();
  if ((type != at::kBFloat16 && type != at::kFloat) || !rows(*q, type, dev) || (k && !rows(*k, type, dev)))
    Py_RETURN_NONE;
  const int64_t B = q->size(0), H = q->size(1), T = q->size(2), d = q->size(3), Hk = k ? k->size(1) : 0;
  if (!angles(*positions, *inv_freq, B, T, dev, &shared) ||
      (k && (k->size(0) != B || k->size(2) != T || k->size(3) != d || Hk < 1)))
    Py_RETURN_NONE;
  if ((q_out && !rows_out(*q_out, *q, dev)) || (k_out && !(k && rows_out(*k_out, *k, dev)))) Py_RETURN_NONE;
  Tensor qo, ko;
  fa_status st;
  {
    NoInterpreter released;
    qo = q_out ? *q_out : make({B, H, T, d}, type, dev);
    if (k) ko = k_out ? *k_out : make({B, Hk, T, d}, type, dev);
    const long long s[12] = {q->stride(0),  q->stride(1),  q->stride(2),  qo.stride(0), qo.stride(1), qo.stride(2),
                             k ? k->stride(0) : 0, k ? k->stride(1) : 0, k ? k->stride(2) : 0,
                             k ? ko.stride(0) : 0, k ? ko.stride(1) : 0, k ? ko.stride(2) : 0};
    st = (back ? fa_rope_bwd : fa_rope)(
        q->const_data_ptr(), k ? k->const_data_ptr() : nullptr, qo.mutable_data_ptr(),
        k ? ko.mutable_data_ptr() : nullptr, s, ints(*positions), shared,
        static_cast<const double*>(inv_freq->const_data_ptr()), static_cast<int>(B), static_cast<int>(H),
        static_cast<int>(Hk), static_cast<int>(T), static_cast<int>(d), static_cast<int>(2 * inv_freq->size(0)), inter,
        mscale, type == at::kFloat ? FA_DTYPE_F32 : FA_DTYPE_BF16, stream_of(dev));
  }
  if (k || st != FA_OK) return answer(st, {qo, ko});
  PyObject* w = THPVariable_Wrap(qo);
  if (!w) return nullptr;
  PyObject* r = PyTuple_Pack(2, w, Py_None);
  Py_DECREF(w);
  return r;
  END_HANDLE_TH_ERRORS
}

// (q, k, v, positions, slots, inv_freq, k_pages, v_pages, interleaved, mscale, q_out or None)
PyObject* rope_append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor* t[8];
  bool inter = false, shared = false;
  float mscale = 1.f;
  const Tensor* q_out = nullptr;
  if (n != 11 || !flag_of(a[8], &inter) || !float_of(a[9], &mscale) ||
      (a[10] != Py_None && !(q_out = tensor_of(a[10]))))
    Py_RETURN_NONE;
  for (int i = 0; i < 8; ++i)
    if (!(t[i] = tensor_of(a[i]))) Py_RETURN_NONE;
  const Tensor &q = *t[0], &k = *t[1], &v = *t[2], &positions = *t[3], &slots = *t[4], &inv_freq = *t[5], &kp = *t[6],
               &vp = *t[7];
  const int dev = device_for(q);
  if (!rows(q, at::kBFloat16, dev) || !rows(k, at::kBFloat16, dev) || !rows(v, at::kBFloat16, dev) ||
      !dense(kp, at::kBFloat16, 4, dev) || !dense(vp, at::kBFloat16, 4, dev) || !dense(slots, at::kInt, 2, dev))
    Py_RETURN_NONE;
  const int64_t B = q.size(0), H = q.size(1), T = q.size(2), d = q.size(3), P = kp.size(0), Hkv = kp.size(2);
  if (!angles(positions, inv_freq, B, T, dev, &shared) || shared || !same_sizes(slots, positions) ||
      !same_sizes(k, v) || !same_sizes(kp, vp) || k.size(0) != B || k.size(1) != Hkv || k.size(2) != T ||
      k.size(3) != d || kp.size(3) != d || !fits(P) || !fits(kp.size(1)))
    Py_RETURN_NONE;
  if (q_out && !rows_out(*q_out, q, dev)) Py_RETURN_NONE;
  Tensor qo;
  fa_status st;
  {
    NoInterpreter released;
    qo = q_out ? *q_out : make({B, H, T, d}, at::kBFloat16, dev);
    const long long s[12] = {q.stride(0), q.stride(1), q.stride(2), qo.stride(0), qo.stride(1), qo.stride(2),
                             k.stride(0), k.stride(1), k.stride(2), v.stride(0),  v.stride(1),  v.stride(2)};
    st = fa_rope_append_paged(
        q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), qo.mutable_data_ptr(), s, ints(positions),
        ints(slots), static_cast<const double*>(inv_freq.const_data_ptr()), kp.mutable_data_ptr(),
        vp.mutable_data_ptr(), static_cast<int>(B), static_cast<int>(H), static_cast<int>(Hkv), static_cast<int>(T),
        static_cast<int>(kp.size(1)), static_cast<int>(P), static_cast<int>(d), static_cast<int>(2 * inv_freq.size(0)),
        inter, mscale, stream_of(dev));
  }
  return answer(st, {qo});
  END_HANDLE_TH_ERRORS
}

// (q, k_pages, v_pages, block_table, seqlens, tree_mask, tree_lens or None, scale or None)
PyObject* tree_decode_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor* t[6];
  const Tensor* lens = nullptr;
  float scale = 0.f;
  if (n != 8 || (a[6] != Py_None && !(lens = tensor_of(a[6]))) || (a[7] != Py_None && !float_of(a[7], &scale)))
    Py_RETURN_NONE;
  for (int i = 0; i < 6; ++i)
    if (!(t[i] = tensor_of(a[i]))) Py_RETURN_NONE;
  const Tensor &q = *t[0], &kp = *t[1], &vp = *t[2], &table = *t[3], &seqlens = *t[4], &mask = *t[5];
  const int dev = device_for(q);
  const bool shared = mask.dim() == 2;
  if (!dense(q, at::kBFloat16, 4, dev) || !dense(kp, at::kBFloat16, 4, dev) || !dense(vp, at::kBFloat16, 4, dev) ||
      !dense(table, at::kInt, 2, dev) || !dense(seqlens, at::kInt, 1, dev) ||
      !dense(mask, at::kInt, shared ? 2 : 3, dev) || (lens && !dense(*lens, at::kInt, 1, dev)))
    Py_RETURN_NONE;
  const int64_t B = q.size(0), Hq = q.size(1), T = q.size(2), d = q.size(3), P = kp.size(0), Hkv = kp.size(2),
                pages = table.size(1);
  if (!same_sizes(kp, vp) || kp.size(3) != d || table.size(0) != B || seqlens.size(0) != B ||
      (lens && lens->size(0) != B) || (!shared && mask.size(0) != B) || mask.size(shared ? 0 : 1) != T ||
      mask.size(shared ? 1 : 2) != (T + 31) / 32 || !fits(B) || !fits(Hq) || !fits(T) || !fits(d) || !fits(P) ||
      !fits(Hkv) || !fits(pages) || !fits(kp.size(1)))
    Py_RETURN_NONE;
  if (a[7] == Py_None) scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  Tensor o, lse;
  fa_status st;
  {
    NoInterpreter released;
    const int sms = at::cuda::getCurrentDeviceProperties()->multiProcessorCount;
    const size_t bytes =
        fa_tree_workspace_bytes(static_cast<int>(B), static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(T),
                                static_cast<int>(pages), static_cast<int>(d), sms);
    const Tensor ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
    o = make({B, Hq, T, d}, at::kBFloat16, dev);
    lse = make({B, Hq, T}, at::kFloat, dev);
    st = fa_tree_decode_paged(
        q.const_data_ptr(), kp.const_data_ptr(), vp.const_data_ptr(), ints(table), ints(seqlens), ints(mask), shared,
        lens ? ints(*lens) : nullptr, o.mutable_data_ptr(), static_cast<float*>(lse.mutable_data_ptr()),
        static_cast<int>(B), static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(T), static_cast<int>(pages),
        static_cast<int>(kp.size(1)), static_cast<int>(P), static_cast<int>(d), scale, ws.mutable_data_ptr(), bytes,
        stream_of(dev));
  }
  return answer(st, {o, lse});
  END_HANDLE_TH_ERRORS
}

#define FA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_METHOD(paged_plan), FA_METHOD(tree_mask), FA_METHOD(rope), FA_METHOD(rope_append_paged),
                         FA_METHOD(tree_decode_paged), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", "Step calls from Python objects to the C ABI.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) { return PyModule_Create(&module); }
