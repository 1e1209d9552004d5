// fastcall.cpp -- repeated calls of include/gl_delta.h and include/gl_ssm.h from Python.
//
// The checks of a call's tensors, its descriptor and the sizes of what it
// returns depend on shapes, strides, types and devices only, and a decoding loop
// makes thousands of calls that agree in all of them: in Python, looking that
// up took longer (8 us of a one-token step) than the launch.  A `Calls` object
// keeps the descriptors that delta.py or ssm.py has checked for one kind of call and its
// numbers (scale, flags, ...), compares the tensors at hand with what they were
// recorded for, allocates the outputs and calls the library: one kind of call,
// one place, no arithmetic.  Nothing is kept of the tensors but their shapes,
// strides, types and devices.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/core/DeviceGuard.h>

#include <cstdint>
#include <exception>
#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "gl_delta.h"
#include "gl_ssm.h"

namespace {

enum Kind { DELTA_FWD, DELTA_BWD, DELTA_STEP, QK_FWD, QK_BWD,
            CONV_FWD, CONV_BWD, CONV_STEP, SSM_FWD, SSM_BWD, SSM_STEP, ADD_FWD, ADD_BWD, GATE_FWD, GATE_BWD, KINDS };
constexpr int kInputs[KINDS] = {7, 10, 8, 7, 9, 5, 7, 5, 10, 13, 10, 5, 7, 3, 4};
constexpr int kOutputs[KINDS] = {3, 6, 1, 2, 4, 2, 4, 1, 3, 9, 1, 2, 5, 1, 3};
constexpr int kMostInputs = 13, kMostOutputs = 9;
constexpr size_t kMostRecords = 32;

struct Shape {  // of an input, or of an output to be made
  bool there = false;
  at::ScalarType type = at::kFloat;
  std::vector<int64_t> sizes, strides;
  bool is(const at::Tensor& t) const {
    return t.scalar_type() == type && t.sizes() == at::IntArrayRef(sizes) && t.strides() == at::IntArrayRef(strides);
  }
};

struct Record {
  Shape in[kMostInputs], out[kMostOutputs];
  c10::Device device{c10::kCPU};
  PyObject* desc = nullptr;  // keeps the descriptor alive
  const void* d = nullptr;
  int64_t ws = 0, count = 0;  // workspace bytes; states of a step
  ~Record() { Py_XDECREF(desc); }
};

struct Calls {
  PyObject_HEAD
  int kind;
  void* fn;
  std::vector<std::shared_ptr<Record>>* records;
};

// Runs f; a C++ exception becomes a Python one.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

bool read_ints(PyObject* seq, std::vector<int64_t>& v) {
  PyObject* fast = PySequence_Fast(seq, "a sequence of integers");
  if (!fast) return false;
  for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(fast); ++i)
    v.push_back(PyLong_AsLongLong(PySequence_Fast_GET_ITEM(fast, i)));
  Py_DECREF(fast);
  return !PyErr_Occurred();
}

// The tensors match r: same ones absent, all on r's device, and as recorded.
bool matches(const Record& r, PyObject* const* args, int n) {
  for (int i = 0; i < n; ++i) {
    if (args[i] == Py_None) {
      if (r.in[i].there) return false;
      continue;
    }
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!r.in[i].there || t.device() != r.device || !r.in[i].is(t)) return false;
  }
  return true;
}

int launch(const Calls* c, const Record& r, int64_t pos0, void* const* in, void* const* out, void* ws, void* stream) {
  const size_t nb = static_cast<size_t>(r.ws);
  const auto* dd = static_cast<const gl_delta_desc_t*>(r.d);
  gl_qknorm_desc_t q;
  const gl_qknorm_desc_t* dq = &q;
  if (c->kind == QK_FWD || c->kind == QK_BWD) {
    q = *static_cast<const gl_qknorm_desc_t*>(r.d);
    q.pos0 = pos0;
  }
  const auto i32 = [&](int i) { return static_cast<const int32_t*>(in[i]); };
  switch (c->kind) {
    case DELTA_FWD:  // q k v log_alpha beta state cu | y state saved
      return reinterpret_cast<decltype(&gl_delta_fwd)>(c->fn)(dd, in[0], in[1], in[2], in[3], in[4], in[5], i32(6), out[0],
                                                              out[1], out[2], ws, nb, stream);
    case DELTA_BWD:  // q k v log_alpha beta state cu dy dstate saved | dq dk dv dlog_alpha dbeta dstate
      return reinterpret_cast<decltype(&gl_delta_bwd)>(c->fn)(dd, in[0], in[1], in[2], in[3], in[4], in[5], i32(6), in[7],
                                                              in[8], in[9], out[0], out[1], out[2], out[3], out[4],
                                                              out[5], ws, nb, stream);
    case DELTA_STEP:  // q k v log_alpha beta slots state y | y
      return reinterpret_cast<decltype(&gl_delta_step)>(c->fn)(dd, in[0], in[1], in[2], in[3], in[4], i32(5), r.count,
                                                               in[6], in[7] ? in[7] : out[0], stream);
    case QK_FWD:  // q k wq wk cos sin pos | q k
      return reinterpret_cast<decltype(&gl_qknorm_rope_fwd)>(c->fn)(dq, in[0], in[1], in[2], in[3], in[4], in[5], i32(6),
                                                                    out[0], out[1], stream);
    case CONV_FWD:  // x w bias state cu | y state
      return reinterpret_cast<decltype(&gl_conv_fwd)>(c->fn)(static_cast<const gl_conv_desc_t*>(r.d), in[0], in[1], in[2],
                                                             in[3], i32(4), out[0], out[1], stream);
    case CONV_BWD:  // x w bias state cu dy dstate | dx dw dbias dstate
      return reinterpret_cast<decltype(&gl_conv_bwd)>(c->fn)(static_cast<const gl_conv_desc_t*>(r.d), in[0], in[1], in[2],
                                                             in[3], i32(4), in[5], in[6], out[0], out[1], out[2], out[3],
                                                             ws, nb, stream);
    case CONV_STEP:  // x w bias slots state | y
      return reinterpret_cast<decltype(&gl_conv_step)>(c->fn)(static_cast<const gl_conv_desc_t*>(r.d), in[0], in[1],
                                                              in[2], i32(3), r.count, in[4], out[0], stream);
    case SSM_FWD:  // x dt A B C skip z dt_bias state cu | y state saved
      return reinterpret_cast<decltype(&gl_ssm_fwd)>(c->fn)(static_cast<const gl_ssm_desc_t*>(r.d), in[0], in[1], in[2],
                                                            in[3], in[4], in[5], in[6], in[7], in[8], i32(9), out[0],
                                                            out[1], out[2], ws, nb, stream);
    case SSM_BWD:  // x dt A B C skip z dt_bias state cu dy dstate saved | dx ddt dA dB dC dskip dz ddt_bias dstate
      return reinterpret_cast<decltype(&gl_ssm_bwd)>(c->fn)(
          static_cast<const gl_ssm_desc_t*>(r.d), in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7], in[8], i32(9),
          in[10], in[11], in[12], out[0], out[1], out[2], out[3], out[4], out[5], out[6], out[7], out[8], ws, nb, stream);
    case SSM_STEP:  // x dt A B C skip z dt_bias slots state | y
      return reinterpret_cast<decltype(&gl_ssm_step)>(c->fn)(static_cast<const gl_ssm_desc_t*>(r.d), in[0], in[1], in[2],
                                                             in[3], in[4], in[5], in[6], in[7], i32(8), r.count, in[9],
                                                             out[0], stream);
    case ADD_FWD:  // x r w wx scale | n r
      return reinterpret_cast<decltype(&gl_addnorm_fwd)>(c->fn)(static_cast<const gl_addnorm_desc_t*>(r.d), in[0], in[1],
                                                                in[2], in[3], in[4], out[0], out[1], stream);
    case ADD_BWD:  // x r w wx scale dn dr | dx dr dw dwx dscale
      return reinterpret_cast<decltype(&gl_addnorm_bwd)>(c->fn)(
          static_cast<const gl_addnorm_desc_t*>(r.d), in[0], in[1], in[2], in[3], in[4], in[5], in[6], out[0], out[1],
          out[2], out[3], out[4], ws, nb, stream);
    case GATE_FWD:  // x z w | y
      return reinterpret_cast<decltype(&gl_gatenorm_fwd)>(c->fn)(static_cast<const gl_gatenorm_desc_t*>(r.d), in[0],
                                                                 in[1], in[2], out[0], stream);
    case GATE_BWD:  // x z w dy | dx dz dw
      return reinterpret_cast<decltype(&gl_gatenorm_bwd)>(c->fn)(static_cast<const gl_gatenorm_desc_t*>(r.d), in[0],
                                                                 in[1], in[2], in[3], out[0], out[1], out[2], ws, nb,
                                                                 stream);
    default:  // q k wq wk cos sin pos dqn dkn | dq dk dwq dwk
      return reinterpret_cast<decltype(&gl_qknorm_rope_bwd)>(c->fn)(dq, in[0], in[1], in[2], in[3], in[4], in[5], i32(6),
                                                                    in[7], in[8], out[0], out[1], out[2], out[3], ws, nb,
                                                                    stream);
  }
}

// call(stream, pos0, *tensors): None if no record matches, the status if the library
// refused, else the tuple of outputs.
PyObject* calls_call(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  auto* c = reinterpret_cast<Calls*>(self);
  return guarded([&]() -> PyObject* {
    const int ni = kInputs[c->kind], no = kOutputs[c->kind];
    if (n != ni + 2) {
      PyErr_SetString(PyExc_TypeError, "wrong number of tensors");
      return nullptr;
    }
    void* stream = PyLong_AsVoidPtr(args[0]);
    const int64_t pos0 = PyLong_AsLongLong(args[1]);
    if (PyErr_Occurred()) return nullptr;
    args += 2;
    for (int i = 0; i < ni; ++i)
      if (args[i] != Py_None && !THPVariable_Check(args[i])) Py_RETURN_NONE;  // refused by the full checks
    std::shared_ptr<const Record> r;  // also while other threads run
    auto& rs = *c->records;
    for (size_t k = 0; k < rs.size(); ++k)
      if (matches(*rs[k], args, ni)) {
        if (k) std::swap(rs[k], rs[0]);
        r = rs[0];
        break;
      }
    if (!r) Py_RETURN_NONE;
    const c10::DeviceGuard guard(r->device);
    void *in[kMostInputs] = {}, *out[kMostOutputs] = {};
    for (int i = 0; i < ni; ++i)
      if (args[i] != Py_None) in[i] = THPVariable_Unpack(args[i]).data_ptr();
    at::Tensor made[kMostOutputs], ws;
    for (int i = 0; i < no; ++i)
      if (r->out[i].there) {
        made[i] = at::empty_strided(r->out[i].sizes, r->out[i].strides,
                                    at::TensorOptions().dtype(r->out[i].type).device(r->device));
        out[i] = made[i].data_ptr();
      }
    if (r->ws) ws = at::empty({r->ws}, at::TensorOptions().dtype(at::kByte).device(r->device));
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = launch(c, *r, pos0, in, out, r->ws ? ws.data_ptr() : nullptr, stream);
    Py_END_ALLOW_THREADS
    if (status) return PyLong_FromLong(status);
    PyObject* res = PyTuple_New(no);
    for (int i = 0; res && i < no; ++i) {
      PyObject* t = Py_None;
      if (made[i].defined()) t = THPVariable_Wrap(std::move(made[i]));
      else Py_INCREF(t);
      if (!t) {
        Py_DECREF(res);
        return nullptr;
      }
      PyTuple_SET_ITEM(res, i, t);
    }
    return res;
  });
}

// record(desc, address of desc, workspace bytes, count, outputs, *tensors), with
// outputs a sequence of None or (sizes, strides, dtype).
PyObject* calls_record(PyObject* self, PyObject* args) {
  auto* c = reinterpret_cast<Calls*>(self);
  return guarded([&]() -> PyObject* {
    const int ni = kInputs[c->kind], no = kOutputs[c->kind];
    if (PyTuple_GET_SIZE(args) != 5 + ni) {
      PyErr_SetString(PyExc_TypeError, "wrong number of tensors");
      return nullptr;
    }
    auto r = std::make_shared<Record>();
    r->d = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, 1));
    r->ws = PyLong_AsLongLong(PyTuple_GET_ITEM(args, 2));
    r->count = PyLong_AsLongLong(PyTuple_GET_ITEM(args, 3));
    if (PyErr_Occurred()) return nullptr;
    r->desc = PyTuple_GET_ITEM(args, 0);
    Py_INCREF(r->desc);
    for (int i = 0; i < ni; ++i) {
      PyObject* a = PyTuple_GET_ITEM(args, 5 + i);
      if (a == Py_None) continue;
      if (!THPVariable_Check(a)) {
        PyErr_SetString(PyExc_TypeError, "a tensor or None");
        return nullptr;
      }
      const at::Tensor& t = THPVariable_Unpack(a);
      Shape& s = r->in[i];
      if (i == 0) r->device = t.device();
      s.there = true;
      s.type = t.scalar_type();
      s.sizes = t.sizes().vec();
      s.strides = t.strides().vec();
    }
    PyObject* outs = PySequence_Fast(PyTuple_GET_ITEM(args, 4), "a sequence of outputs");
    if (!outs) return nullptr;
    bool ok = PySequence_Fast_GET_SIZE(outs) == no;
    if (!ok) PyErr_SetString(PyExc_TypeError, "wrong number of outputs");
    for (int i = 0; ok && i < no; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(outs, i);
      if (o == Py_None) continue;
      PyObject *sizes, *strides, *dtype;
      ok = PyArg_ParseTuple(o, "OOO", &sizes, &strides, &dtype) && read_ints(sizes, r->out[i].sizes) &&
           read_ints(strides, r->out[i].strides);
      if (ok && !THPDtype_Check(dtype)) {
        PyErr_SetString(PyExc_TypeError, "a dtype");
        ok = false;
      }
      if (!ok) break;
      r->out[i].there = true;
      r->out[i].type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    }
    Py_DECREF(outs);
    if (!ok) return nullptr;
    auto& rs = *c->records;
    if (rs.size() >= kMostRecords) rs.pop_back();
    rs.insert(rs.begin(), std::move(r));
    Py_RETURN_NONE;
  });
}

PyObject* calls_new(PyTypeObject* type, PyObject* args, PyObject*) {
  int kind;
  PyObject* fn;
  if (!PyArg_ParseTuple(args, "iO", &kind, &fn)) return nullptr;
  void* p = PyLong_AsVoidPtr(fn);
  if (PyErr_Occurred()) return nullptr;
  if (kind < 0 || kind >= KINDS || !p) {
    PyErr_SetString(PyExc_ValueError, "unknown kind of call");
    return nullptr;
  }
  auto* c = reinterpret_cast<Calls*>(type->tp_alloc(type, 0));
  if (!c) return nullptr;
  c->kind = kind;
  c->fn = p;
  c->records = new (std::nothrow) std::vector<std::shared_ptr<Record>>();
  if (!c->records) {
    Py_DECREF(c);
    return PyErr_NoMemory();
  }
  return reinterpret_cast<PyObject*>(c);
}

void calls_dealloc(PyObject* self) {
  delete reinterpret_cast<Calls*>(self)->records;
  Py_TYPE(self)->tp_free(self);
}

PyMethodDef methods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(calls_call)), METH_FASTCALL,
     "call(stream, pos0, *tensors): None if no record matches, a status, or the outputs"},
    {"record", calls_record, METH_VARARGS, "record(desc, address, workspace bytes, count, outputs, *tensors)"},
    {nullptr, nullptr, 0, nullptr}};

PyTypeObject type = {PyVarObject_HEAD_INIT(nullptr, 0)};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", "Repeated calls of gl_delta.h and gl_ssm.h.", -1, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
  type.tp_name = "weight_scans_amd._fastcall.Calls";
  type.tp_basicsize = sizeof(Calls);
  type.tp_flags = Py_TPFLAGS_DEFAULT;
  type.tp_new = calls_new;
  type.tp_dealloc = calls_dealloc;
  type.tp_methods = methods;
  if (PyType_Ready(&type) < 0) return nullptr;
  PyObject* m = PyModule_Create(&module);
  if (!m) return nullptr;
  Py_INCREF(&type);
  if (PyModule_AddObject(m, "Calls", reinterpret_cast<PyObject*>(&type)) < 0) {
    Py_DECREF(&type);
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
