// f8_grad.cpp -- the stream on which a leaf's gradient is accumulated, which torch
// does not show to Python: the one that was current when the first graph that holds
// the leaf was made.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_cpp_function.h>

#include <exception>

namespace {

// on_default_stream(node): whether an accumulation node (torch._C._functions.AccumulateGrad,
// the caller has checked) runs on its device's default stream.
PyObject* on_default_stream(PyObject*, PyObject* node) {
  try {
    const auto stream = reinterpret_cast<torch::autograd::THPCppFunction*>(node)->cdata->stream();
    return PyBool_FromLong(stream.has_value() && *stream == c10::Stream(c10::Stream::DEFAULT, stream->device()));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {{"on_default_stream", on_default_stream, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "f8_grad", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_f8_grad() { return PyModule_Create(&module); }
