// Stands in for PyTorch's header where a test builds csrc/pycall.cpp without
// a GPU: CPU tensors (whose device index is -1) are those of the current
// device, so that every check of a tensor's type, shape and strides runs.
#pragma once
#include <torch/csrc/autograd/python_variable.h>

namespace c10::hip {
inline int current_device() { return -1; }
}  // namespace c10::hip

// (after PyTorch's own declarations)
#define is_cuda is_cpu
