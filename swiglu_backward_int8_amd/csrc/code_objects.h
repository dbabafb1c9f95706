// Every HIP source of the library is a code object of its own, which the runtime
// loads onto a device at the first launch of one of its kernels.  A function per
// source loads it before that; siluquant_prepare calls them all.
#ifndef SILUQUANT_CODE_OBJECTS_H
#define SILUQUANT_CODE_OBJECTS_H

#include <hip/hip_runtime.h>

namespace code_objects {

// Asking for a kernel's attributes makes the runtime load its code object on the
// current device.
template <class Kernel>
inline hipError_t load(Kernel kernel) {
  hipFuncAttributes attr;
  return hipFuncGetAttributes(&attr, reinterpret_cast<const void*>(kernel));
}

__attribute__((visibility("hidden"))) hipError_t load_i8gemm();
__attribute__((visibility("hidden"))) hipError_t load_rmsnorm();
__attribute__((visibility("hidden"))) hipError_t load_mxfp4();
__attribute__((visibility("hidden"))) hipError_t load_mxfp4gemm();

}  // namespace code_objects

#endif
