// memset.h -- the status of a memset at a C entry point.
#pragma once

#include <cuda_runtime_api.h>

#include <string>

#include "dopt_internal.h"

namespace dopt {

// An error is reported here, not left for the next call to find.
inline int check_memset(cudaError_t e, const std::string& fn) {
  if (e == cudaSuccess) return DOPT_OK;
  (void)cudaGetLastError();
  return fail(DOPT_E_CUDA, fn + cudaGetErrorString(e));
}

}  // namespace dopt
