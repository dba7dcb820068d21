// dg_status.hip -- texts of libdg's status codes and of the last failed HIP call.
// In a file of its own, because the traffic records of the benchmark belong to the sources
// that decide how kernels run: rewording an error must not make them stale.
#include <hip/hip_runtime.h>

#include <cstdio>

#include "dg.h"
#include "dg_common.hpp"

namespace dg {

thread_local char g_last_hip_error[256] = "";

dg_status record_hip_error(hipError_t e) {
  std::snprintf(g_last_hip_error, sizeof(g_last_hip_error), "%s", hipGetErrorString(e));
  return DG_ERROR_LAUNCH_FAILED;
}

}  // namespace dg

extern "C" {

const char* dg_status_string(dg_status s) {
  switch (s) {
    case DG_SUCCESS: return "DG_SUCCESS";
    case DG_ERROR_INVALID_VALUE: return "DG_ERROR_INVALID_VALUE: invalid argument (pointer, alignment, stride, size or dtype)";
    case DG_ERROR_NOT_SUPPORTED:
      return "DG_ERROR_NOT_SUPPORTED: shape not supported (K % 128 != 0, contiguous M % 128 != 0, or a "
             "limit of the entry point, see dg.h)";
    case DG_ERROR_LAUNCH_FAILED: return "DG_ERROR_LAUNCH_FAILED: a HIP call failed";
    case DG_ERROR_SCRATCH_LIMIT:
      return "DG_ERROR_SCRATCH_LIMIT: the call needs more split-K scratch than the allocation-free entry point "
             "holds (16 MiB of partial tiles); use dg_fp8_gemm_nt with a workspace";
    case DG_ERROR_WORKSPACE:
      return "DG_ERROR_WORKSPACE: the workspace is missing, not 256-byte aligned or smaller than the entry point's "
             "size function says (dense GEMMs: dg_get_workspace_size(m, n, k))";
  }
  return "DG_UNKNOWN_STATUS";
}

const char* dg_last_hip_error(void) { return dg::g_last_hip_error; }

}  // extern "C"
