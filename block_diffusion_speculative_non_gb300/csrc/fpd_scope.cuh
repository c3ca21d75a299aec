// fpd_scope.cuh — what every entry point opens: its NVTX range and, in the FPD_DEBUG build, its own error check.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <string>

#include "fpd_internal.cuh"

namespace fpd {

fpd_status set_last_error(fpd_status s, const char* msg);   // message of the calling thread (fpd_last_error)

// NVTX range over one entry point; with FPD_DEBUG the call's kernels are also waited for and checked.
struct ApiScope {
  const char* name;
  cudaStream_t st;
  ApiScope(const char* n, void* s) : name(n), st((cudaStream_t)s) { nvtxRangePushA(n); }
  ~ApiScope() { nvtxRangePop(); }
  fpd_status done(fpd_status r) const {
#ifdef FPD_DEBUG
    if (r != FPD_OK) return r;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) return r;
    cudaError_t e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return set_last_error(FPD_ERR_CUDA, (std::string(name) + ": " + cudaGetErrorString(e)).c_str());
    int32_t code = 0;
    if (cudaMemcpyFromSymbol(&code, g_device_check, sizeof(code)) == cudaSuccess && code != 0)
      return set_last_error(FPD_ERR_DEVICE_CHECK, (std::string(name) + ": device check " + std::to_string(code)).c_str());
#endif
    return r;
  }
};

}  // namespace fpd
