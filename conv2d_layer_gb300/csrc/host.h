// host.h - host-side state shared by the library's C entry points (defined in
// api.cu): per-device data, the profiling ring and the tensor-map encoder.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "conv2d.h"

namespace c2d {

constexpr size_t kMaxDynSmem = 232448;  // 227 KB opt-in per block

struct DevInfo {
  bool init = false;
  int sms = 0;
  int* err = nullptr;  // device-side error word (bounded waits)
};
// Data of the current device, looked up on its first call; returns a CONV2D status.
int device_info(DevInfo** out);
// SM count used for sizing when no device is visible (workspace queries on a machine without a GPU).
int sms_for_sizing();

int prof_begin(const char* name, cudaStream_t st);
void prof_end(int slot, cudaStream_t st);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled, or null when the driver does not offer it.
EncodeTiledFn encode_fn();

#define LAUNCH(name, st, call)                \
  do {                                        \
    const int _slot = prof_begin(name, st);   \
    const cudaError_t _e = (call);            \
    prof_end(_slot, st);                      \
    if (_e != cudaSuccess) return CONV2D_ERR_CUDA; \
  } while (0)

}  // namespace c2d
