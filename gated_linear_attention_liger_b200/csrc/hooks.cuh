// hooks.cuh -- what the library's translation units share on the host side (defined in
// liger_attn.cu): the thread's last error, launch counting, the caller's timing events, and
// device properties.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "liger_attn.h"

namespace liger {

void set_last_error(liger_status status, const char* message);
void clear_last_error();
void count_kernel_launches(int n);
void mark_dominant_start(cudaStream_t s);
void mark_dominant_stop(cudaStream_t s);
int device_sm_count();
uint64_t bounded_wait_ns();   // give-up time of one wait

typedef CUresult (*TensorMapEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncodeFn tensor_map_encoder();   // null if the driver has none

}  // namespace liger
