// Host-side helpers shared by the library's translation units: error
// reporting through bwd_last_error() and launch checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "bwd.h"

namespace bwd {
namespace host {

// Records a printf-style message as this thread's last error and returns s.
bwd_status fail(bwd_status s, const char* fmt, ...);

// BWD_ERR_CUDA with the runtime's name and description of e.
bwd_status cuda_fail(cudaError_t e, const char* what);

// BWD_OK, or BWD_ERR_CUDA if the last launch on this thread failed.
bwd_status check_launch(const char* what);

// This thread's last error message ("" if none).
const char* last_error();

// Host scalars of an Adam update: bias corrections in binary64, rounded once.
struct AdamScalars {
  float b1, omb1, b2, omb2, eps, step_size, inv_bc2s;
  float decay;  // 1 - lr * weight_decay (decoupled weight decay), 1 for Adam
};
AdamScalars adam_scalars(const bwd_adamw_hparams& hp);

// A count of steps in device memory, and the scalars of the step that it last
// counted.
struct StepCount {
  int64_t taken;
  float step_size, inv_bc2s;
};
// Counts a step, unless *grad_scale is not finite, and forms its scalars.
bwd_status advance(StepCount* count, const float* grad_scale, const bwd_adamw_hparams& hp, void* stream);

// BWD_OK, or BWD_ERR_INVALID_ARG where a hyper-parameter is outside its range.
bwd_status check_hparams(const bwd_adam_hparams* hp);
bwd_status check_hparams(const bwd_adamw_hparams* hp);

// Reads and clears the 8-bit products' fault word (see bwd_check_device).
bwd_status take_fp8_fault(unsigned int* fault);

// Unique id of the current CUDA context (the driver's cuCtxGetId, unique for
// the life of the process).  Per-device state cached by the library (the
// uploaded code tables, kernel attributes) belongs to one context: after a
// cudaDeviceReset or a released primary context the id changes and the state
// is set up again.  Initialises the device's primary context if none is
// current.
bwd_status current_context_id(unsigned long long* id);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// p is a multiple of `bytes` (a power of two): element pointers must be
// aligned to their element size, or device accesses through them fault.
inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace host
}  // namespace bwd
