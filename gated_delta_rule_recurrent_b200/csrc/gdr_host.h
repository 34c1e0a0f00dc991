// Host-side helpers shared by the library's translation units (gdr_api.cu
// defines them, gdr_linear_api.cu uses them). Internal: nothing here is
// exported from the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <string>

#include "gdr.h"

namespace gdr_host {

// Records `what` as the calling thread's last error and returns `status`.
int fail(int status, const std::string& what);

// The launch that gdr_last_launch reports to the calling thread; an empty one
// stands for a call that queued nothing.
void set_last_launch(const gdr_launch_info& info);

bool aligned16(const void* ptr);

// The current device: its ordinal, SM count and the largest shared memory a
// block may opt in to. Returns a gdr_status.
struct Device {
  int ordinal = 0;
  int sms = 0;
  int smem_optin = 0;
};
int current_device(Device* out);

// cuTensorMapEncodeTiled of the driver, or nullptr.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// gdr_linear_api.cu's copy of the device error word (each translation unit
// has its own): read, and cleared when `reset`.
cudaError_t linear_device_error(unsigned int* flags, bool reset);

#ifdef GDR_TEST_HOOKS
// The test hooks of gdr_linear_api.cu's kernels.
cudaError_t linear_set_hooks(long long wait_limit_cycles, int hold_tile);
#endif

}  // namespace gdr_host
