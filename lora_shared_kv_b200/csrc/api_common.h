// What the translation units of the C ABI share: the error text, device facts,
// tensor maps and the checks of the common arguments (defined in lrkv_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lrkv_internal.h"

namespace lrkv {
namespace api {

struct DeviceInfo {
  int sms = 0;
  int major = 0;
  int smem_optin = 0;
};

// Set the thread's error text and return `s`.
lrkv_status fail(lrkv_status s, const char* fmt, ...);
lrkv_status cuda_fail(cudaError_t e, const char* what);

// Facts of the current device; LRKV_ERR_UNSUPPORTED unless it is an sm_100 GPU.
lrkv_status device_info(DeviceInfo* out);

// Spin cap and stall flag of a launch (disarms lrkv_debug_stall_next_launch).
void take_stall_hook(unsigned* spin_cap, int* stall);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 4-D tensor map of elements of `type` (elem_bytes each), dims/strides innermost
// first (strides in elements, for dims 1..3).  A dimension of extent 1 gets a
// packed stride.
lrkv_status make_map4(CUtensorMap* m, const void* base, const uint64_t dims[4], const int64_t strides_el[3],
                      const uint32_t box[4], CUtensorMapSwizzle swz, const char* what,
                      CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, int elem_bytes = 2);

lrkv_status check_problem(const lrkv_problem* p);
lrkv_status check_kv(const lrkv_kv_view* kv, const lrkv_problem* p);
lrkv_status check_u(const lrkv_u_view* u, const lrkv_problem* p, int rows_needed);
float scale_of(const lrkv_problem* p);

}  // namespace api
}  // namespace lrkv
