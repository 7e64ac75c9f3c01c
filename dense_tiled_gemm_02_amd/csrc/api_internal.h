// Helpers the C ABI's translation units share (host only).
#pragma once

#include "../../include/gemm.h"

namespace dtg {

// The longest contraction, and the largest size of a grouped or 4-bit product:
// kernels round it up to whole steps, and run a few steps ahead, in 32 bits.
constexpr int64_t kMaxSize = (int64_t(1) << 31) - 4096;

// Store `msg` as the calling thread's last error (gemm_last_error) and return st.
gemm_status record_error(gemm_status st, const char* msg);

// gemm_device_query for `device`, cached per device.
gemm_status cached_device_info(int device, gemm_device_info* info);

}  // namespace dtg
