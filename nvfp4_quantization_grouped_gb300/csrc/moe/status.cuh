// status.cuh -- the word in which the grouped products of a device report what
// went wrong, and what a query takes out of it.
#pragma once

#include <stdint.h>

#include "gsa.h"

namespace gemm_status {

enum : uint32_t { ERR_SPLIT = 1, ERR_TIMEOUT = 2 };

// The report that the next query takes: one at a time, a timeout (results are
// incomplete) before a bad split (nothing was written).  0: none.
__host__ __device__ inline uint32_t next_report(uint32_t word) {
    return word & ERR_TIMEOUT ? ERR_TIMEOUT : word & ERR_SPLIT;
}

inline gsa_status status_of(uint32_t report) {
    if (report == ERR_TIMEOUT) return GSA_ERR_DEVICE_TIMEOUT;
    return report == ERR_SPLIT ? GSA_ERR_INVALID_ARG : GSA_OK;
}

}  // namespace gemm_status
