#pragma once
// Launchers of the output norm (kda_norm.hip).
#include <hip/hip_runtime.h>

#include "kda.h"

namespace kda_host {
// rows of p.D elements; with cu the live rows are cu[N] * rpt <= rows
hipError_t launch_norm(kda_dtype dt, int64_t rows, const kda_norm& p, const int32_t* cu, int N, int rpt,
                       const void* x, const void* z, void* y, hipStream_t s);
size_t norm_bwd_ws_bytes(int D);
hipError_t launch_norm_bwd(kda_dtype dt, int64_t rows, const kda_norm& p, const int32_t* cu, int N, int rpt,
                           const void* x, const void* z, const void* dy, void* dx, void* dz, void* dw,
                           void* db, void* ws, hipStream_t s);
}  // namespace kda_host
