// Launchers behind include/nvfp4_layers.h (host side; arguments checked by the
// entry points).  dt and gamma_dt: 0 BF16, 1 FP32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

namespace nvfp4 {

// Bytes from which on a launch streams past the caches (256 MB hold little of it
// until the next reader comes).
constexpr int64_t kStreamBytes = int64_t(128) << 20;

hipError_t launch_dropout(const void* x, int dt, int64_t rows, int64_t cols, int64_t ld_x, float p, uint64_t seed,
                          void* y, int64_t ld_y, hipStream_t s);

hipError_t launch_rms_norm(const void* x, const void* residual, int dt, int64_t rows, int64_t cols, int64_t ld_x,
                           int64_t ld_r, const void* gamma, int gamma_dt, float eps, float p, uint64_t seed, void* h,
                           int64_t ld_h, void* y, int64_t ld_y, uint8_t* codes, uint8_t* scales, float* rstd,
                           hipStream_t s);

int64_t rms_norm_back_workspace(int64_t rows, int64_t cols);
hipError_t launch_rms_norm_back(const void* dy, const void* dh, const void* h, int dt, int64_t rows, int64_t cols,
                                int64_t ld_dy, int64_t ld_dh, int64_t ld_h, const void* gamma, int gamma_dt,
                                const float* rstd, float p, uint64_t seed, void* dx, int64_t ld_dx, void* dresidual,
                                int64_t ld_dr, float* dgamma, void* workspace, hipStream_t s);

int64_t linear_ce_workspace(int64_t T, int64_t V, int64_t H, bool train);
hipError_t launch_linear_ce(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                            const int64_t* labels, float* loss, float* lse, void* workspace, hipStream_t s);
hipError_t launch_linear_ce_back(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w,
                                 int64_t ld_w, const int64_t* labels, const float* lse, const float* dloss, void* dx,
                                 int64_t ld_dx, void* dw, int dw_dt, int64_t ld_dw, int accumulate, void* workspace,
                                 hipStream_t s);

}  // namespace nvfp4
