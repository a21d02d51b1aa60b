// Launchers behind include/nvfp4_blocks.h (host side; arguments checked by the
// entry points).  dt and gamma_dt: 0 BF16, 1 FP32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "layers_launch.hpp"

namespace nvfp4 {

hipError_t launch_gated_act(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols,
                            int64_t ld_g, int64_t ld_u, void* y, int64_t ld_y, int8_t* gate_codes,
                            uint8_t* gate_scales, int8_t* up_codes, uint8_t* up_scales, hipStream_t s);
hipError_t launch_gated_act_back(int act, const int8_t* gate_codes, const uint8_t* gate_scales, const int8_t* up_codes,
                                 const uint8_t* up_scales, const void* dy, int dt, int64_t rows, int64_t cols,
                                 int64_t ld_dy, void* dgate, int64_t ld_dg, void* dup, int64_t ld_du, void* y,
                                 int64_t ld_y, hipStream_t s);

// up null: act(gate) alone; act 0 and up null: gate itself
hipError_t launch_int8_quantize(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols,
                                int64_t ld_g, int64_t ld_u, int8_t* codes, int64_t ld_codes, float* scales,
                                hipStream_t s);

int64_t int8_gemm_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda, const float* a_scales,
                            const int8_t* b, int64_t ldb, const float* b_scales, void* c, int c_dt, int64_t ldc,
                            void* workspace, int64_t workspace_bytes, hipStream_t s);

hipError_t launch_block_norms(const void* x, const void* residual, const void* gate, int dt, int64_t rows,
                              int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_gate, int gate_act,
                              const void* post_gamma, const void* pre_gamma, int gamma_dt, float eps, float scale,
                              void* h, int64_t ld_h, void* y, int64_t ld_y, int8_t* codes, int64_t ld_codes,
                              float* scales, float* post_rstd, float* pre_rstd, hipStream_t s);

int64_t block_norms_back_workspace(int64_t rows, int64_t cols);
hipError_t launch_block_norms_back(const void* dy, const void* dh, const void* h, const void* x, const void* gate,
                                   int dt, int64_t rows, int64_t cols, int64_t ld_dy, int64_t ld_dh, int64_t ld_h,
                                   int64_t ld_x, int64_t ld_gate, int gate_act, const void* post_gamma,
                                   const void* pre_gamma, int gamma_dt, const float* post_rstd, const float* pre_rstd,
                                   float scale, void* dx, int64_t ld_dx, void* dresidual, int64_t ld_dr, void* dgate,
                                   int64_t ld_dgate, float* dpost_gamma, float* dpre_gamma, void* workspace,
                                   hipStream_t s);

}  // namespace nvfp4
