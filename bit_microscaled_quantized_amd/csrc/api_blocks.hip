// C-ABI entry points of include/nvfp4_blocks.h: argument validation on the host,
// then asynchronous launches on the caller's stream.
#include "../../include/nvfp4_blocks.h"
#include "blocks_launch.hpp"

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool known(int dt) { return dt == NVFP4_BF16 || dt == NVFP4_F32; }
bool known_act(int act) { return act >= NVFP4_ACT_NONE && act <= NVFP4_ACT_RELU2; }
uintptr_t size_of(int dt) { return dt == NVFP4_BF16 ? 2 : 4; }
hipStream_t on(void* stream) { return static_cast<hipStream_t>(stream); }
nvfp4_status done(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EHIP; }

nvfp4_status check_rows(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols >= (int64_t(1) << 32)) return NVFP4_ESHAPE;
  // element indices fit 32 bits, and so does the number of lanes a launch takes (16 a row or more)
  if (rows > (int64_t(1) << 28) - 16 || (rows > 0 && cols > ((int64_t(1) << 32) - 1) / rows)) return NVFP4_ESHAPE;
  return NVFP4_OK;
}

// ld of a tensor that is used (p given): at least cols, and offsets that stay far inside 64 bits.
bool ld_ok(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  if (p == nullptr) return true;
  return ld >= cols && ld < (int64_t(1) << 40) && (rows == 0 || ld <= (int64_t(1) << 40) / rows);
}

// Rows of codes: 16-byte pieces, which cover the columns.
nvfp4_status check_codes(const int8_t* codes, int64_t ld, const float* scales, int64_t rows, int64_t cols) {
  if (cols >= (int64_t(1) << 31) || !ld_ok(codes, ld, rows, cols)) return NVFP4_ESHAPE;
  if (ld % 16 != 0 || !aligned(codes, 16) || !aligned(scales, 4)) return NVFP4_EALIGN;
  return NVFP4_OK;
}

nvfp4_status quantize(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols, int64_t ld_gate,
                      int64_t ld_up, int8_t* codes, int64_t ld_codes, float* scales, void* stream) {
  if (!known(dt) || !known_act(act)) return NVFP4_EINVAL;
  if (rows > 0 && (gate == nullptr || codes == nullptr || scales == nullptr)) return NVFP4_EINVAL;
  nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (!ld_ok(gate, ld_gate, rows, cols) || !ld_ok(up, ld_up, rows, cols)) return NVFP4_ESHAPE;
  st = check_codes(codes, ld_codes, scales, rows, cols);
  if (st != NVFP4_OK) return st;
  if (!aligned(gate, size_of(dt)) || !aligned(up, size_of(dt))) return NVFP4_EALIGN;
  return done(nvfp4::launch_int8_quantize(act, gate, up, dt, rows, cols, ld_gate, ld_up, codes, ld_codes, scales,
                                          on(stream)));
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_int8_quantize(const void* x, int dt, int64_t rows, int64_t cols, int64_t ld_x, int8_t* codes,
                                 int64_t ld_codes, float* scales, void* stream) {
  return quantize(NVFP4_ACT_NONE, x, nullptr, dt, rows, cols, ld_x, 0, codes, ld_codes, scales, stream);
}

nvfp4_status nvfp4_int8_quantize_gated(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols,
                                       int64_t ld_gate, int64_t ld_up, int8_t* codes, int64_t ld_codes, float* scales,
                                       void* stream) {
  return quantize(act, gate, up, dt, rows, cols, ld_gate, ld_up, codes, ld_codes, scales, stream);
}

nvfp4_status nvfp4_int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t* bytes) {
  if (bytes == nullptr) return NVFP4_EINVAL;
  // M * N: the lanes of a launch, 256 for 64 x 64 sums, fit 32 bits
  if (M < 0 || N < 1 || K < 16 || M >= (int64_t(1) << 24) || N >= (int64_t(1) << 24) || M * N > (int64_t(1) << 35) ||
      K > 131056 || K % 16 != 0)
    return NVFP4_ESHAPE;
  *bytes = nvfp4::int8_gemm_workspace(M, N, K);
  return NVFP4_OK;
}

nvfp4_status nvfp4_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda, const float* a_scales,
                             const int8_t* b, int64_t ldb, const float* b_scales, void* c, int c_dt, int64_t ldc,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  if (!known(c_dt)) return NVFP4_EINVAL;
  if (M > 0 && (a == nullptr || a_scales == nullptr || b == nullptr || b_scales == nullptr || c == nullptr))
    return NVFP4_EINVAL;
  int64_t most = 0;
  const nvfp4_status st = nvfp4_int8_gemm_workspace_size(M, N, K, &most);
  if (st != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  constexpr int64_t kMaxLd = int64_t(1) << 23;  // 256 rows of an operand stay within 32-bit byte offsets
  if (lda < K || ldb < K || lda >= kMaxLd || ldb >= kMaxLd || !ld_ok(c, ldc, M, N)) return NVFP4_ESHAPE;
  if (lda % 16 != 0 || ldb % 16 != 0 || !aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 4) ||
      !aligned(b_scales, 4) || !aligned(c, size_of(c_dt)) || !aligned(workspace, 16))
    return NVFP4_EALIGN;
  return done(nvfp4::launch_int8_gemm(M, N, K, a, lda, a_scales, b, ldb, b_scales, c, c_dt, ldc, workspace,
                                      workspace_bytes, on(stream)));
}

nvfp4_status nvfp4_block_norms(const void* x, const void* residual, const void* gate, int dt, int64_t rows,
                               int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_gate, int gate_act,
                               const void* post_gamma, const void* pre_gamma, int gamma_dt, float eps, float scale,
                               void* h, int64_t ld_h, void* y, int64_t ld_y, int8_t* codes, int64_t ld_codes,
                               float* scales, float* post_rstd, float* pre_rstd, void* stream) {
  if (!known(dt) || !known(gamma_dt) || (gate_act != NVFP4_GATE_LINEAR && gate_act != NVFP4_GATE_SIGMOID) ||
      !(eps >= 0.0f) || !__builtin_isfinite(scale))
    return NVFP4_EINVAL;
  if ((codes == nullptr) != (scales == nullptr) || (y != nullptr && codes != nullptr)) return NVFP4_EINVAL;
  if (rows > 0 && (x == nullptr || post_gamma == nullptr || pre_gamma == nullptr || (y == nullptr && codes == nullptr)))
    return NVFP4_EINVAL;
  nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (!ld_ok(x, ld_x, rows, cols) || !ld_ok(residual, ld_r, rows, cols) || !ld_ok(h, ld_h, rows, cols) ||
      !ld_ok(y, ld_y, rows, cols) || (ld_gate != 0 && !ld_ok(gate, ld_gate, rows, cols)))
    return NVFP4_ESHAPE;
  if (codes != nullptr && (st = check_codes(codes, ld_codes, scales, rows, cols)) != NVFP4_OK) return st;
  const uintptr_t es = size_of(dt), gs = size_of(gamma_dt);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(gate, es) || !aligned(h, es) || !aligned(y, es) ||
      !aligned(post_gamma, gs) || !aligned(pre_gamma, gs) || !aligned(post_rstd, 4) || !aligned(pre_rstd, 4))
    return NVFP4_EALIGN;
  return done(nvfp4::launch_block_norms(x, residual, gate, dt, rows, cols, ld_x, ld_r, ld_gate, gate_act, post_gamma,
                                        pre_gamma, gamma_dt, eps, scale, h, ld_h, y, ld_y, codes, ld_codes, scales,
                                        post_rstd, pre_rstd, on(stream)));
}

nvfp4_status nvfp4_block_norms_backward_workspace_size(int64_t rows, int64_t cols, int64_t* bytes) {
  if (bytes == nullptr) return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  *bytes = nvfp4::block_norms_back_workspace(rows, cols);
  return NVFP4_OK;
}

nvfp4_status nvfp4_block_norms_backward(const void* dy, const void* dh, const void* h, const void* x, const void* gate,
                                        int dt, int64_t rows, int64_t cols, int64_t ld_dy, int64_t ld_dh, int64_t ld_h,
                                        int64_t ld_x, int64_t ld_gate, int gate_act, const void* post_gamma,
                                        const void* pre_gamma, int gamma_dt, const float* post_rstd,
                                        const float* pre_rstd, float scale, void* dx, int64_t ld_dx, void* dresidual,
                                        int64_t ld_dr, void* dgate, int64_t ld_dgate, float* dpost_gamma,
                                        float* dpre_gamma, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!known(dt) || !known(gamma_dt) || (gate_act != NVFP4_GATE_LINEAR && gate_act != NVFP4_GATE_SIGMOID) ||
      !__builtin_isfinite(scale))
    return NVFP4_EINVAL;
  if (gate == nullptr && dgate != nullptr) return NVFP4_EINVAL;
  if (rows > 0 && (dy == nullptr || h == nullptr || x == nullptr || post_gamma == nullptr || pre_gamma == nullptr ||
                   post_rstd == nullptr || pre_rstd == nullptr ||
                   (dx == nullptr && dresidual == nullptr && dgate == nullptr && dpost_gamma == nullptr &&
                    dpre_gamma == nullptr)))
    return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  const bool shared = gate != nullptr && ld_gate == 0;
  const bool sums = dpost_gamma != nullptr || dpre_gamma != nullptr || (shared && dgate != nullptr);
  const int64_t need = sums ? nvfp4::block_norms_back_workspace(rows, cols) : 0;
  if (need > 0 && workspace == nullptr) return NVFP4_EINVAL;
  if (workspace_bytes < need) return NVFP4_ESHAPE;
  if (!ld_ok(dy, ld_dy, rows, cols) || !ld_ok(dh, ld_dh, rows, cols) || !ld_ok(h, ld_h, rows, cols) ||
      !ld_ok(x, ld_x, rows, cols) || !ld_ok(dx, ld_dx, rows, cols) || !ld_ok(dresidual, ld_dr, rows, cols) ||
      (!shared && (!ld_ok(gate, ld_gate, rows, cols) || !ld_ok(dgate, ld_dgate, rows, cols))))
    return NVFP4_ESHAPE;
  const uintptr_t es = size_of(dt), gs = size_of(gamma_dt);
  if (!aligned(dy, es) || !aligned(dh, es) || !aligned(h, es) || !aligned(x, es) || !aligned(gate, es) ||
      !aligned(dx, es) || !aligned(dresidual, es) || !aligned(dgate, shared ? 4 : es) || !aligned(post_gamma, gs) ||
      !aligned(pre_gamma, gs) || !aligned(post_rstd, 4) || !aligned(pre_rstd, 4) || !aligned(dpost_gamma, 4) ||
      !aligned(dpre_gamma, 4) || !aligned(workspace, 4))
    return NVFP4_EALIGN;
  return done(nvfp4::launch_block_norms_back(dy, dh, h, x, gate, dt, rows, cols, ld_dy, ld_dh, ld_h, ld_x, ld_gate,
                                             gate_act, post_gamma, pre_gamma, gamma_dt, post_rstd, pre_rstd, scale, dx,
                                             ld_dx, dresidual, ld_dr, dgate, ld_dgate, dpost_gamma, dpre_gamma,
                                             workspace, on(stream)));
}

nvfp4_status nvfp4_gated_act(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols,
                             int64_t ld_gate, int64_t ld_up, void* y, int64_t ld_y, int8_t* gate_codes,
                             uint8_t* gate_scales, int8_t* up_codes, uint8_t* up_scales, void* stream) {
  if (!known(dt) || !known_act(act)) return NVFP4_EINVAL;
  if ((gate_codes == nullptr) != (gate_scales == nullptr) || (up_codes == nullptr) != (up_scales == nullptr))
    return NVFP4_EINVAL;
  if (rows > 0 && (gate == nullptr || (y == nullptr && gate_codes == nullptr) ||
                   (up_codes != nullptr) != (up != nullptr && gate_codes != nullptr)))
    return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (!ld_ok(gate, ld_gate, rows, cols) || !ld_ok(up, ld_up, rows, cols) || !ld_ok(y, ld_y, rows, cols))
    return NVFP4_ESHAPE;
  const uintptr_t es = size_of(dt);
  if (!aligned(gate, es) || !aligned(up, es) || !aligned(y, es)) return NVFP4_EALIGN;
  return done(nvfp4::launch_gated_act(act, gate, up, dt, rows, cols, ld_gate, ld_up, y, ld_y, gate_codes, gate_scales,
                                      up_codes, up_scales, on(stream)));
}

nvfp4_status nvfp4_gated_act_backward(int act, const int8_t* gate_codes, const uint8_t* gate_scales,
                                      const int8_t* up_codes, const uint8_t* up_scales, const void* dy, int dt,
                                      int64_t rows, int64_t cols, int64_t ld_dy, void* dgate, int64_t ld_dgate,
                                      void* dup, int64_t ld_dup, void* y, int64_t ld_y, void* stream) {
  if (!known(dt) || !known_act(act)) return NVFP4_EINVAL;
  if ((gate_codes == nullptr) != (gate_scales == nullptr) || (up_codes == nullptr) != (up_scales == nullptr))
    return NVFP4_EINVAL;
  if (rows > 0 && (gate_codes == nullptr || (dgate == nullptr && dup == nullptr && y == nullptr) ||
                   (dup != nullptr && up_codes == nullptr) ||
                   (dy != nullptr) != (dgate != nullptr || dup != nullptr)))
    return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (!ld_ok(dy, ld_dy, rows, cols) || !ld_ok(dgate, ld_dgate, rows, cols) || !ld_ok(dup, ld_dup, rows, cols) ||
      !ld_ok(y, ld_y, rows, cols))
    return NVFP4_ESHAPE;
  const uintptr_t es = size_of(dt);
  if (!aligned(dy, es) || !aligned(dgate, es) || !aligned(dup, es) || !aligned(y, es)) return NVFP4_EALIGN;
  return done(nvfp4::launch_gated_act_back(act, gate_codes, gate_scales, up_codes, up_scales, dy, dt, rows, cols, ld_dy,
                                           dgate, ld_dgate, dup, ld_dup, y, ld_y, on(stream)));
}

}  // extern "C"
