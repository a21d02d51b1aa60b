// C-ABI entry points of include/nvfp4_layers.h: argument validation on the
// host, then asynchronous launches on the caller's stream.
#include "../../include/nvfp4_layers.h"
#include "layers_launch.hpp"

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool known(int dt) { return dt == NVFP4_BF16 || dt == NVFP4_F32; }
uintptr_t size_of(int dt) { return dt == NVFP4_BF16 ? 2 : 4; }

// 65536 p must round to at most 65535: some elements are kept.
bool drop_ok(float p) { return p >= 0.0f && p < 1.0f - 0x1p-17f; }

nvfp4_status check_rows(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return NVFP4_ESHAPE;
  // element indices fit 32 bits, and so does the number of lanes a launch takes (16 a row or more)
  if (rows > (int64_t(1) << 28) - 16 || (rows > 0 && cols > ((int64_t(1) << 32) - 1) / rows)) return NVFP4_ESHAPE;
  if (cols >= (int64_t(1) << 32)) return NVFP4_ESHAPE;
  return NVFP4_OK;
}

// ld of a tensor that is used (p given): at least cols, and offsets that stay far inside 64 bits.
bool ld_ok(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  if (p == nullptr) return true;
  return ld >= cols && ld < (int64_t(1) << 40) && (rows == 0 || ld <= (int64_t(1) << 40) / rows);
}

// 256 rows of an operand stay within 32-bit byte offsets.
constexpr int64_t kMaxLd = int64_t(1) << 22;

nvfp4_status done(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EHIP; }

nvfp4_status check_loss(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                        const int64_t* labels, const float* lse, const void* workspace, int64_t workspace_bytes,
                        bool train) {
  if (T > 0 && (x == nullptr || w == nullptr || labels == nullptr || lse == nullptr)) return NVFP4_EINVAL;
  int64_t need = 0;
  const nvfp4_status st = nvfp4_linear_cross_entropy_workspace_size(T, V, H, train ? 1 : 0, &need);
  if (st != NVFP4_OK) return st;
  if (need > 0 && workspace == nullptr) return NVFP4_EINVAL;
  if (workspace_bytes < need) return NVFP4_ESHAPE;
  if (ld_x < H || ld_w < H || ld_x >= kMaxLd || ld_w >= kMaxLd) return NVFP4_ESHAPE;
  if (!aligned(x, 16) || !aligned(w, 16) || ld_x % 8 != 0 || ld_w % 8 != 0 || !aligned(labels, 8) ||
      !aligned(lse, 4) || !aligned(workspace, 16))
    return NVFP4_EALIGN;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_dropout(const void* x, int dt, int64_t rows, int64_t cols, int64_t ld_x, float p, uint64_t seed,
                           void* y, int64_t ld_y, void* stream) {
  if (!known(dt) || !drop_ok(p)) return NVFP4_EINVAL;
  if (rows > 0 && (x == nullptr || y == nullptr)) return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (!ld_ok(x, ld_x, rows, cols) || !ld_ok(y, ld_y, rows, cols)) return NVFP4_ESHAPE;
  if (!aligned(x, size_of(dt)) || !aligned(y, size_of(dt))) return NVFP4_EALIGN;
  return done(nvfp4::launch_dropout(x, dt, rows, cols, ld_x, p, seed, y, ld_y, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_rms_norm(const void* x, const void* residual, int dt, int64_t rows, int64_t cols, int64_t ld_x,
                            int64_t ld_r, const void* gamma, int gamma_dt, float eps, float p, uint64_t seed, void* h,
                            int64_t ld_h, void* y, int64_t ld_y, uint8_t* codes, uint8_t* scales, float* rstd,
                            void* stream) {
  if (!known(dt) || !known(gamma_dt) || !drop_ok(p) || !(eps >= 0.0f)) return NVFP4_EINVAL;
  if ((codes == nullptr) != (scales == nullptr) || (y != nullptr && codes != nullptr)) return NVFP4_EINVAL;
  if (rows > 0 && (x == nullptr || gamma == nullptr || (y == nullptr && codes == nullptr))) return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (!ld_ok(x, ld_x, rows, cols) || !ld_ok(residual, ld_r, rows, cols) || !ld_ok(h, ld_h, rows, cols) ||
      !ld_ok(y, ld_y, rows, cols))
    return NVFP4_ESHAPE;
  const uintptr_t es = size_of(dt);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(h, es) || !aligned(y, es) ||
      !aligned(gamma, size_of(gamma_dt)) || !aligned(rstd, 4))
    return NVFP4_EALIGN;
  return done(nvfp4::launch_rms_norm(x, residual, dt, rows, cols, ld_x, ld_r, gamma, gamma_dt, eps, p, seed, h, ld_h, y,
                                     ld_y, codes, scales, rstd, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_rms_norm_backward_workspace_size(int64_t rows, int64_t cols, int64_t* bytes) {
  if (bytes == nullptr) return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  *bytes = nvfp4::rms_norm_back_workspace(rows, cols);
  return NVFP4_OK;
}

nvfp4_status nvfp4_rms_norm_backward(const void* dy, const void* dh, const void* h, int dt, int64_t rows, int64_t cols,
                                     int64_t ld_dy, int64_t ld_dh, int64_t ld_h, const void* gamma, int gamma_dt,
                                     const float* rstd, float p, uint64_t seed, void* dx, int64_t ld_dx,
                                     void* dresidual, int64_t ld_dr, float* dgamma, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
  if (!known(dt) || !known(gamma_dt) || !drop_ok(p)) return NVFP4_EINVAL;
  if (rows > 0 && (dy == nullptr || h == nullptr || gamma == nullptr || rstd == nullptr ||
                   (dx == nullptr && dresidual == nullptr && dgamma == nullptr)))
    return NVFP4_EINVAL;
  const nvfp4_status st = check_rows(rows, cols);
  if (st != NVFP4_OK) return st;
  const int64_t need = dgamma == nullptr ? 0 : nvfp4::rms_norm_back_workspace(rows, cols);
  if (need > 0 && workspace == nullptr) return NVFP4_EINVAL;
  if (workspace_bytes < need) return NVFP4_ESHAPE;
  if (!ld_ok(dy, ld_dy, rows, cols) || !ld_ok(dh, ld_dh, rows, cols) || !ld_ok(h, ld_h, rows, cols) ||
      !ld_ok(dx, ld_dx, rows, cols) || !ld_ok(dresidual, ld_dr, rows, cols))
    return NVFP4_ESHAPE;
  const uintptr_t es = size_of(dt);
  if (!aligned(dy, es) || !aligned(dh, es) || !aligned(h, es) || !aligned(dx, es) || !aligned(dresidual, es) ||
      !aligned(gamma, size_of(gamma_dt)) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(workspace, 4))
    return NVFP4_EALIGN;
  return done(nvfp4::launch_rms_norm_back(dy, dh, h, dt, rows, cols, ld_dy, ld_dh, ld_h, gamma, gamma_dt, rstd, p, seed,
                                          dx, ld_dx, dresidual, ld_dr, dgamma, workspace,
                                          static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_linear_cross_entropy_workspace_size(int64_t T, int64_t V, int64_t H, int train, int64_t* bytes) {
  if (bytes == nullptr) return NVFP4_EINVAL;
  if (T < 0 || T >= (int64_t(1) << 22) || V <= 0 || H <= 0 || V >= (int64_t(1) << 24) || H >= kMaxLd ||
      H % 8 != 0)
    return NVFP4_ESHAPE;
  // the lanes of a launch (256 for 128 x 128 logits or more) fit 32 bits
  if (T > (int64_t(1) << 37) / V) return NVFP4_ESHAPE;
  *bytes = T == 0 ? 0 : nvfp4::linear_ce_workspace(T, V, H, train != 0);
  return NVFP4_OK;
}

nvfp4_status nvfp4_linear_cross_entropy(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w,
                                        int64_t ld_w, const int64_t* labels, float* loss, float* lse, void* workspace,
                                        int64_t workspace_bytes, void* stream) {
  if (T > 0 && loss == nullptr) return NVFP4_EINVAL;
  const nvfp4_status st =
      check_loss(T, V, H, x, ld_x, w, ld_w, labels, lse, workspace, workspace_bytes, false);
  if (st != NVFP4_OK) return st;
  if (!aligned(loss, 4)) return NVFP4_EALIGN;
  return done(nvfp4::launch_linear_ce(T, V, H, x, ld_x, w, ld_w, labels, loss, lse, workspace,
                                      static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_linear_cross_entropy_backward(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x,
                                                 const void* w, int64_t ld_w, const int64_t* labels, const float* lse,
                                                 const float* dloss, void* dx, int64_t ld_dx, void* dw, int dw_dt,
                                                 int64_t ld_dw, float beta, void* workspace, int64_t workspace_bytes,
                                                 void* stream) {
  if (!known(dw_dt) || (beta != 0.0f && beta != 1.0f)) return NVFP4_EINVAL;
  if (T > 0 && (dloss == nullptr || (dx == nullptr && dw == nullptr))) return NVFP4_EINVAL;
  const nvfp4_status st = check_loss(T, V, H, x, ld_x, w, ld_w, labels, lse, workspace, workspace_bytes, true);
  if (st != NVFP4_OK) return st;
  if ((dx != nullptr && (ld_dx < H || ld_dx >= kMaxLd)) || (dw != nullptr && (ld_dw < H || ld_dw >= kMaxLd)))
    return NVFP4_ESHAPE;
  if (!aligned(dloss, 4) || !aligned(dx, 16) || !aligned(dw, 16) || (dx != nullptr && ld_dx % 8 != 0) ||
      (dw != nullptr && ld_dw % (dw_dt == NVFP4_BF16 ? 8 : 4) != 0))
    return NVFP4_EALIGN;
  return done(nvfp4::launch_linear_ce_back(T, V, H, x, ld_x, w, ld_w, labels, lse, dloss, dx, ld_dx, dw, dw_dt, ld_dw,
                                           beta == 1.0f ? 1 : 0, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
