// C ABI of the norms, of the balance loss and of the ScaledSwiGLU by itself:
// argument validation and launches.  The contracts are in include/moe_mi355x.h.
#include "moe_mi355x.h"

#include <hip/hip_runtime.h>

#include "kernels.hpp"

using namespace moe;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool bad_type(int t) { return t != MOE_TYPE_BF16 && t != MOE_TYPE_F32; }

// T x H rows of a norm; a checkpoint needs whole blocks of 32
int check_norm(int x_type, int w_type, int64_t T, int H, const void* codes, const void* scales) {
    if (bad_type(x_type) || bad_type(w_type)) return MOE_ERR_ARG;
    if ((codes == nullptr) != (scales == nullptr)) return MOE_ERR_ARG;
    if (T < 0 || T > INT32_MAX || H < 8 || (H % 8) || H > kMaxNormH) return MOE_ERR_SHAPE;
    if (codes && (H % 32)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

int check_swiglu(int64_t rows, int I, const void* codes, const void* scales) {
    if ((codes == nullptr) != (scales == nullptr)) return MOE_ERR_ARG;
    if (rows < 0 || rows > INT32_MAX || I < 8 || (I % 8) || I > kMaxSwigluI) return MOE_ERR_SHAPE;
    if (codes && (I % 32)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

// x, the stream it joins, gamma; without a residual the stream is x
int check_rmsnorm(int x_type, int stream_type, int w_type, int64_t T, int H, const void* residual) {
    if (bad_type(x_type) || bad_type(stream_type) || bad_type(w_type)) return MOE_ERR_ARG;
    if (x_type != stream_type && (x_type == MOE_TYPE_F32 || (T > 0 && !residual))) return MOE_ERR_ARG;
    if (T < 0 || T > INT32_MAX || H < 8 || (H % 8) || H > kMaxNormH) return MOE_ERR_SHAPE;
    return MOE_OK;
}

int check_balance(int64_t T, int E, int k, float coef, float zcoef) {
    if (E < 1 || E > kMaxExperts || k < 1 || k > E || T < 0 || T > INT32_MAX / k) return MOE_ERR_SHAPE;
    if (coef - coef != 0.f || zcoef - zcoef != 0.f) return MOE_ERR_ARG;     // finite
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_rmsnorm_workspace_bytes(int64_t T, int H) {
    if (T < 0 || T > INT32_MAX || H < 8 || (H % 8) || H > kMaxNormH) return 0;
    return rmsnorm_workspace_bytes(T, H);
}

int moe_rmsnorm_fwd(int x_type, int stream_type, int w_type, int64_t T, int H, const void* x,
                    const void* residual, const void* gamma, float eps, void* h, uint16_t* y, float* rstd,
                    uint8_t* codes, float* scales, hipStream_t stream) {
    const int st = check_rmsnorm(x_type, stream_type, w_type, T, H, residual);
    if (st != MOE_OK) return st;
    if ((codes == nullptr) != (scales == nullptr) || !(eps >= 0.f)) return MOE_ERR_ARG;
    if (T > 0 && (!x || (residual && !h) || (!y && !codes))) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(h) || !aligned16(y) ||
        !aligned16(codes) || !aligned16(scales))
        return MOE_ERR_ALIGN;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_rmsnorm_fwd(x, x_type == MOE_TYPE_F32, residual, stream_type == MOE_TYPE_F32, T,
                                         H, gamma, w_type == MOE_TYPE_F32, eps, h, y, rstd, codes, scales,
                                         stream));
}

int moe_rmsnorm_bwd(int stream_type, int w_type, int64_t T, int H, const uint16_t* dy, const void* h,
                    const float* rstd, const void* gamma, const void* dres, void* dx, uint16_t* dx_branch,
                    void* dgamma, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const int st = check_rmsnorm(stream_type, stream_type, w_type, T, H, nullptr);
    if (st != MOE_OK) return st;
    if (T > 0 && (!dy || !h || !rstd || !dx)) return MOE_ERR_NULL;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(gamma) || !aligned16(dres) || !aligned16(dx) ||
        !aligned16(dx_branch) || !aligned16(dgamma) || !aligned16(workspace))
        return MOE_ERR_ALIGN;
    if (dgamma) {
        if (!workspace) return MOE_ERR_NULL;
        if (workspace_bytes < rmsnorm_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE;
    }
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_rmsnorm_bwd(dy, h, stream_type == MOE_TYPE_F32, rstd, T, H, gamma,
                                         w_type == MOE_TYPE_F32, dres, dx, dx_branch, dgamma, workspace,
                                         stream));
}

size_t moe_balance_workspace_bytes(int E) {
    return E < 1 || E > kMaxExperts ? 0 : balance_workspace_bytes(E);
}

int moe_balance_fwd(const float* logits, int64_t T, int E, int k, const int32_t* topk_expert,
                    const uint8_t* mask, float balance_coef, float z_coef, float* losses, int32_t* counts,
                    int32_t* tokens, float* mean_prob, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const int st = check_balance(T, E, k, balance_coef, z_coef);
    if (st != MOE_OK) return st;
    if (!losses || !counts || !tokens || !workspace || (T > 0 && (!logits || !topk_expert))) return MOE_ERR_NULL;
    if (!aligned16(logits) || !aligned16(workspace)) return MOE_ERR_ALIGN;
    if (workspace_bytes < balance_workspace_bytes(E)) return MOE_ERR_WORKSPACE;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_balance_fwd(logits, T, E, k, topk_expert, mask, balance_coef, z_coef, losses,
                                         counts, tokens, mean_prob, workspace, stream));
}

int moe_balance_bwd(const float* logits, int64_t T, int E, int k, const uint8_t* mask, float balance_coef,
                    float z_coef, const int32_t* counts, const int32_t* tokens, const float* dloss,
                    const float* dlogits_in, float* dlogits, hipStream_t stream) {
    const int st = check_balance(T, E, k, balance_coef, z_coef);
    if (st != MOE_OK) return st;
    if (!counts || !tokens || (T > 0 && (!logits || !dlogits))) return MOE_ERR_NULL;
    if (!aligned16(logits) || !aligned16(dlogits_in) || !aligned16(dlogits)) return MOE_ERR_ALIGN;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_balance_bwd(logits, T, E, k, mask, balance_coef, z_coef, counts, tokens,
                                         dloss, dlogits_in, dlogits, stream));
}

size_t moe_layernorm_workspace_bytes(int64_t T, int H) {
    if (T < 0 || T > INT32_MAX || H < 8 || (H % 8) || H > kMaxNormH) return 0;
    return layernorm_workspace_bytes(T, H);
}

int moe_layernorm_fwd(int x_type, int w_type, int64_t T, int H, const void* x, const void* gamma,
                      const void* beta, float eps, uint16_t* y, float* mean, float* rstd,
                      uint8_t* xhat_codes, uint8_t* xhat_scales, hipStream_t stream) {
    const int st = check_norm(x_type, w_type, T, H, xhat_codes, xhat_scales);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.f)) return MOE_ERR_ARG;
    if (T > 0 && (!x || !y)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y) ||
        !aligned16(xhat_codes))
        return MOE_ERR_ALIGN;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_layernorm_fwd(x, x_type == MOE_TYPE_F32, T, H, gamma, beta,
                                           w_type == MOE_TYPE_F32, eps, y, mean, rstd, xhat_codes,
                                           xhat_scales, stream));
}

int moe_layernorm_bwd(int x_type, int w_type, int64_t T, int H, const uint16_t* dy, const void* x,
                      const float* mean, const float* rstd, const uint8_t* xhat_codes,
                      const uint8_t* xhat_scales, const void* gamma, const void* dres, void* dx,
                      void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    const int st = check_norm(x_type, w_type, T, H, xhat_codes, xhat_scales);
    if (st != MOE_OK) return st;
    if (T > 0 && (!dy || !dx || !rstd || (!xhat_codes && (!x || !mean)))) return MOE_ERR_NULL;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(xhat_codes) || !aligned16(gamma) ||
        !aligned16(dres) || !aligned16(dx) || !aligned16(dgamma) || !aligned16(dbeta) ||
        !aligned16(workspace))
        return MOE_ERR_ALIGN;
    if (dgamma || dbeta) {
        if (!workspace) return MOE_ERR_NULL;
        if (workspace_bytes < layernorm_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE;
    }
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_layernorm_bwd(dy, x, x_type == MOE_TYPE_F32, mean, rstd, xhat_codes,
                                           xhat_scales, T, H, gamma, w_type == MOE_TYPE_F32, dres,
                                           dx, dgamma, dbeta, workspace, stream));
}

int moe_swiglu_fwd(int64_t rows, int I, const uint16_t* a1, const float* prob, uint16_t* a2,
                   uint8_t* a1_codes, uint8_t* a1_scales, hipStream_t stream) {
    const int st = check_swiglu(rows, I, a1_codes, a1_scales);
    if (st != MOE_OK) return st;
    if (rows > 0 && (!a1 || !a2)) return MOE_ERR_NULL;
    if (!aligned16(a1) || !aligned16(a2) || !aligned16(a1_codes)) return MOE_ERR_ALIGN;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_swiglu_fwd(a1, prob, rows, I, a2, a1_codes, a1_scales, stream));
}

int moe_swiglu_bwd(int64_t rows, int I, const uint16_t* da2, const uint16_t* a1,
                   const uint8_t* a1_codes, const uint8_t* a1_scales, const float* prob,
                   uint16_t* da1, float* dprob, hipStream_t stream) {
    const int st = check_swiglu(rows, I, a1_codes, a1_scales);
    if (st != MOE_OK) return st;
    if ((a1 != nullptr) && a1_codes) return MOE_ERR_ARG;
    if (rows > 0 && (!da2 || !da1 || (!a1 && !a1_codes))) return MOE_ERR_NULL;
    if (!aligned16(da2) || !aligned16(a1) || !aligned16(a1_codes) || !aligned16(da1))
        return MOE_ERR_ALIGN;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_swiglu_bwd(da2, a1, a1_codes, a1_scales, prob, rows, I, da1, dprob,
                                        stream));
}

}  // extern "C"
