// Internal launcher interface between the C ABI (capi.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kMaxExperts = 64;
constexpr int kMaxTopK = 64;

typedef uint16_t bf16_t;

// A table of per-matrix (per-expert) device pointers, passed by value in the
// kernel arguments (64 x 8 B = 512 B).
struct MatTable {
    const void* p[kMaxExperts];
};

// ---- routing / permutation
size_t route_workspace_bytes(int64_t T, int E, int k);
// The no-allocation routing scratch: a static device array of this many bytes
// per device; route_scratch() returns its device address on the current
// device (taken once per device).
constexpr size_t kRouteScratchBytes = (size_t)8 << 20;
constexpr int kMaxDevices = 64;
hipError_t route_scratch(void** ptr);
hipError_t launch_route(const float* logits, int T, int E, int k, uint32_t flags,
                        int32_t* topk_expert, float* topk_prob, int32_t* split_sizes,
                        int32_t* expert_offsets, int32_t* dest_row, int32_t* src_token,
                        void* ws, hipStream_t s);
hipError_t launch_route_bwd(const float* topk_prob, const float* dprob_perm,
                            const int32_t* dest_row, const int32_t* topk_expert,
                            const float* logits, int T, int E, int k, uint32_t flags,
                            float* dlogits, hipStream_t s);
hipError_t launch_permute(const bf16_t* x, int T, int H, int k, const int32_t* dest_row,
                          const float* topk_prob, bf16_t* xp, float* prob_perm, hipStream_t s);
hipError_t launch_unpermute(const bf16_t* yp, int T, int H, int k, const int32_t* dest_row,
                            const float* topk_prob, bf16_t* y, hipStream_t s);

// ---- router linear layer
size_t router_bwd_workspace_bytes(int64_t T, int H, int E);
hipError_t launch_check_routing(const int32_t* split, int E, int64_t rows,
                                const int32_t* dest_row, const int32_t* src_token,
                                const int32_t* topk_expert, int64_t T, int k, int32_t* status,
                                hipStream_t s);
hipError_t launch_router_logits(const bf16_t* x, const bf16_t* w, int T, int H, int E,
                                float* logits, hipStream_t s);
hipError_t launch_router_bwd(const float* dlogits, const bf16_t* x, const bf16_t* w, int T,
                             int H, int E, int k, const int32_t* dest_row, const bf16_t* dxp,
                             bf16_t* dx, bf16_t* dw, void* ws, hipStream_t s);

// ---- MXFP8
int64_t colwise_block_bound(int64_t rows, int ngroups);
// scales_t: store the E8M0 scales block-major ([K/32][rows] for rowwise,
// [P_g/32][cols] per group for grouped columnwise), the layout the grouped
// GEMM reads with one coalesced load per K step; false = the public layout.
// Rowwise (rcodes given), grouped columnwise (ccodes given) or both, from one
// read of each matrix.
// p2_rows_pad > 0: the GEMM operand layouts (row-pair layout, common.hpp):
// row codes at expert-padded rows (groups from their 32-padded row bases),
// block-major row scales [cols/32][p2_rows_pad] (rscales_t required); grouped
// columnwise codes in the row-pair layout of [cols, 64-padded group rows] per
// group at cols * (sum of the earlier groups' 64-padded sizes), scales as in
// the public layout (cscales_t: block-major).  0: the public layouts.
hipError_t launch_quant(const MatTable& src, int nmat, const int32_t* sizes, int ngroups,
                        int64_t rows, int64_t cols, const MatTable* rcodes,
                        const MatTable* rscales, bool rscales_t, const MatTable* ccodes,
                        const MatTable* cscales, bool cscales_t, hipStream_t s,
                        const char* name, const float* fixed_amax = nullptr,
                        int64_t p2_rows_pad = 0, const int32_t* gather = nullptr);
// Per-tensor FP8: fixed_amax (device, one float per matrix) replaces the block
// maxima, so every block of matrix m gets the scale of amax[m].
// gather (one matrix, both orientations): row r of the quantized matrix is
// row gather[r] of src, so a permutation of token rows and their
// quantization are one pass.
// amax[m] = max |x| over matrix m's n values (n a multiple of 8); ws holds
// amax_workspace_bytes(nmat) bytes.
size_t amax_workspace_bytes(int nmat);
hipError_t launch_amax(const MatTable& src, int nmat, int64_t n, void* ws, float* amax,
                       hipStream_t s, const char* name);
// amax over the rows of a gathered matrix: rows x cols values, row r being
// row gather[r] of x (cols a multiple of 8); ws as for launch_amax(.., 1, ..).
hipError_t launch_amax_gather(const bf16_t* x, const int32_t* gather, int64_t rows, int64_t cols,
                              void* ws, float* amax, hipStream_t s, const char* name);
// The final reduction alone, over per-workgroup partials written elsewhere
// (the FP8 SwiGLU GEMM epilogues): amax[0] = the largest of part[0..nparts).
hipError_t launch_amax_final(const uint32_t* part, int nparts, float* amax, hipStream_t s,
                             const char* name);
hipError_t launch_quant_rows(const MatTable& src, const MatTable& codes, const MatTable& scales,
                             int nmat, int64_t rows, int64_t cols, hipStream_t s,
                             const char* name = "mx_quant_rows", bool scales_t = false,
                             int64_t p2_rows_pad = 0);
hipError_t launch_quant_cols(const MatTable& src, const MatTable& codes, const MatTable& scales,
                             int nmat, const int32_t* sizes, int ngroups, int64_t rows,
                             int64_t cols, hipStream_t s, const char* name = "mx_quant_cols",
                             bool scales_t = false, int64_t p2_rows_pad = 0);
// Bytes of an R x K 8-bit matrix in the row-pair layout.
inline size_t p2_bytes(int64_t R, int64_t K) {
    return (size_t)((R + 1) / 2) * (size_t)(((K + 63) / 64) * 128);
}
hipError_t launch_dequant_rows(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                               int64_t cols, bf16_t* out, hipStream_t s);
hipError_t launch_dequant_cols(const uint8_t* codes, const uint8_t* scales, const int32_t* sizes,
                               int ngroups, int64_t rows, int64_t cols, bf16_t* out,
                               hipStream_t s);

// ---- layer norm, ScaledSwiGLU
// xh as MXFP8 rows (codes [T, H], scales [T, H/32]) when codes is given.
constexpr int kMaxNormH = 32768;
constexpr int kMaxSwigluI = 1 << 20;
size_t layernorm_workspace_bytes(int64_t T, int H);
hipError_t launch_layernorm_fwd(const void* x, bool x_f32, int64_t T, int H, const void* gamma,
                                const void* beta, bool w_f32, float eps, bf16_t* y, float* mean,
                                float* rstd, uint8_t* codes, uint8_t* scales, hipStream_t s);
// xh from codes and scales when given, else from x, mean and rstd.
hipError_t launch_layernorm_bwd(const bf16_t* dy, const void* x, bool x_f32, const float* mean,
                                const float* rstd, const uint8_t* codes, const uint8_t* scales,
                                int64_t T, int H, const void* gamma, bool w_f32, const void* dres,
                                void* dx, void* dgamma, void* dbeta, void* ws, hipStream_t s);
hipError_t launch_swiglu_fwd(const bf16_t* a1, const float* prob, int64_t rows, int I, bf16_t* a2,
                             uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_swiglu_bwd(const bf16_t* da2, const bf16_t* a1, const uint8_t* codes,
                             const uint8_t* scales, const float* prob, int64_t rows, int I,
                             bf16_t* da1, float* dprob, hipStream_t s);

// ---- RMS norm with the residual's addition (h = x + residual in the stream's
// type, s_f32; written when there is a residual), y and / or 8-bit rows
size_t rmsnorm_workspace_bytes(int64_t T, int H);
hipError_t launch_rmsnorm_fwd(const void* x, bool x_f32, const void* residual, bool s_f32, int64_t T,
                              int H, const void* gamma, bool w_f32, float eps, void* h, bf16_t* y,
                              float* rstd, uint8_t* codes, float* scales, hipStream_t s);
hipError_t launch_rmsnorm_bwd(const bf16_t* dy, const void* h, bool s_f32, const float* rstd, int64_t T,
                              int H, const void* gamma, bool w_f32, const void* dres, void* dx,
                              bf16_t* branch, void* dgamma, void* ws, hipStream_t s);

// ---- balance and z loss of the router's logits
size_t balance_workspace_bytes(int E);
hipError_t launch_balance_fwd(const float* logits, int64_t T, int E, int k, const int32_t* topk,
                              const uint8_t* mask, float coef, float zcoef, float* loss, int32_t* counts,
                              int32_t* tokens, float* mean_prob, void* ws, hipStream_t s);
hipError_t launch_balance_bwd(const float* logits, int64_t T, int E, int k, const uint8_t* mask, float coef,
                              float zcoef, const int32_t* counts, const int32_t* tokens, const float* dloss,
                              const float* add, float* dlogits, hipStream_t s);

// ---- 8-bit blocks of 128 (block8.hpp): rows (scales [blocks][rows]), weights
// (scales [N/128][K/128], transposed codes on request), rows to bf16
hipError_t launch_quant_rows128(const bf16_t* x, int64_t rows, int cols, uint8_t* codes, float* scales,
                                hipStream_t s, const char* name);
hipError_t launch_quant_weights128(const MatTable& w, int nmat, int N, int K, const MatTable& codes,
                                   const MatTable& scales, const MatTable* codes_t, hipStream_t s);
hipError_t launch_dequant_rows128(const uint8_t* codes, const float* scales, const int32_t* src, int64_t x_rows,
                                  int64_t rows, int cols, bf16_t* out, hipStream_t s, const char* name);

// One grouped product of such operands: y rows of expert e = x rows times w_e^T.
struct BlockGemm {
    const uint8_t* x;           // [x_rows, K] codes
    const float* x_scale;       // [K/128][x_rows]
    int64_t x_rows;
    const int32_t* src;         // row r is x row src[r]; NULL: r
    const int32_t* split;
    int E;
    int64_t rows;
    int N, K;
    MatTable w;                 // [N, K] codes
    MatTable w_scale;           // block (n, k) at n * sn + k * sk
    int sn, sk;
    bf16_t* y;                  // [rows, N]
};
hipError_t launch_gemm_block(const BlockGemm& p, hipStream_t s, const char* name);

// Their weight gradients on bf16 operands: dw_e [N, K] = dy_e^T x_e.
struct WgradBlock {
    const bf16_t* dy;           // [rows, N]
    const bf16_t* x;            // [rows, K]
    const int32_t* split;
    int E;
    int64_t rows;
    int N, K;
    MatTable dw;
};
hipError_t launch_wgrad_block(const WgradBlock& p, hipStream_t s, const char* name);

}  // namespace moe
