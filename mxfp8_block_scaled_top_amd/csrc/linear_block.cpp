// C ABI of the 128-block 8-bit formats and of the grouped linear map over them:
// argument validation and launches.  The contracts are in include/moe_mi355x.h.
//
//   forward   y_e  = x^_e w^_e^T       8-bit operands, both blocked along K
//   dgrad     dx_e = Q(dy_e) w^_e      dy quantized along N here, the weights'
//                                      transposed codes with the same scales
//   wgrad     dW_e = dy_e^T x^_e       bf16 operands, x^ decoded here: blocks
//                                      along the rows would give both operands
//                                      a scale per output row and column, two
//                                      vector operations per product element;
//                                      and x^ = code * scale rounded to bf16
//                                      (2^-8 of each product at most) keeps dy
//                                      as it is
//
// 4099 rows over 8 experts of 4096 x 14336, us, the clock settled: dy's codes 12,
// dgrad 329 to 338, decoding 33, wgrad 476 to 504 (the clock of two cards).
#include "moe_mi355x.h"

#include <hip/hip_runtime.h>

#include "block8.hpp"
#include "kernels.hpp"
#include "mlp.hpp"

using namespace moe;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t al(size_t x) { return (x + 255) & ~(size_t)255; }

// x_rows: rows of the 8-bit operand; with src_token they are gathered
int check_block(int E, int N, int K, int64_t rows, int64_t x_rows, const void* src_token) {
    if (E < 1 || E > kMaxExperts) return MOE_ERR_SHAPE;
    if (N < 32 || K < 32 || (N % 32) || (K % 32)) return MOE_ERR_SHAPE;
    if (rows < 0 || rows > INT32_MAX || x_rows < 0 || x_rows > INT32_MAX) return MOE_ERR_SHAPE;
    if (!src_token && x_rows != rows) return MOE_ERR_SHAPE;
    // offsets inside one bf16 weight (gradient), 256 rows and the gathered codes
    if ((int64_t)N * K * 2 >= ((int64_t)1 << 31)) return MOE_ERR_SHAPE;
    if (N > (1 << 22) || K > (1 << 22)) return MOE_ERR_SHAPE;
    if (src_token && x_rows * K >= ((int64_t)1 << 31)) return MOE_ERR_SHAPE;
    // the kernels count tiles of 256 rows and 256 columns in int (smaller ones here: room)
    const int64_t widest = N > K ? N : K;
    if ((rows / 64 + E) * ((widest + 127) / 128) > INT32_MAX) return MOE_ERR_SHAPE;
    return MOE_OK;
}

struct BwdWs {
    uint8_t* dyq;
    float* dys;
    bf16_t* x;
    size_t bytes;
};

BwdWs carve(void* base, int64_t rows, int N, int K) {
    uint8_t* p = (uint8_t*)base;
    size_t off = 0;
    auto take = [&](size_t n) {
        uint8_t* r = p ? p + off : nullptr;
        off += al(n);
        return r;
    };
    BwdWs w{};
    w.dyq = take((size_t)rows * N);
    w.dys = (float*)take((size_t)rows * blocks_of(N) * 4);
    w.x = (bf16_t*)take((size_t)rows * K * 2);
    take(256);
    w.bytes = off;
    return w;
}

}  // namespace

namespace moe {
size_t linear_block_bwd_workspace_bytes(int64_t rows, int N, int K, int E) {
    if (check_block(E, N, K, rows, rows, nullptr) != MOE_OK) return 0;
    return carve(nullptr, rows, N, K).bytes;
}
}  // namespace moe

#define MOE_TRY(x)                                 \
    do {                                           \
        if ((x) != hipSuccess) return MOE_ERR_HIP; \
    } while (0)

extern "C" {

int fp8_block_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, float* scales,
                       hipStream_t stream) {
    if (rows < 0 || rows > INT32_MAX || cols < 8 || (cols % 8) || cols > INT32_MAX) return MOE_ERR_SHAPE;
    if (rows > 0 && (!x || !codes || !scales)) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_ALIGN;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    MOE_TRY(launch_quant_rows128(x, rows, (int)cols, codes, scales, stream, "fp8_block_quantize"));
    return MOE_OK;
}

int fp8_block_quantize_weights(int nmat, int64_t N, int64_t K, const uint16_t* const* w,
                               uint8_t* const* codes, float* const* scales, uint8_t* const* codes_t,
                               hipStream_t stream) {
    if (nmat < 1 || nmat > kMaxExperts) return MOE_ERR_SHAPE;
    // blocks of 256 threads for every 128 columns, at most 2^32 - 1 threads in a row
    if (N < 8 || K < 8 || (N % 8) || (K % 8) || N > (1 << 22) || K > (1 << 30)) return MOE_ERR_SHAPE;
    if (!w || !codes || !scales) return MOE_ERR_NULL;
    MatTable tw{}, tc{}, ts{}, tt{};
    for (int m = 0; m < nmat; ++m) {
        if (!w[m] || !codes[m] || !scales[m] || (codes_t && !codes_t[m])) return MOE_ERR_NULL;
        tw.p[m] = w[m];
        tc.p[m] = codes[m];
        ts.p[m] = scales[m];
        if (codes_t) tt.p[m] = codes_t[m];
        if (!aligned16(tw.p[m]) || !aligned16(tc.p[m]) || ((uintptr_t)ts.p[m] & 3) || !aligned16(tt.p[m]))
            return MOE_ERR_ALIGN;
    }
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    MOE_TRY(launch_quant_weights128(tw, nmat, (int)N, (int)K, tc, ts, codes_t ? &tt : nullptr, stream));
    return MOE_OK;
}

int grouped_linear_block_fwd(int E, int N, int K, int64_t rows, const uint8_t* x_codes,
                             const float* x_scales, int64_t x_rows, const int32_t* src_token,
                             const int32_t* split_sizes, const uint8_t* const* w_codes,
                             const float* const* w_scales, uint16_t* y, hipStream_t stream) {
    const int st = check_block(E, N, K, rows, x_rows, src_token);
    if (st != MOE_OK) return st;
    if (!split_sizes || !w_codes || !w_scales) return MOE_ERR_NULL;
    if (rows > 0 && (!y || (x_rows > 0 && (!x_codes || !x_scales)))) return MOE_ERR_NULL;
    BlockGemm g{};
    for (int e = 0; e < E; ++e) {
        if (!w_codes[e] || !w_scales[e]) return MOE_ERR_NULL;
        if (!aligned16(w_codes[e]) || ((uintptr_t)w_scales[e] & 3)) return MOE_ERR_ALIGN;
        g.w.p[e] = w_codes[e];
        g.w_scale.p[e] = w_scales[e];
    }
    if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(y)) return MOE_ERR_ALIGN;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    g.x = x_codes;
    g.x_scale = x_scales;
    g.x_rows = x_rows;
    g.src = src_token;
    g.split = split_sizes;
    g.E = E;
    g.rows = rows;
    g.N = N;
    g.K = K;
    g.sn = (int)blocks_of(K);
    g.sk = 1;
    g.y = y;
    MOE_TRY(launch_gemm_block(g, stream, "linear_block_fwd"));
    return MOE_OK;
}

int grouped_linear_block_bwd(int E, int N, int K, int64_t rows, const uint16_t* dy,
                             const uint8_t* x_codes, const float* x_scales, int64_t x_rows,
                             const int32_t* src_token, const int32_t* split_sizes,
                             const uint8_t* const* w_codes_t, const float* const* w_scales, uint16_t* dx,
                             uint16_t* const* dw, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    const int st = check_block(E, N, K, rows, x_rows, src_token);
    if (st != MOE_OK) return st;
    if (!split_sizes || !workspace) return MOE_ERR_NULL;
    if (dx && (!w_codes_t || !w_scales)) return MOE_ERR_NULL;
    BlockGemm g{};
    WgradBlock wg{};
    for (int e = 0; e < E; ++e) {
        if ((dx && (!w_codes_t[e] || !w_scales[e])) || (dw && !dw[e])) return MOE_ERR_NULL;
        if (dx && (!aligned16(w_codes_t[e]) || ((uintptr_t)w_scales[e] & 3))) return MOE_ERR_ALIGN;
        if (dw && !aligned16(dw[e])) return MOE_ERR_ALIGN;
        if (dx) {
            g.w.p[e] = w_codes_t[e];
            g.w_scale.p[e] = w_scales[e];
        }
        if (dw) wg.dw.p[e] = dw[e];
        for (int d = 0; dw && d < e; ++d)
            if (dw[d] == dw[e]) return MOE_ERR_ARG;     // an output of its own for every expert
    }
    if (rows > 0 && (!dy || (dw && x_rows > 0 && (!x_codes || !x_scales)))) return MOE_ERR_NULL;
    if (!aligned16(dy) || !aligned16(x_codes) || !aligned16(x_scales) || !aligned16(dx) || !aligned16(workspace))
        return MOE_ERR_ALIGN;
    const BwdWs ws = carve(workspace, rows, N, K);
    if (workspace_bytes < ws.bytes) return MOE_ERR_WORKSPACE;
    if (!moe_device_supported()) return MOE_ERR_UNSUPPORTED;
    if (dx && rows > 0) {
        MOE_TRY(launch_quant_rows128(dy, rows, N, ws.dyq, ws.dys, stream, "linear_block_quant_dy"));
        g.x = ws.dyq;
        g.x_scale = ws.dys;
        g.x_rows = rows;
        g.split = split_sizes;
        g.E = E;
        g.rows = rows;
        g.N = K;
        g.K = N;
        g.sn = 1;
        g.sk = (int)blocks_of(K);
        g.y = dx;
        MOE_TRY(launch_gemm_block(g, stream, "linear_block_dgrad"));
    }
    if (dw) {
        MOE_TRY(launch_dequant_rows128(x_codes, x_scales, src_token, x_rows, rows, K, ws.x, stream,
                                       "linear_block_decode_x"));
        wg.dy = dy;
        wg.x = ws.x;
        wg.split = split_sizes;
        wg.E = E;
        wg.rows = rows;
        wg.N = N;
        wg.K = K;
        MOE_TRY(launch_wgrad_block(wg, stream, "linear_block_wgrad"));
    }
    return MOE_OK;
}

}  // extern "C"
