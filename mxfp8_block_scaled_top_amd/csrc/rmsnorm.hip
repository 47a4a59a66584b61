// RMS norm in front of the router, with the residual's addition and the rows
// in 8 bits, forward and backward, for gfx950.
//
//   forward   h = x + residual (rounded to the stream's type),
//             rstd = (sum h^2 / H + eps)^-1/2,  y = h rstd gamma,
//             as bf16 rows (the router's) and / or as E4M3 rows with an fp32
//             scale per 128 values (the experts': block8.hpp), from the fp32 y
//   backward  xh = h rstd,  g = dy gamma,  dx = rstd (g - xh mean(g xh)) [+ dres],
//             dgamma = sum_t dy xh
//
// Bound by HBM bytes, and built like the layer norm (norm.hpp): every row is
// read once and stays in registers, sums are fp32, a workgroup walks over rows
// with gamma in registers, the gradient of gamma leaves as one partial row per
// workgroup and is added in a fixed order by a second kernel.  The norm is
// taken of the stored (rounded) h, which is what the backward sees.  A block of
// 128 values is the 16 lanes of a row of lanes, so its largest magnitude takes
// four lane shifts.  The scales are stored [blocks][rows], the order in which
// the products read them; a row's 4-byte pieces of it are 2% of its bytes.
//
// Measured (a copy of 1 GiB: 5.1 TB/s): forward of 8192 x 4096 bf16 with residual, y
// and codes 54 us (5.6 TB/s), into an fp32 stream 85, of fp32 rows 99; 4096 x 16384 bf16
// 110, fp32 193 (all 5.1 to 5.5 TB/s).  Backward of 16384 x 2048 over an fp32 stream, with
// the residual's gradient and the bf16 copy, 103 to 104 + 5 us (5.2 TB/s); 8192 x 4096 bf16 45.
// Above 8192 columns gamma's gradient reads dy and h again: 4096 x 16384 bf16 117 us for
// 68 without it, fp32 with residual 242 for 174.  One row of 4096: 2.9 us, the time
// of an empty launch and a read after it.
#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"
#include "norm.hpp"
#include "trace.hpp"

namespace moe {

namespace {

struct RmsFwd {
    const void* x;
    const void* residual;   // NULL: h = x, which is not written
    const void* gamma;
    void* h;
    bf16_t* y;              // or NULL
    float* rstd;            // or NULL
    uint8_t* codes;         // or NULL
    float* scales;
    int64_t T;
    int H;
    int w_f32;
    float eps;
};

template <bool XF32, bool SF32, class S>
__global__ __launch_bounds__(S::kThreads) void rms_fwd_kernel(RmsFwd a) {
    constexpr int kV = S::kV, kPer = S::kPer;
    __shared__ float red[2][16][1];
    const int l = S::place();
    const int nc = a.H / 8;
    const float inv = 1.f / (float)a.H;
    const int64_t step = (int64_t)gridDim.x * S::kRows;
    int64_t r0 = (int64_t)blockIdx.x * S::kRows;    // the same for the workgroup
    const int mine = S::row();
    Raw8<XF32> nx[kV];
    Raw8<SF32> nr[kV];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            nx[v] = Raw8<XF32>{};
            nr[v] = Raw8<SF32>{};
            if (row < a.T && c < nc) {
                nx[v] = load_raw<XF32>(a.x, row * a.H + c * 8);
                if (a.residual) nr[v] = load_raw<SF32>(a.residual, row * a.H + c * 8);
            }
        }
    };
    load(r0 + mine);
    float gm[kV][8];
    auto load_w = [&](int v) {
        const int c = l + v * kPer;
        load_w8(c < nc ? a.gamma : nullptr, a.w_f32, (int64_t)c * 8, 1.f, gm[v]);
    };
    if (!S::kLean)
#pragma unroll
        for (int v = 0; v < kV; ++v) load_w(v);
    int flip = 0;
    for (; r0 < a.T; r0 += step) {
        const int64_t r = r0 + mine;
        const bool live = r < a.T;
        float x[kV][8];
        float q[1] = {0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            unpack<XF32>(nx[v], x[v]);
            if (a.residual) {
                float d[8];
                unpack<SF32>(nr[v], d);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[v][k] += d[k];
                Raw8<SF32> w;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (SF32) {
                        w.w[0][k] = __float_as_uint(x[v][k]);
                        w.w[1][k] = __float_as_uint(x[v][4 + k]);
                    } else {
                        w.w[0][k] = pack_bf16x2(x[v][2 * k], x[v][2 * k + 1]);
                    }
                }
                unpack<SF32>(w, x[v]);
                const int c = l + v * kPer;
                if (live && c < nc) {
                    u32x4* o = (u32x4*)((char*)a.h + (r * a.H + c * 8) * (SF32 ? 4 : 2));
#pragma unroll
                    for (int k = 0; k < (SF32 ? 2 : 1); ++k) __builtin_nontemporal_store(w.w[k], o + k);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) q[0] += x[v][k] * x[v][k];
        }
        if (!S::kLean) load(r + step);      // the next row's, in flight through this row's work
        row_sum<S, 1>(q, red[flip]);
        flip ^= 1;
        const float rstd = inv_sqrt(q[0] * inv + a.eps);
        if (live && l == 0 && a.rstd) a.rstd[r] = rstd;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            const bool in = live && c < nc;
            if (S::kLean) load_w(v);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[v][k] = x[v][k] * rstd * gm[v][k];
            if (a.y && in) store8<false>(a.y, r * a.H + c * 8, x[v]);
            if (a.codes) {                  // every lane, for the block's maximum
                if (!in)
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[v][k] = 0.f;      // 0 rstd may be NaN
                float scale;
                const u32x2 w = blk_encode8(x[v], scale);
                if (in) {
                    __builtin_nontemporal_store(w, (u32x2*)(a.codes + r * a.H + c * 8));
                    if ((c & 15) == 0) a.scales[(int64_t)(c >> 4) * a.T + r] = scale;
                }
            }
        }
        if (S::kLean) load(r + step);
    }
}

struct RmsBwd {
    const bf16_t* dy;
    const void* h;
    const float* rstd;
    const void* gamma;
    const void* dres;
    void* dx;
    bf16_t* branch;    // dx again in bf16, or NULL
    float* part;       // [gridDim.x][H], or NULL
    int64_t T;
    int H;
    int w_f32;
};

// What a row brings: dy and h, as loaded.  They are unpacked twice, for the
// sums and for dx: fewer registers than the fp32 values would hold.
template <bool SF32, int kV>
struct RmsRow {
    float rstd;
    Raw8<false> dy[kV];
    Raw8<SF32> h[kV];
};

// kSums: also gamma's gradient, one partial row of H floats per workgroup.
template <bool SF32, class S, bool kSums>
__global__ __launch_bounds__(S::kThreads) void rms_bwd_kernel(RmsBwd a) {
    constexpr int kV = S::kV, kRows = S::kRows, kPer = S::kPer;
    constexpr int kPart = kRows * S::kLanes / 64;   // rows left after each wave has added its own
    // The next row's loads go out ahead of a row's work for an fp32 stream, behind it
    // for a bf16 one (us, ahead / behind, other data in every call: fp32 16384 x 2048
    // 104.2 / 106.0, 8192 x 4096 106.0 / 110.3, 4096 x 8192 110.2 / 113.9, bf16 the same to
    // 0.5%; the same data in every call, part of it in the last-level cache: fp32 104.3 /
    // 101.6, bf16 50.3 / 44.6).
    constexpr bool kPrefetch = SF32 && !S::kLean;
    __shared__ float red[2][16][1];
    __shared__ float comb[kSums && kPart > 1 ? 8 * kPer * kV : 1];
    const int l = S::place();
    const int nc = a.H / 8;
    const float inv = 1.f / (float)a.H;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t r0 = (int64_t)blockIdx.x * kRows;       // the same for the workgroup
    const int mine = S::row();
    using Row = RmsRow<SF32, kV>;
    auto load = [&](int64_t row, Row& n) {
        const bool live = row < a.T;
        n.rstd = live ? a.rstd[row] : 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            n.dy[v] = Raw8<false>{};
            n.h[v] = Raw8<SF32>{};
            if (live && c < nc) {
                const int64_t at = row * a.H + c * 8;
                n.dy[v] = load_raw<false>(a.dy, at);
                n.h[v] = load_raw<SF32>(a.h, at);
            }
        }
    };
    // step v of a row: dy and xh, both 0 in lanes past the row's end (0 rstd
    // is NaN where rstd is not finite, but only the row's own lanes then)
    auto values = [&](const Row& w, int v, float (&dy)[8], float (&xh)[8]) {
        unpack<false>(w.dy[v], dy);
        unpack<SF32>(w.h[v], xh);
        const float r = l + v * kPer < nc ? w.rstd : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) xh[k] *= r;
    };
    Row next;
    load(r0 + mine, next);
    float gm[kV][8];
    float dg[kSums ? kV : 1][8];
    auto load_w = [&](int v) {
        const int c = l + v * kPer;
        load_w8(c < nc ? a.gamma : nullptr, a.w_f32, (int64_t)c * 8, 1.f, gm[v]);
    };
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        if (!S::kLean) load_w(v);
        if constexpr (kSums)
#pragma unroll
            for (int k = 0; k < 8; ++k) dg[v][k] = 0.f;
    }
    int flip = 0;
    for (; r0 < a.T; r0 += step) {
        const int64_t r = r0 + mine;
        Row row = next;
        Raw8<SF32> res[kV];                     // the residual's gradient, used last
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            res[v] = Raw8<SF32>{};
            if (a.dres && r < a.T && c < nc) res[v] = load_raw<SF32>(a.dres, r * a.H + c * 8);
        }
        if (kPrefetch) load(r + step, next);
        float s[1] = {0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            float dy[8], xh[8];
            if (S::kLean) load_w(v);
            values(row, v, dy, xh);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float t = dy[k] * xh[k];
                s[0] += t * gm[v][k];
                if constexpr (kSums) dg[v][k] += t;
            }
        }
        row_sum<S, 1>(s, red[flip]);
        flip ^= 1;
        const float c2 = s[0] * inv;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            forget(row.dy[v]);
            forget(row.h[v]);
        }
        if (r < a.T) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = l + v * kPer;
                if (c >= nc) continue;
                float dy[8], xh[8], d[8], o[8];
                if (S::kLean) load_w(v);
                values(row, v, dy, xh);
                unpack<SF32>(res[v], d);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = row.rstd * (dy[k] * gm[v][k] - xh[k] * c2) + d[k];
                store8<SF32>(a.dx, r * a.H + c * 8, o);
                if (a.branch) store8<false>(a.branch, r * a.H + c * 8, o);
            }
        }
        if (!kPrefetch) load(r + step, next);
    }
    if constexpr (!kSums) return;
    float* out = a.part + (int64_t)blockIdx.x * a.H;
    const int part = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) / S::kWpr;
    // the rows of a wave, then the workgroup's in order through LDS
    if constexpr (S::kLanes < 64)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float& t = dg[0][k];
            static_assert(S::kLanes == 64 || kV == 1, "short rows have one step");
            if (S::kLanes == 16) t += __shfl_xor(t, 16);
            t += __shfl_xor(t, 32);
        }
#pragma unroll
    for (int w = 0; w < kPart; ++w) {
        if (kPart > 1) __syncthreads();
        if (part != w || (S::kLanes < 64 && (threadIdx.x & 63) >= S::kLanes)) continue;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            if (c >= nc) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float* q = &dg[v][4 * h];
                float4 t = make_float4(q[0], q[1], q[2], q[3]);
                if (kPart > 1) {
                    float4* m = (float4*)comb + 2 * c + h;
                    if (w > 0) {
                        const float4 o = *m;
                        t = make_float4(o.x + t.x, o.y + t.y, o.z + t.z, o.w + t.w);
                    }
                    if (w < kPart - 1) *m = t;
                }
                if (w == kPart - 1) ((float4*)out)[2 * c + h] = t;
            }
        }
    }
}

// gamma's gradient of rows too wide for a workgroup to hold its sums beside
// the row: a second read of dy and h.  A wave has 512 columns; workgroup (x, y)
// adds rows y, y + gridDim.y, .. of 4 waves each and writes its columns of
// partial row y.
template <bool SF32>
__global__ __launch_bounds__(256) void rms_cols_kernel(RmsBwd a) {
    __shared__ float comb[3][512];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int c = blockIdx.x * 64 + lane;
    const bool in = c < a.H / 8;
    float dg[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[k] = 0.f;
#pragma unroll 4
    for (int64_t r = (int64_t)blockIdx.y * 4 + wave; r < a.T; r += (int64_t)gridDim.y * 4) {
        if (!in) continue;
        const int64_t at = r * a.H + c * 8;
        float dy[8], xh[8];
        unpack<false>(load_raw<false>(a.dy, at), dy);
        unpack<SF32>(load_raw<SF32>(a.h, at), xh);
        const float rstd = a.rstd[r];
#pragma unroll
        for (int k = 0; k < 8; ++k) dg[k] += dy[k] * (xh[k] * rstd);
    }
    if (wave > 0)
#pragma unroll
        for (int k = 0; k < 8; ++k) comb[wave - 1][k * 64 + lane] = dg[k];
    __syncthreads();
    if (wave > 0 || !in) return;
    float* out = a.part + (int64_t)blockIdx.y * a.H + c * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int w = 0; w < 3; ++w) dg[k] += comb[w][k * 64 + lane];
        out[k] = dg[k];
    }
}

// The np partial rows added in a fixed order.  A workgroup has 8 columns and
// 128 threads on each, every one with every 128th row: few dependent loads.
__global__ __launch_bounds__(1024) void rms_dw_reduce_kernel(const float* __restrict__ part, int np,
                                                             int H, int w_f32, void* dgamma) {
    __shared__ float red[128][9];
    const int q = threadIdx.x >> 3, col = threadIdx.x & 7;
    const int i = blockIdx.x * 8 + col;                  // H is a multiple of 8
    float t = 0.f;
#pragma unroll 4
    for (int p = q; p < np; p += 128) t += part[(int64_t)p * H + i];
    red[q][col] = t;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    t = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += red[q * 16 + w][col];     // 8 threads per column, 16 rows each
    t += __shfl_xor(t, 8);
    t += __shfl_xor(t, 16);
    t += __shfl_xor(t, 32);
    if (q) return;
    if (w_f32) ((float*)dgamma)[i] = t;
    else ((bf16_t*)dgamma)[i] = (bf16_t)f32_to_bf16(t);
}

// Rows up to kRmsSumsH have gamma's sums beside them in registers; wider ones
// read dy and h again for them (4096 x 8192, fp32 stream: 108 us with the sums,
// 134 with a kernel of their own; bf16 49 and 63; 300 rows 17.0 and 15.8).
//
// One wave per 512 columns of a row as far as a workgroup goes, not half as many
// with two steps each (us, one step / two: fp32 stream 16384 x 1024 52.5 / 54.5, 16384 x 2048
// 101.2 / 103.4, 8192 x 4096 104.3 / 108.0, 4096 x 8192 108.5 / 116.6; bf16 41.0 / 41.2,
// 42.0 / 42.2, 44.6 / 46.2, 48.8 / 53.0).
constexpr int kRmsSumsH = 8192;
template <class F>
void with_bwd_shape(int H, F&& f) {
    if (H <= 128) f(Shape<16, 1, 1, 32>{});
    else if (H <= 256) f(Shape<32, 1, 1, 16>{});
    else if (H <= 512) f(Shape<64, 1, 1, 8>{});
    else if (H <= 1024) f(Shape<64, 2, 1, 8>{});
    else if (H <= 2048) f(Shape<64, 4, 1, 4>{});
    else if (H <= 4096) f(Shape<64, 8, 1, 2>{});
    else if (H <= 8192) f(Shape<64, 16, 1, 1>{});
    else if (H <= 16384) f(Shape<64, 16, 2, 1>{});
    else f(Shape<64, 16, 4, 1>{});
}

template <class S>
unsigned bwd_groups(int64_t T) {
    return groups_of<S>(T, S::kThreads >= 1024 ? 1 : 2);
}

// Partial rows of gamma's gradient.
int rms_parts(int64_t T, int H) {
    if (H > kRmsSumsH) {    // about 1024 workgroups of the column kernel
        const int64_t need = (T + 3) / 4, cap = 1024 / ((H + 511) / 512);
        return (int)(need < cap ? need : cap);
    }
    int n = 0;
    with_bwd_shape(H, [&](auto s) { n = (int)bwd_groups<decltype(s)>(T); });
    return n;
}

template <bool XF32, bool SF32>
void run_fwd(const RmsFwd& a, hipStream_t s) {
    with_fwd_shape(a.H, [&](auto sh) {
        using S = decltype(sh);
        rms_fwd_kernel<XF32, SF32, S><<<fwd_groups<S>(a.T), S::kThreads, 0, s>>>(a);
    });
}

template <bool SF32>
hipError_t run_bwd(const RmsBwd& a, hipStream_t s) {
    const bool sums = a.part && a.H <= kRmsSumsH;
    if (a.part && !sums) {
        TraceScope ts("rmsnorm_cols", s);
        rms_cols_kernel<SF32><<<dim3((unsigned)((a.H + 511) / 512), (unsigned)rms_parts(a.T, a.H)),
                                256, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    TraceScope ts("rmsnorm_bwd", s);
    with_bwd_shape(a.H, [&](auto sh) {
        using S = decltype(sh);
        if (!sums)
            rms_bwd_kernel<SF32, S, false><<<bwd_groups<S>(a.T), S::kThreads, 0, s>>>(a);
        else if constexpr (8 * S::kPer * S::kV <= kRmsSumsH)
            rms_bwd_kernel<SF32, S, true><<<bwd_groups<S>(a.T), S::kThreads, 0, s>>>(a);
    });
    return hipGetLastError();
}

}  // namespace

size_t rmsnorm_workspace_bytes(int64_t T, int H) {
    return (size_t)rms_parts(T, H) * (size_t)H * sizeof(float) + 256;
}

hipError_t launch_rmsnorm_fwd(const void* x, bool x_f32, const void* residual, bool s_f32, int64_t T,
                              int H, const void* gamma, bool w_f32, float eps, void* h, bf16_t* y,
                              float* rstd, uint8_t* codes, float* scales, hipStream_t s) {
    if (T == 0) return hipSuccess;
    RmsFwd a{x, residual, gamma, h, y, rstd, codes, scales, T, H, w_f32 ? 1 : 0, eps};
    TraceScope ts("rmsnorm_fwd", s);
    if (x_f32) run_fwd<true, true>(a, s);
    else if (s_f32) run_fwd<false, true>(a, s);
    else run_fwd<false, false>(a, s);
    return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const bf16_t* dy, const void* h, bool s_f32, const float* rstd, int64_t T,
                              int H, const void* gamma, bool w_f32, const void* dres, void* dx,
                              bf16_t* branch, void* dgamma, void* ws, hipStream_t s) {
    if (T > 0) {
        RmsBwd a{dy, h, rstd, gamma, dres, dx, branch, dgamma ? (float*)ws : nullptr, T, H, w_f32 ? 1 : 0};
        const hipError_t e = s_f32 ? run_bwd<true>(a, s) : run_bwd<false>(a, s);
        if (e != hipSuccess) return e;
    }
    if (!dgamma) return hipSuccess;
    TraceScope ts("rmsnorm_dw_reduce", s);
    rms_dw_reduce_kernel<<<(unsigned)(H / 8), 1024, 0, s>>>((const float*)ws, T > 0 ? rms_parts(T, H) : 0,
                                                            H, w_f32 ? 1 : 0, dgamma);
    return hipGetLastError();
}

}  // namespace moe
