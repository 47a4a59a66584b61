// Layer norm in front of the router, forward and backward, for gfx950.
//
//   forward   mean = sum x / H,  var = sum (x - mean)^2 / H,
//             rstd = (var + eps)^-1/2,  xh = (x - mean) rstd,
//             y = xh gamma + beta; optionally xh as MXFP8 rows, the 8-bit
//             checkpoint that the backward reads in place of x
//   backward  g = dy gamma,  dx = rstd (g - mean(g) - xh mean(g xh)) [+ dres],
//             dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Both are bound by HBM bytes (about 10 operations per element).  Every row
// is read once: one or several waves (or a part of one) hold it in registers,
// 8 neighbouring values per lane and step (16 bytes of bf16), and all sums
// over the row come from the registers, the variance around the mean already
// known, so nothing cancels.  Sums are fp32; the only roundings to fewer bits
// are the stored y, dx and codes.
//
// A workgroup walks over rows with gamma (and beta) in registers: read per
// row they would be more bytes from L2 than the row itself.  The backward
// keeps its workgroup's dgamma and dbeta in registers over that walk and
// writes them once, as one partial row per workgroup; a second kernel adds
// the partial rows in a fixed order (no atomics: the same bits every time).
//
// Measured with bf16 rows, 168 MB a pass: forward with checkpoint 31 us at
// 16384 x 2048 and 8192 x 4096 (5.4 TB/s; a large copy reaches 5.2); backward
// from the checkpoint 40 to 43 us (4.0 to 4.3 TB/s), of which the rows' kernel
// 36 us and the second one 4 us.  One row of 4096: 3.1 us, the launch and two trips to
// memory.
#include "common.hpp"
#include "kernels.hpp"
#include "norm.hpp"
#include "trace.hpp"

namespace moe {

namespace {

struct LnFwd {
    const void* x;
    const void* gamma;
    const void* beta;
    bf16_t* y;
    float* mean;
    float* rstd;
    uint8_t* codes;
    uint8_t* scales;
    int64_t T;
    int H;
    int w_f32;
    float eps;
};

template <bool XF32, class S>
__global__ __launch_bounds__(S::kThreads) void ln_fwd_kernel(LnFwd a) {
    constexpr int kV = S::kV, kPer = S::kPer;
    __shared__ float red[2][16][1];
    const int l = S::place();
    const int nc = a.H / 8;
    const float inv = 1.f / (float)a.H;
    const int64_t step = (int64_t)gridDim.x * S::kRows;
    int64_t r0 = (int64_t)blockIdx.x * S::kRows;    // the same for the workgroup
    const int mine = S::row();
    Raw8<XF32> next[kV];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            next[v] = Raw8<XF32>{};
            if (row < a.T && c < nc) next[v] = load_raw<XF32>(a.x, row * a.H + c * 8);
        }
    };
    load(r0 + mine);
    float gm[kV][8], bt[kV][8];
    auto load_w = [&](int v) {
        const int c = l + v * kPer;
        load_w8(c < nc ? a.gamma : nullptr, a.w_f32, (int64_t)c * 8, 1.f, gm[v]);
        load_w8(c < nc ? a.beta : nullptr, a.w_f32, (int64_t)c * 8, 0.f, bt[v]);
    };
    if (!S::kLean)
#pragma unroll
        for (int v = 0; v < kV; ++v) load_w(v);
    for (; r0 < a.T; r0 += step) {
        const int64_t r = r0 + mine;
        float x[kV][8];
        float s[1] = {0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            unpack<XF32>(next[v], x[v]);
#pragma unroll
            for (int k = 0; k < 8; ++k) s[0] += x[v][k];
        }
        if (!S::kLean) load(r + step);      // the next row's, in flight through this row's work
        row_sum<S, 1>(s, red[0]);
        const float mean = s[0] * inv;
        float q[1] = {0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const bool in = l + v * kPer < nc;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[v][k] = in ? x[v][k] - mean : 0.f;
                q[0] += x[v][k] * x[v][k];
            }
        }
        row_sum<S, 1>(q, red[1]);
        const float rstd = inv_sqrt(q[0] * inv + a.eps);
        if (r < a.T) {
            if (l == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = l + v * kPer;
                if (c >= nc) continue;
                if (S::kLean) load_w(v);
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[v][k] *= rstd;
                    y[k] = x[v][k] * gm[v][k] + bt[v][k];
                }
                store8<false>(a.y, r * a.H + c * 8, y);
                if (a.codes) mx_store8(x[v], a.codes + r * a.H + c * 8,
                                       a.scales + r * (a.H / 32) + c / 4);
            }
        }
        if (S::kLean) load(r + step);
    }
}

struct LnBwd {
    const bf16_t* dy;
    const void* x;
    const float* mean;
    const float* rstd;
    const uint8_t* codes;
    const uint8_t* scales;
    const void* gamma;
    const void* dres;
    void* dx;
    float* part;       // [gridDim.x][2 H], or NULL
    int64_t T;
    int H;
    int w_f32;
};

enum LnSaved { LN_BF16 = 0, LN_F32 = 1, LN_MX_BF16 = 2, LN_MX_F32 = 3 };  // xh from x or from codes; dx type

// 8 values of xh as they are kept: x's words, or 8 codes and their scale
template <int kSaved>
struct SavedRaw {
    Raw8<kSaved == LN_F32> x;
};
template <>
struct SavedRaw<LN_MX_BF16> {
    u32x2 codes;
    uint32_t scale;
};
template <>
struct SavedRaw<LN_MX_F32> : SavedRaw<LN_MX_BF16> {};

template <int kSaved>
__device__ __forceinline__ void forget_saved(SavedRaw<kSaved>& r) {
    if constexpr (kSaved >= LN_MX_BF16) forget(r.codes);
    else forget(r.x);
}

// What a row brings: dy, the saved row and the residual's gradient, as loaded.
// They are unpacked twice, for the sums and for dx: fewer registers than the
// fp32 values would hold over the sums.
template <int kSaved, int kV>
struct LnRow {
    float rstd, mean;
    Raw8<false> dy[kV];
    SavedRaw<kSaved> x[kV];
};

// kSums: also the weights' gradients, one partial row of 2H floats per workgroup.
template <int kSaved, class S, bool kSums>
__global__ __launch_bounds__(S::kThreads) void ln_bwd_kernel(LnBwd a) {
    constexpr bool XF32 = kSaved == LN_F32 || kSaved == LN_MX_F32;
    constexpr bool kMx = kSaved >= LN_MX_BF16;
    constexpr int kV = S::kV, kRows = S::kRows, kPer = S::kPer;
    constexpr int kPart = kRows * S::kLanes / 64;   // rows left after each wave has added its own
    // The next row is loaded during the current one where dx is fp32; with
    // the smaller bf16 rows the other waves hide the loads as well, with
    // fewer registers (16384 x 2048: fp32 69 against 73 us without, bf16 45.5
    // against 44.0).
    constexpr bool kPrefetch = XF32 && !S::kLean;
    __shared__ float red[2][16][2];
    __shared__ float comb[kSums && kPart > 1 ? 8 * kPer * kV : 1];
    const int l = S::place();
    const int nc = a.H / 8;
    const float inv = 1.f / (float)a.H;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t r0 = (int64_t)blockIdx.x * kRows;       // the same for the workgroup
    const int mine = S::row();
    using Row = LnRow<kSaved, kV>;
    auto load = [&](int64_t row, Row& n) {
        const bool live = row < a.T;
        n.rstd = live ? a.rstd[row] : 0.f;
        n.mean = !kMx && live ? a.mean[row] : 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            n.dy[v] = Raw8<false>{};
            n.x[v] = SavedRaw<kSaved>{};
            if (live && c < nc) {
                const int64_t at = row * a.H + c * 8;
                n.dy[v] = load_raw<false>(a.dy, at);
                if constexpr (kMx) {
                    n.x[v].codes = __builtin_nontemporal_load((const u32x2*)(a.codes + at));
                    n.x[v].scale = a.scales[row * (a.H / 32) + c / 4];
                } else {
                    n.x[v].x = load_raw<XF32>(a.x, at);
                }
            }
        }
    };
    // step v of a row: dy and xh.  A lane past the row's end must add nothing to
    // the sums: it holds dy = 0 and, with a mean of 0 of its own, xh = 0 (mean
    // rstd itself may be past fp32's range where (x - mean) rstd is not).  The
    // widest rows skip such lanes instead: 1024 x 32768 fp32 126 us, with the
    // lanes' means 154; for all the other widths skipping costs 1 to 2%.
    auto values = [&](const Row& w, int v, float (&dy)[8], float (&xh)[8]) {
        unpack<false>(w.dy[v], dy);
        if constexpr (kMx) {
            mx_decode8(w.x[v].codes, w.x[v].scale, xh);
        } else {
            unpack<XF32>(w.x[v].x, xh);
            const float mean = S::kLean || l + v * kPer < nc ? w.mean : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) xh[k] = (xh[k] - mean) * w.rstd;
        }
    };
    Row next;
    load(r0 + mine, next);
    float gm[kV][8];
    float dg[kSums ? kV : 1][8], db[kSums ? kV : 1][8];
    auto load_w = [&](int v) {
        const int c = l + v * kPer;
        load_w8(c < nc ? a.gamma : nullptr, a.w_f32, (int64_t)c * 8, 1.f, gm[v]);
    };
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        if (!S::kLean) load_w(v);
        if constexpr (kSums)
#pragma unroll
            for (int k = 0; k < 8; ++k) dg[v][k] = db[v][k] = 0.f;
    }
    int flip = 0;
    for (; r0 < a.T; r0 += step) {
        const int64_t r = r0 + mine;
        Row row = next;
        Raw8<XF32> res[kV];                     // the residual's gradient, used last
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * kPer;
            res[v] = Raw8<XF32>{};
            if (a.dres && r < a.T && c < nc) res[v] = load_raw<XF32>(a.dres, r * a.H + c * 8);
        }
        if (kPrefetch) load(r + step, next);    // in flight through this row's work
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            float dy[8], xh[8];
            if (S::kLean && l + v * kPer >= nc) continue;
            if (S::kLean) load_w(v);
            values(row, v, dy, xh);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float g = dy[k] * gm[v][k];
                s[0] += g;
                s[1] += g * xh[k];
                if constexpr (kSums) {
                    dg[v][k] += dy[k] * xh[k];
                    db[v][k] += dy[k];
                }
            }
        }
        row_sum<S, 2>(s, red[flip]);
        flip ^= 1;
        const float c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            forget(row.dy[v]);
            forget_saved(row.x[v]);
        }
        if (r < a.T) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = l + v * kPer;
                if (c >= nc) continue;
                float dy[8], xh[8], d[8], o[8];
                if (S::kLean) load_w(v);
                values(row, v, dy, xh);
                unpack<XF32>(res[v], d);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    o[k] = row.rstd * (dy[k] * gm[v][k] - c1 - xh[k] * c2) + d[k];
                store8<XF32>(a.dx, r * a.H + c * 8, o);
            }
        }
        if (!kPrefetch) load(r + step, next);
    }
    if constexpr (!kSums) return;
    float* out = a.part + (int64_t)blockIdx.x * 2 * a.H;
    const int part = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) / S::kWpr;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        // the rows of a wave, then the workgroup's in order through LDS
        if constexpr (S::kLanes < 64)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float& t = which ? db[0][k] : dg[0][k];
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
                float4 t[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float* q = which ? &db[v][4 * h] : &dg[v][4 * h];
                    t[h] = make_float4(q[0], q[1], q[2], q[3]);
                    if (kPart > 1) {
                        float4* m = (float4*)comb + 2 * c + h;
                        if (w > 0) {
                            const float4 o = *m;
                            t[h] = make_float4(o.x + t[h].x, o.y + t[h].y, o.z + t[h].z, o.w + t[h].w);
                        }
                        if (w < kPart - 1) *m = t[h];
                    }
                    if (w == kPart - 1) ((float4*)(out + which * a.H))[2 * c + h] = t[h];
                }
            }
        }
    }
}

// The weights' gradients of rows too wide for a workgroup to hold their sums
// beside the row: a second read of dy and of the saved rows.  A wave has 512
// columns; workgroup (x, y) adds rows y, y + gridDim.y, .. of 4 waves each and
// writes its columns of partial row y.
template <int kSaved>
__global__ __launch_bounds__(256) void ln_cols_kernel(LnBwd a) {
    constexpr bool kMx = kSaved >= LN_MX_BF16;
    __shared__ float comb[3][2][512];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int c = blockIdx.x * 64 + lane;
    const bool in = c < a.H / 8;
    float dg[8], db[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[k] = db[k] = 0.f;
#pragma unroll 4
    for (int64_t r = (int64_t)blockIdx.y * 4 + wave; r < a.T; r += (int64_t)gridDim.y * 4) {
        if (!in) continue;
        const int64_t at = r * a.H + c * 8;
        float dy[8], xh[8];
        unpack<false>(load_raw<false>(a.dy, at), dy);
        if constexpr (kMx) {
            mx_load8(a.codes + at, a.scales + r * (a.H / 32) + c / 4, xh);
        } else {
            unpack<kSaved == LN_F32>(load_raw<kSaved == LN_F32>(a.x, at), xh);
            const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
            for (int k = 0; k < 8; ++k) xh[k] = (xh[k] - mean) * rstd;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            dg[k] += dy[k] * xh[k];
            db[k] += dy[k];
        }
    }
    if (wave > 0)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            comb[wave - 1][0][k * 64 + lane] = dg[k];
            comb[wave - 1][1][k * 64 + lane] = db[k];
        }
    __syncthreads();
    if (wave > 0 || !in) return;
    float* out = a.part + (int64_t)blockIdx.y * 2 * a.H + c * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            dg[k] += comb[w][0][k * 64 + lane];
            db[k] += comb[w][1][k * 64 + lane];
        }
        out[k] = dg[k];
        out[a.H + k] = db[k];
    }
}

// dgamma (columns [0, H)) and dbeta ([H, 2H)): the np partial rows added in a
// fixed order.  A workgroup has 16 columns (64 bytes of a partial row) and 64
// threads on each, every one with every 64th row: few dependent loads, and
// enough workgroups to cover the chip at usual widths.
__global__ __launch_bounds__(1024) void ln_dw_reduce_kernel(const float* __restrict__ part, int np,
                                                            int H, int w_f32, void* dgamma,
                                                            void* dbeta) {
    __shared__ float red[64][17];
    const int q = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int i = blockIdx.x * 16 + col;                 // 2H is a multiple of 16
    float t = 0.f;
#pragma unroll 8
    for (int p = q; p < np; p += 64) t += part[(int64_t)p * 2 * H + i];
    red[q][col] = t;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const int q4 = threadIdx.x >> 4;                     // 4 threads per column, 16 rows each
    t = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += red[q4 * 16 + w][col];
    t += __shfl_xor(t, 16);
    t += __shfl_xor(t, 32);
    if (q4) return;
    void* o = i < H ? dgamma : dbeta;
    const int c = i < H ? i : i - H;
    if (!o) return;
    if (w_f32) ((float*)o)[c] = t;
    else ((bf16_t*)o)[c] = (bf16_t)f32_to_bf16(t);
}

// The backward's: one step per lane, since every column of a row also has two
// running sums, and many rows side by side, since every workgroup writes a
// partial row of them.  16384 x 2048 on inputs in turn, from codes / bf16 / fp32:
// 43 / 44 / 70 us; one wave on a row with 4 steps, 4 rows in a workgroup
// 41 / 44 / 76, with 8 rows 51 / 54 / 165, its fp32 form spilling; these 4 waves
// with half as many rows and twice the workgroups 42 / 41 / 72.  Rows above 8192
// would spill their sums: those are added by a kernel of their own, which
// reads the rows again (2048 x 16384: 60 us; with the sums beside the row 76).
constexpr int kLnSumsH = 8192;      // wider: the sums in a kernel of their own
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

// Partial rows of the weights' gradients.
int ln_parts(int64_t T, int H) {
    if (H > kLnSumsH) {     // about 1024 workgroups of the column kernel
        const int64_t need = (T + 3) / 4, cap = 1024 / ((H + 511) / 512);
        return (int)(need < cap ? need : cap);
    }
    int n = 0;
    with_bwd_shape(H, [&](auto s) { n = (int)bwd_groups<decltype(s)>(T); });
    return n;
}

template <bool XF32>
void run_fwd(const LnFwd& a, hipStream_t s) {
    with_fwd_shape(a.H, [&](auto sh) {
        using S = decltype(sh);
        ln_fwd_kernel<XF32, S><<<fwd_groups<S>(a.T), S::kThreads, 0, s>>>(a);
    });
}
template <int kSaved>
hipError_t run_bwd(const LnBwd& a, hipStream_t s) {
    const bool sums = a.part && a.H <= kLnSumsH;
    if (a.part && !sums) {
        TraceScope ts("layernorm_cols", s);
        ln_cols_kernel<kSaved><<<dim3((unsigned)((a.H + 511) / 512), (unsigned)ln_parts(a.T, a.H)),
                                 256, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    TraceScope ts("layernorm_bwd", s);
    with_bwd_shape(a.H, [&](auto sh) {
        using S = decltype(sh);
        if (!sums)
            ln_bwd_kernel<kSaved, S, false><<<bwd_groups<S>(a.T), S::kThreads, 0, s>>>(a);
        else if constexpr (8 * S::kPer * S::kV <= kLnSumsH)
            ln_bwd_kernel<kSaved, S, true><<<bwd_groups<S>(a.T), S::kThreads, 0, s>>>(a);
    });
    return hipGetLastError();
}

}  // namespace

size_t layernorm_workspace_bytes(int64_t T, int H) {
    return (size_t)ln_parts(T, H) * 2 * (size_t)H * sizeof(float) + 256;
}

hipError_t launch_layernorm_fwd(const void* x, bool x_f32, int64_t T, int H, const void* gamma,
                                const void* beta, bool w_f32, float eps, bf16_t* y, float* mean,
                                float* rstd, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    if (T == 0) return hipSuccess;
    LnFwd a{x, gamma, beta, y, mean, rstd, codes, scales, T, H, w_f32 ? 1 : 0, eps};
    TraceScope ts("layernorm_fwd", s);
    if (x_f32) run_fwd<true>(a, s);
    else run_fwd<false>(a, s);
    return hipGetLastError();
}

hipError_t launch_layernorm_bwd(const bf16_t* dy, const void* x, bool x_f32, const float* mean,
                                const float* rstd, const uint8_t* codes, const uint8_t* scales,
                                int64_t T, int H, const void* gamma, bool w_f32, const void* dres,
                                void* dx, void* dgamma, void* dbeta, void* ws, hipStream_t s) {
    const bool want = dgamma || dbeta;
    if (T > 0) {
        LnBwd a{dy, x, mean, rstd, codes, scales, gamma, dres, dx, want ? (float*)ws : nullptr,
                T, H, w_f32 ? 1 : 0};
        const hipError_t e = codes ? (x_f32 ? run_bwd<LN_MX_F32>(a, s) : run_bwd<LN_MX_BF16>(a, s))
                                   : (x_f32 ? run_bwd<LN_F32>(a, s) : run_bwd<LN_BF16>(a, s));
        if (e != hipSuccess) return e;
    }
    if (!want) return hipSuccess;
    TraceScope ts("layernorm_dw_reduce", s);
    ln_dw_reduce_kernel<<<(unsigned)(2 * H / 16), 1024, 0, s>>>(
        (const float*)ws, ln_parts(T, H), H, w_f32 ? 1 : 0, dgamma, dbeta);
    return hipGetLastError();
}

}  // namespace moe
