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
// is read once: kWpr waves hold it in registers, 8 neighbouring values per
// lane and step (16 bytes of bf16), and all sums over the row come from the
// registers, the variance around the mean already known, so nothing cancels.
// Sums are fp32; the only roundings to fewer bits are the stored y, dx and
// codes.
//
// A workgroup walks over rows with gamma (and beta) in registers: read per
// row they would be more bytes from L2 than the row itself.  The backward
// keeps its workgroup's dgamma and dbeta in registers over that walk and
// writes them once, as one partial row per workgroup; a second kernel adds
// the partial rows in a fixed order (no atomics: the same bits every time).
#include "common.hpp"
#include "kernels.hpp"
#include "trace.hpp"

namespace moe {

namespace {

// 8 values of a row of bf16 or fp32, as fp32
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if (F32) {
        const u32x4 a = __builtin_nontemporal_load((const u32x4*)((const float*)p + i));
        const u32x4 b = __builtin_nontemporal_load((const u32x4*)((const float*)p + i) + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = __uint_as_float(a[k]);
            v[4 + k] = __uint_as_float(b[k]);
        }
    } else {
        const u32x4 a = __builtin_nontemporal_load((const u32x4*)((const bf16_t*)p + i));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = lo_bf16(a[k]);
            v[2 * k + 1] = hi_bf16(a[k]);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
    if (F32) {
        u32x4 a, b;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(v[k]);
            b[k] = __float_as_uint(v[4 + k]);
        }
        __builtin_nontemporal_store(a, (u32x4*)((float*)p + i));
        __builtin_nontemporal_store(b, (u32x4*)((float*)p + i) + 1);
    } else {
        u32x4 a;
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
        __builtin_nontemporal_store(a, (u32x4*)((bf16_t*)p + i));
    }
}

// 8 weights (gamma or beta) of either type; `fill` where there are none
__device__ __forceinline__ void load_w8(const void* p, int f32, int64_t i, float fill,
                                        float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fill;
    if (!p) return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = f32 ? ((const float*)p)[i + k] : bf16_to_f32(((const bf16_t*)p)[i + k]);
}

// Sum of N values over the kWpr waves of a row; every lane gets it.  `red`
// holds the partial sums of the workgroup's waves; two calls in a row use
// different ones, so one barrier per call is enough.
template <int kWpr, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) v[n] += __shfl_xor(v[n], o);
    if (kWpr == 1) return;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) red[wave][n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = 0.f;
#pragma unroll
        for (int w = 0; w < kWpr; ++w) v[n] += red[w][n];
    }
}

constexpr int rows_per_wg(int wpr) { return wpr >= 4 ? 1 : 4 / wpr; }
constexpr int threads_per_wg(int wpr) { return wpr >= 4 ? 64 * wpr : 256; }

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

template <bool XF32, int kWpr, int kV>
__global__ __launch_bounds__(threads_per_wg(kWpr)) void ln_fwd_kernel(LnFwd a) {
    __shared__ float red[2][16][1];
    constexpr int kRows = rows_per_wg(kWpr);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int l = (wave % kWpr) * 64 + lane;
    const int nc = a.H / 8;
    float gm[kV][8], bt[kV][8];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int c = l + v * 64 * kWpr;
        load_w8(c < nc ? a.gamma : nullptr, a.w_f32, (int64_t)c * 8, 1.f, gm[v]);
        load_w8(c < nc ? a.beta : nullptr, a.w_f32, (int64_t)c * 8, 0.f, bt[v]);
    }
    const float inv = 1.f / (float)a.H;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.T; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t r = r0 + wave / kWpr;      // one row for all waves of a barrier
        const bool live = r < a.T;
        float x[kV][8];
        float s[1] = {0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * 64 * kWpr;
            if (live && c < nc)
                load8<XF32>(a.x, r * a.H + c * 8, x[v]);
            else
#pragma unroll
                for (int k = 0; k < 8; ++k) x[v][k] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s[0] += x[v][k];
        }
        row_sum<kWpr, 1>(s, red[0]);
        const float mean = s[0] * inv;
        float q[1] = {0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const bool in = l + v * 64 * kWpr < nc;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[v][k] = in ? x[v][k] - mean : 0.f;
                q[0] += x[v][k] * x[v][k];
            }
        }
        row_sum<kWpr, 1>(q, red[1]);
        const float rstd = 1.f / sqrtf(q[0] * inv + a.eps);
        if (!live) continue;
        if (l == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * 64 * kWpr;
            if (c >= nc) continue;
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

template <int kSaved, int kWpr, int kV>
__global__ __launch_bounds__(threads_per_wg(kWpr)) void ln_bwd_kernel(LnBwd a) {
    constexpr bool XF32 = kSaved == LN_F32 || kSaved == LN_MX_F32;
    constexpr bool kMx = kSaved >= LN_MX_BF16;
    constexpr int kRows = rows_per_wg(kWpr);
    __shared__ float red[2][16][2];
    __shared__ float comb[kRows > 1 ? kRows : 1][kRows > 1 ? 64 * kV * 8 : 1];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int l = (wave % kWpr) * 64 + lane;
    const int nc = a.H / 8;
    float gm[kV][8], dg[kV][8], db[kV][8];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int c = l + v * 64 * kWpr;
        load_w8(c < nc ? a.gamma : nullptr, a.w_f32, (int64_t)c * 8, 1.f, gm[v]);
#pragma unroll
        for (int k = 0; k < 8; ++k) dg[v][k] = db[v][k] = 0.f;
    }
    const float inv = 1.f / (float)a.H;
    int flip = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.T; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t r = r0 + wave / kWpr;
        const bool live = r < a.T;
        const float rstd = live ? a.rstd[r] : 0.f;
        const float mean = (!kMx && live) ? a.mean[r] : 0.f;
        float xh[kV][8], dy[kV][8];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * 64 * kWpr;
            if (live && c < nc) {
                load8<false>(a.dy, r * a.H + c * 8, dy[v]);
                if (kMx) {
                    mx_load8(a.codes + r * a.H + c * 8, a.scales + r * (a.H / 32) + c / 4, xh[v]);
                } else {
                    load8<XF32>(a.x, r * a.H + c * 8, xh[v]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) xh[v][k] = (xh[v][k] - mean) * rstd;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) dy[v][k] = xh[v][k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float g = dy[v][k] * gm[v][k];
                s[0] += g;
                s[1] += g * xh[v][k];
                dg[v][k] += dy[v][k] * xh[v][k];
                db[v][k] += dy[v][k];
            }
        }
        row_sum<kWpr, 2>(s, red[flip]);
        flip ^= 1;
        if (!live) continue;
        const float c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = l + v * 64 * kWpr;
            if (c >= nc) continue;
            float d[8], o[8];
            if (a.dres)
                load8<XF32>(a.dres, r * a.H + c * 8, d);
            else
#pragma unroll
                for (int k = 0; k < 8; ++k) d[k] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = rstd * (dy[v][k] * gm[v][k] - c1 - xh[v][k] * c2) + d[k];
            store8<XF32>(a.dx, r * a.H + c * 8, o);
        }
    }
    if (!a.part) return;
    float* out = a.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (kRows > 1) {   // the workgroup's rows are added in wave order
            if (which) __syncthreads();
#pragma unroll
            for (int v = 0; v < kV; ++v)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    comb[wave][(v * 64 + lane) * 8 + k] = which ? db[v][k] : dg[v][k];
            __syncthreads();
            for (int i = threadIdx.x; i < a.H; i += threads_per_wg(kWpr)) {
                float t = 0.f;
#pragma unroll
                for (int w = 0; w < kRows; ++w) t += comb[w][i];
                out[which * a.H + i] = t;
            }
        } else {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = l + v * 64 * kWpr;
                if (c >= nc) continue;
                float4* o = (float4*)(out + which * a.H + c * 8);
                const float* t = which ? db[v] : dg[v];
                o[0] = make_float4(t[0], t[1], t[2], t[3]);
                o[1] = make_float4(t[4], t[5], t[6], t[7]);
            }
        }
    }
}

// dgamma (columns [0, H)) and dbeta ([H, 2H)): the np partial rows added in a
// fixed order, 64 columns per workgroup, 16 waves over the rows.
__global__ __launch_bounds__(1024) void ln_dw_reduce_kernel(const float* __restrict__ part, int np,
                                                            int H, int w_f32, void* dgamma,
                                                            void* dbeta) {
    __shared__ float red[16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int i = blockIdx.x * 64 + lane;
    float t = 0.f;
    if (i < 2 * H)
        for (int p = wave; p < np; p += 16) t += part[(int64_t)p * 2 * H + i];
    red[wave][lane] = t;
    __syncthreads();
    if (wave != 0 || i >= 2 * H) return;
    t = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += red[w][lane];
    void* o = i < H ? dgamma : dbeta;
    const int c = i < H ? i : i - H;
    if (!o) return;
    if (w_f32) ((float*)o)[c] = t;
    else ((bf16_t*)o)[c] = (bf16_t)f32_to_bf16(t);
}

// Waves per row: as few as hold a row with at most 4 steps (32 values) per
// lane, so that a row's sums need few or no barriers.
int ln_wpr(int H) { return H <= 2048 ? 1 : H <= 8192 ? 4 : 16; }
int ln_steps(int H, int wpr) {
    const int per = 512 * wpr;
    const int v = (H + per - 1) / per;
    return v <= 1 ? 1 : v <= 2 ? 2 : 4;
}

// Workgroups of the backward: each writes a partial row of 2H floats.
int ln_bwd_groups(int64_t T, int H) {
    const int rows = rows_per_wg(ln_wpr(H));
    const int64_t need = (T + rows - 1) / rows;
    const int64_t cap = 512;
    return (int)(need < cap ? need : cap);
}

template <bool XF32, int kWpr, int kV>
void run_fwd(const LnFwd& a, hipStream_t s) {
    const int64_t need = (a.T + rows_per_wg(kWpr) - 1) / rows_per_wg(kWpr);
    const int64_t cap = kWpr == 16 ? 512 : 2048;
    ln_fwd_kernel<XF32, kWpr, kV>
        <<<(unsigned)(need < cap ? need : cap), threads_per_wg(kWpr), 0, s>>>(a);
}
template <int kSaved, int kWpr, int kV>
void run_bwd(const LnBwd& a, int groups, hipStream_t s) {
    ln_bwd_kernel<kSaved, kWpr, kV><<<(unsigned)groups, threads_per_wg(kWpr), 0, s>>>(a);
}

template <bool XF32>
void pick_fwd(const LnFwd& a, hipStream_t s) {
    const int w = ln_wpr(a.H), v = ln_steps(a.H, w);
#define LN_CASE(W, V) if (w == W && v == V) return run_fwd<XF32, W, V>(a, s);
    LN_CASE(1, 1) LN_CASE(1, 2) LN_CASE(1, 4) LN_CASE(4, 2) LN_CASE(4, 4) LN_CASE(16, 2)
    LN_CASE(16, 4)
#undef LN_CASE
}
template <int kSaved>
void pick_bwd(const LnBwd& a, int groups, hipStream_t s) {
    const int w = ln_wpr(a.H), v = ln_steps(a.H, w);
#define LN_CASE(W, V) if (w == W && v == V) return run_bwd<kSaved, W, V>(a, groups, s);
    LN_CASE(1, 1) LN_CASE(1, 2) LN_CASE(1, 4) LN_CASE(4, 2) LN_CASE(4, 4) LN_CASE(16, 2)
    LN_CASE(16, 4)
#undef LN_CASE
}

}  // namespace

size_t layernorm_workspace_bytes(int64_t T, int H) {
    return (size_t)ln_bwd_groups(T, H) * 2 * (size_t)H * sizeof(float) + 256;
}

hipError_t launch_layernorm_fwd(const void* x, bool x_f32, int64_t T, int H, const void* gamma,
                                const void* beta, bool w_f32, float eps, bf16_t* y, float* mean,
                                float* rstd, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    if (T == 0) return hipSuccess;
    LnFwd a{x, gamma, beta, y, mean, rstd, codes, scales, T, H, w_f32 ? 1 : 0, eps};
    TraceScope ts("layernorm_fwd", s);
    if (x_f32) pick_fwd<true>(a, s);
    else pick_fwd<false>(a, s);
    return hipGetLastError();
}

hipError_t launch_layernorm_bwd(const bf16_t* dy, const void* x, bool x_f32, const float* mean,
                                const float* rstd, const uint8_t* codes, const uint8_t* scales,
                                int64_t T, int H, const void* gamma, bool w_f32, const void* dres,
                                void* dx, void* dgamma, void* dbeta, void* ws, hipStream_t s) {
    const bool want = dgamma || dbeta;
    const int groups = ln_bwd_groups(T, H);
    if (T > 0) {
        LnBwd a{dy, x, mean, rstd, codes, scales, gamma, dres, dx, want ? (float*)ws : nullptr,
                T, H, w_f32 ? 1 : 0};
        TraceScope ts("layernorm_bwd", s);
        if (codes) {
            if (x_f32) pick_bwd<LN_MX_F32>(a, groups, s);
            else pick_bwd<LN_MX_BF16>(a, groups, s);
        } else {
            if (x_f32) pick_bwd<LN_F32>(a, groups, s);
            else pick_bwd<LN_BF16>(a, groups, s);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!want) return hipSuccess;
    TraceScope ts("layernorm_dw_reduce", s);
    ln_dw_reduce_kernel<<<(unsigned)((2 * H + 63) / 64), 1024, 0, s>>>(
        (const float*)ws, groups, H, w_f32 ? 1 : 0, dgamma, dbeta);
    return hipGetLastError();
}

}  // namespace moe
