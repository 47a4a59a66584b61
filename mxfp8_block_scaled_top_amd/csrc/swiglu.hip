// ScaledSwiGLU by itself, forward and backward, for gfx950: the activation
// between two grouped linear calls (grouped_mlp_* has it in its GEMMs'
// epilogues).
//
//   forward   [g, u] = a1,  a2 = p silu(g) u; optionally a1 as MXFP8 rows, the
//             8-bit checkpoint that the backward reads in place of a1
//   backward  sig = sigmoid(g), s = g sig:
//             dg = da2 p u sig (1 + g (1 - sig)),  du = da2 p s,
//             dp = sum_i da2 s u
//
// Elementwise but for dp, so bound by HBM bytes: every value is read and
// written once, 8 neighbouring columns per lane (16 bytes of bf16), past the
// caches.  The forward spreads the 8-column pieces of all rows over the grid;
// the backward gives a row to one wave, or to four when rows are long, whose
// fp32 sums give dp without atomics.
//
// Measured at 16384 x 14336, 1.89 GB a pass: forward with checkpoint 300 us
// (6.3 TB/s; a large copy reaches 5.2, a pass that reads more than it writes
// more), backward from the checkpoint 346 us (5.5 TB/s).  Two rows: 2.6 us.
#include "common.hpp"
#include "kernels.hpp"
#include "trace.hpp"

namespace moe {

namespace {

__device__ __forceinline__ void load_bf8(const bf16_t* p, float (&v)[8]) {
    const u32x4 a = __builtin_nontemporal_load((const u32x4*)p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = lo_bf16(a[k]);
        v[2 * k + 1] = hi_bf16(a[k]);
    }
}

__device__ __forceinline__ void store_bf8(bf16_t* p, const float (&v)[8]) {
    u32x4 a;
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    __builtin_nontemporal_store(a, (u32x4*)p);
}

__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __expf(-x));
}

__global__ __launch_bounds__(256) void swiglu_fwd_kernel(const bf16_t* __restrict__ a1,
                                                         const float* __restrict__ prob,
                                                         int64_t n, int cpr,
                                                         bf16_t* __restrict__ a2,
                                                         uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t I = (int64_t)cpr * 8;
    const int64_t r = i / cpr;
    const int64_t c = (i - r * cpr) * 8;
    float g[8], u[8], o[8];
    load_bf8(a1 + r * 2 * I + c, g);
    load_bf8(a1 + r * 2 * I + I + c, u);
    const float p = prob ? prob[r] : 1.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = p * (g[k] * sigmoid(g[k])) * u[k];
    store_bf8(a2 + r * I + c, o);
    if (codes) {   // 4 neighbouring lanes hold a block of 32 columns of one row
        uint8_t* q = codes + r * 2 * I + c;
        uint8_t* s = scales + (r * 2 * I + c) / 32;
        mx_store8(g, q, s);
        mx_store8(u, q + I, s + I / 32);
    }
}

template <bool kMx, int kWpr>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(
    const bf16_t* __restrict__ da2, const bf16_t* __restrict__ a1,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    const float* __restrict__ prob, int64_t rows, int cpr, bf16_t* __restrict__ da1,
    float* __restrict__ dprob) {
    __shared__ float red[4];
    constexpr int kRows = 4 / kWpr;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t I = (int64_t)cpr * 8;
    const int64_t r = (int64_t)blockIdx.x * kRows + wave / kWpr;
    const bool live = r < rows;
    float part = 0.f;
    if (live) {
        const float p = prob ? prob[r] : 1.f;
        for (int ch = (wave % kWpr) * 64 + lane; ch < cpr; ch += 64 * kWpr) {
            const int64_t c = (int64_t)ch * 8, at = r * 2 * I + c;
            float d[8], g[8], u[8], dg[8], du[8];
            load_bf8(da2 + r * I + c, d);
            if (kMx) {
                mx_load8(codes + at, scales + at / 32, g);
                mx_load8(codes + at + I, scales + (at + I) / 32, u);
            } else {
                load_bf8(a1 + at, g);
                load_bf8(a1 + at + I, u);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float sg = sigmoid(g[k]), sl = g[k] * sg, dp = d[k] * p;
                dg[k] = dp * u[k] * sg * (1.f + g[k] * (1.f - sg));
                du[k] = dp * sl;
                part += d[k] * sl * u[k];
            }
            store_bf8(da1 + at, dg);
            store_bf8(da1 + at + I, du);
        }
    }
    if (!dprob) return;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) part += __shfl_xor(part, o);
    if (kWpr == 1) {
        if (live && lane == 0) dprob[r] = part;
        return;
    }
    if (lane == 0) red[wave] = part;
    __syncthreads();
    if (threadIdx.x == 0) dprob[r] = ((red[0] + red[1]) + red[2]) + red[3];
}

// Rows of one launch: a grid of 256-thread workgroups stays below 2^31
// threads (the callers below walk the rows in such slabs).
int64_t slab_rows(int64_t rows, int64_t wg_per_row) {
    const int64_t most = ((int64_t)1 << 22) / (wg_per_row > 0 ? wg_per_row : 1);
    return rows < (most > 1 ? most : 1) ? rows : (most > 1 ? most : 1);
}

}  // namespace

hipError_t launch_swiglu_fwd(const bf16_t* a1, const float* prob, int64_t rows, int I, bf16_t* a2,
                             uint8_t* codes, uint8_t* scales, hipStream_t s) {
    const int cpr = I / 8;
    const int64_t slab = slab_rows(rows, (cpr + 255) / 256);
    for (int64_t r = 0; r < rows; r += slab) {
        const int64_t m = rows - r < slab ? rows - r : slab;
        const int64_t n = m * cpr, at = r * 2 * I;
        TraceScope ts("swiglu_fwd", s);
        swiglu_fwd_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(
            a1 + at, prob ? prob + r : nullptr, n, cpr, a2 + at / 2, codes ? codes + at : nullptr,
            scales ? scales + at / 32 : nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_swiglu_bwd(const bf16_t* da2, const bf16_t* a1, const uint8_t* codes,
                             const uint8_t* scales, const float* prob, int64_t rows, int I,
                             bf16_t* da1, float* dprob, hipStream_t s) {
    const int cpr = I / 8;
    const bool wide = cpr > 256;        // a row of one wave: at most 4 pieces per lane
    const int64_t slab = slab_rows(rows, 1);
    for (int64_t r = 0; r < rows; r += slab) {
        const int64_t m = rows - r < slab ? rows - r : slab, at = r * 2 * I;
        const unsigned grid = (unsigned)(wide ? m : (m + 3) / 4);
        const bf16_t* d = da2 + at / 2;
        const float* p = prob ? prob + r : nullptr;
        float* dp = dprob ? dprob + r : nullptr;
        TraceScope ts("swiglu_bwd", s);
#define SWIGLU_BWD(MX, W)                                                                       \
    swiglu_bwd_kernel<MX, W><<<grid, 256, 0, s>>>(d, a1 ? a1 + at : nullptr,                    \
                                                  codes ? codes + at : nullptr,                 \
                                                  scales ? scales + at / 32 : nullptr, p, m, cpr, \
                                                  da1 + at, dp)
        if (codes && wide) SWIGLU_BWD(true, 4);
        else if (codes) SWIGLU_BWD(true, 1);
        else if (wide) SWIGLU_BWD(false, 4);
        else SWIGLU_BWD(false, 1);
#undef SWIGLU_BWD
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
