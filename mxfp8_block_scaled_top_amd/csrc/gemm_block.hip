// Grouped product of 8-bit operands with an fp32 scale for each block of 128,
// for gfx950:
//
//   y[r, n] = sum_kb sx[kb, r] sw[n/128, kb] sum_{k in kb} qx[r, k] qw[n, k]
//
// The sum inside a block of 128 is one v_mfma_f32_16x16x128_f8f6f4 (fp32, no
// scales); its 16 x 16 result is multiplied by the block's two scales and
// added to the accumulators by ordinary fma, in fp32.  The weights are the
// instruction's first operand, the rows the second, so that a lane holds four
// neighbouring outputs of one row and needs one row scale for them.
#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"
#include "trace.hpp"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr int kBM = 128, kBN = 128, kThreads = 256;

__device__ __forceinline__ i32x8 frag(const uint8_t* lds, int row, int swz, int g) {
    const u32x4 a = *(const u32x4*)(lds + row * 128 + ((g ^ swz) << 4));
    const u32x4 b = *(const u32x4*)(lds + row * 128 + (((g + 4) ^ swz) << 4));
    return (i32x8){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

__global__ __launch_bounds__(kThreads) void gemm_block_kernel(BlockGemm p, int ntn) {
    __shared__ __attribute__((aligned(16))) uint8_t lw[kBN * 128], lx[kBM * 128];
    __shared__ int sched[3][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid < 64) {
        const int n = clamp_group_size(tid < p.E ? p.split[tid] : 0, p.rows);
        sched[0][tid] = wave_incl_scan((n + kBM - 1) / kBM);
        sched[1][tid] = wave_incl_scan(n) - n;
        sched[2][tid] = n;
    }
    __syncthreads();
    const int t = blockIdx.x / ntn, n0 = (blockIdx.x % ntn) * kBN;
    int e = 0;
    while (e < p.E && sched[0][e] <= t) ++e;
    if (e >= p.E) return;
    const int m0 = (t - (e ? sched[0][e - 1] : 0)) * kBM;
    const int64_t row0 = sched[1][e] + m0;
    const int rows = min(sched[2][e] - m0, kBM);
    const uint8_t* w = (const uint8_t*)p.w.p[e];
    const float* ws = (const float*)p.w_scale.p[e];
    // each thread fills chunk tid % 8 of rows tid / 8 + 32 i
    const int ch = tid & 7;
    const uint8_t *px[4], *pw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = tid / 8 + 32 * i;
        int64_t from = -1;
        if (r < rows) from = p.src ? p.src[row0 + r] : row0 + r;
        if (from >= p.x_rows) from = -1;
        px[i] = from >= 0 ? p.x + from * p.K + ch * 16 : nullptr;
        pw[i] = n0 + r < p.N ? w + (int64_t)(n0 + r) * p.K + ch * 16 : nullptr;
    }
    const int wn = (wave & 1) * 64, wm = (wave >> 1) * 64, l16 = lane & 15, g = lane >> 4;
    const float* ps[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int r = wm + m * 16 + l16;
        int64_t from = -1;
        if (r < rows) from = p.src ? p.src[row0 + r] : row0 + r;
        if (from >= p.x_rows) from = -1;
        ps[m] = from >= 0 ? p.x_scale + from : nullptr;
    }
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[i][m] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const int nkb = (int)blocks_of(p.K);
    for (int kb = 0; kb < nkb; ++kb) {
        const bool in = kb * 128 + ch * 16 < p.K;
        u32x4 vx[4], vw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            vx[i] = vw[i] = (u32x4){0, 0, 0, 0};
            if (in && px[i]) vx[i] = *(const u32x4*)(px[i] + kb * 128);
            if (in && pw[i]) vw[i] = *(const u32x4*)(pw[i] + kb * 128);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = tid / 8 + 32 * i;
            *(u32x4*)(lx + r * 128 + ((ch ^ ((r >> 1) & 7)) << 4)) = vx[i];
            *(u32x4*)(lw + r * 128 + ((ch ^ (((r >> 3) & 6) | ((r >> 1) & 1))) << 4)) = vw[i];
        }
        __syncthreads();
        const float sw = ws[(n0 / 128) * p.sn + kb * p.sk];
        i32x8 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = wn + ((l16 >> 2) << 4) + 4 * i + (l16 & 3);
            a[i] = frag(lw, r, ((r >> 3) & 6) | ((r >> 1) & 1), g);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int r = wm + m * 16 + l16;
            const i32x8 b = frag(lx, r, (r >> 1) & 7, g);
            const float s = ps[m] ? ps[m][(int64_t)kb * p.x_rows] * sw : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 z = {0.f, 0.f, 0.f, 0.f};
                const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i], b, z, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][m][q] = __builtin_fmaf(d[q], s, acc[i][m][q]);
            }
        }
    }
    // a lane's 16 outputs of a row are neighbours: n = 16 g + 4 i + q
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int r = wm + m * 16 + l16, n = n0 + wn + 16 * g;
        if (r >= rows || n >= p.N) continue;        // N is a multiple of 32
        u32x4* y = (u32x4*)(p.y + (row0 + r) * p.N + n);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            y[h] = (u32x4){pack_bf16x2(acc[2 * h][m][0], acc[2 * h][m][1]), pack_bf16x2(acc[2 * h][m][2], acc[2 * h][m][3]),
                           pack_bf16x2(acc[2 * h + 1][m][0], acc[2 * h + 1][m][1]),
                           pack_bf16x2(acc[2 * h + 1][m][2], acc[2 * h + 1][m][3])};
    }
}

}  // namespace

hipError_t launch_gemm_block(const BlockGemm& p, hipStream_t s, const char* name) {
    const int ntn = (p.N + kBN - 1) / kBN;
    const int64_t tiles = (p.rows + (int64_t)p.E * (kBM - 1)) / kBM * ntn;
    if (tiles == 0) return hipSuccess;
    TraceScope ts(name, s);
    gemm_block_kernel<<<(unsigned)tiles, kThreads, 0, s>>>(p, ntn);
    return hipGetLastError();
}

}  // namespace moe
