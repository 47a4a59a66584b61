// Grouped product of 8-bit operands with an fp32 scale for each block of 128,
// for gfx950:
//
//   y[r, n] = sum_kb sx[kb, r] sw[n/128, kb] sum_{k in kb} qx[r, k] qw[n, k]
//
// The sum inside a block of 128 is one v_mfma_f32_16x16x128_f8f6f4 (fp32, no
// scales); its 16 x 16 result is multiplied by the block's two scales and
// added to the accumulators by ordinary fma, in fp32.
//
// What that costs: a matrix instruction takes 32 cycles of its SIMD and its
// four fma 16 of the vector unit, which runs beside it; on registers alone
// the pair reaches 3.6 PFLOP/s where the matrix instruction alone reaches 4.5.
// The accumulators have to be ordinary registers (the vector unit does not
// read accumulation registers), 128 of them, so a wave has 64 x 128 outputs
// and a SIMD two waves, and the two hide each other's waits.
//
//   * Tile 256 columns (weights) x 32 kMT rows, 8 waves, 4 along the weights:
//     64 x 16 kMT outputs each.
//   * The weights are the instruction's first operand, the rows the second: a
//     lane holds outputs of one row per fragment and needs one row scale for
//     them.  A fragment's weight rows are picked (wrow) such that the lane's
//     outputs of four fragments are 16 neighbours: y leaves in 32-byte pieces
//     per lane, whole lines per row, without a pass through LDS.
//   * K steps of one block: 128 bytes per operand row are whole lines.  Both
//     operands and the scales reach LDS by direct loads, kStages - 1 steps
//     ahead; 16-byte chunks are XOR-swizzled by row bits.
//   * Any K order inside a block will do as long as both operands agree: lane
//     group g reads chunks g and g + 4 of a row.
//   * Rows past the end, columns past N and bytes past K read zeros (offsets
//     past the buffer resource).
#include "block8.hpp"
#include "common.hpp"
#include "dma.hpp"
#include "kernels.hpp"
#include "trace.hpp"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr int kBN = 256, kThreads = 512;
constexpr uint32_t kOob = 0x80000000u;      // offset that reads zeros
constexpr int kWB = kBN * kBlk;             // a stage's weights

// Bits that swizzle a row's chunks: a fragment's reads take 16 rows of one
// chunk (weights: rows 16a + 4t + b for a fixed t), two per 256 bytes.
__device__ __forceinline__ int xswz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int wswz(int r) { return ((r >> 3) & 6) | ((r >> 1) & 1); }

__device__ __forceinline__ i32x8 frag(const uint8_t* row, int swz, int g) {
    const u32x4 a = *(const u32x4*)(row + ((g ^ swz) << 4));
    const u32x4 b = *(const u32x4*)(row + (((g + 4) ^ swz) << 4));
    return (i32x8){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

template <int kMT, int kStages>
__global__ __launch_bounds__(kThreads, 2) void gemm_block_kernel(BlockGemm p, int ntn) {
    constexpr int kBM = 32 * kMT, kXB = kBM * kBlk;
    constexpr int kStageB = kWB + kXB + 2048;       // weights, rows, scales of rows (1 KB) and weights
    constexpr int kXI = kMT / 2;                    // row loads per wave and step
    constexpr int kPer = 4 + kXI + 1;               // loads per wave and step
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages * kStageB];
    __shared__ int sched[3][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (tid < 64) {
        const int n = clamp_group_size(tid < p.E ? p.split[tid] : 0, p.rows);
        sched[0][tid] = wave_incl_scan((n + kBM - 1) / kBM);
        sched[1][tid] = wave_incl_scan(n) - n;
        sched[2][tid] = n;
    }
    __syncthreads();
    // XCD x (workgroups go round robin) takes a contiguous eighth of the tiles
    // that there are
    const int total = sched[0][63] * ntn, chunk = (total + 7) >> 3;
    const int i0 = blockIdx.x >> 3;
    int t = (blockIdx.x & 7) * chunk + i0;
    if (i0 >= chunk || t >= total) return;
    int e = 0;
    while (e < p.E - 1 && sched[0][e] * ntn <= t) ++e;
    t -= (e ? sched[0][e - 1] : 0) * ntn;
    const int rows_e = __builtin_amdgcn_readfirstlane(sched[2][e]);
    const int mt = (rows_e + kBM - 1) / kBM;
    const int band = t / (8 * ntn), b0 = band * 8, bm = min(mt - b0, 8);
    const int tr = t - band * 8 * ntn;
    const int m0 = __builtin_amdgcn_readfirstlane((b0 + tr % bm) * kBM);
    const int n0 = __builtin_amdgcn_readfirstlane((tr / bm) * kBN);
    const int64_t row0 = __builtin_amdgcn_readfirstlane(sched[1][e]) + (int64_t)m0;
    e = __builtin_amdgcn_readfirstlane(e);
    const int rows = min(rows_e - m0, kBM);
    const int nkb = (p.K + kBlk - 1) / kBlk;

    // ---- loads: instruction j of a wave covers 8 tile rows, 8 lanes each
    uint32_t ow[4], ox[kXI], os;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = (wave * 4 + j) * 8 + (lane >> 3), c = (lane & 7) ^ wswz(r);
        ow[j] = n0 + r < p.N ? (uint32_t)(n0 + r) * (uint32_t)p.K + (c << 4) : kOob;
    }
    auto source = [&](int r) -> int64_t {       // row of x, from the buffer's base; -1: none
        if (r >= rows) return -1;
        if (!p.src) return r;
        const int s = p.src[row0 + r];
        return s >= 0 && s < p.x_rows ? s : -1;
    };
#pragma unroll
    for (int j = 0; j < kXI; ++j) {
        const int r = (wave * kXI + j) * 8 + (lane >> 3), c = (lane & 7) ^ xswz(r);
        const int64_t s = source(r);
        ox[j] = s >= 0 ? (uint32_t)(s * p.K) + (c << 4) : kOob;
    }
    // waves 0 .. 3 load the rows' scales, the others the two of the weights
    const bool row_scales = wave < 4;
    const int64_t xbase = p.src ? 0 : row0;
    if (row_scales) {
        const int64_t s = wave * 64 + lane < kBM ? source(wave * 64 + lane) : -1;
        os = s >= 0 ? (uint32_t)s * 4u : kOob;
    } else {
        const int nb = n0 / kBlk + (lane & 1);
        os = nb * kBlk < p.N ? (uint32_t)(nb * p.sn) * 4u : kOob;
    }
    const uint64_t wbase = (uint64_t)p.w.p[e];
    const i32x4 rw = rsrc_at(wbase, 0x7fffffff), rx = rsrc_at((uint64_t)(p.x + xbase * p.K), 0x7fffffff);
    const uint64_t sbase = row_scales ? (uint64_t)(p.x_scale + xbase) : (uint64_t)p.w_scale.p[e];
    const uint64_t sstep = row_scales ? (uint64_t)p.x_rows * 4u : (uint64_t)p.sk * 4u;
    const uint32_t l0 = lds_u32(lds);
    const int tail = p.K & (kBlk - 1);          // bytes of the last block, 0: all
    auto issue = [&](int kb, int stage) {
        const bool live = kb < nkb;
        if (tail && kb == nkb - 1) {            // chunks past K
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((((lane & 7) ^ wswz((wave * 4 + j) * 8 + (lane >> 3))) << 4) >= tail) ow[j] = kOob;
#pragma unroll
            for (int j = 0; j < kXI; ++j)
                if ((((lane & 7) ^ xswz((wave * kXI + j) * 8 + (lane >> 3))) << 4) >= tail) ox[j] = kOob;
        }
        const uint32_t base = l0 + stage * kStageB;
        Dma dw{rw, (uint32_t)(live ? kb * kBlk : 0)}, dx{rx, dw.soff};
        if (!live) dw.rs[2] = dx.rs[2] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) dma16(dw, ow[j], base + (wave * 4 + j) * 1024);
#pragma unroll
        for (int j = 0; j < kXI; ++j) dma16(dx, ox[j], base + kWB + (wave * kXI + j) * 1024);
        const i32x4 rs = rsrc_at(sbase + (live ? kb * sstep : 0), live ? 0x7fffffff : 0);
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                         base + kWB + kXB + (row_scales ? wave * 256 : 1024 + (wave - 4) * 256)),
                     "v"(os), "s"(rs)
                     : "memory");
    };

    const int wn = (wave & 3) * 64, wm = (wave >> 2) * (16 * kMT), l16 = lane & 15, g = lane >> 4;
    f32x4 acc[4][kMT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < kMT; ++m) acc[i][m] = (f32x4){0.f, 0.f, 0.f, 0.f};
    // a lane's fragment rows: their swizzles do not depend on the fragment
    const int wr = wn + ((l16 >> 2) << 4) + (l16 & 3);      // + 4 i
    const int xr = wm + l16;                                // + 16 m

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(s, s);
    int stage = 0, fill = kStages - 1;
    for (int kb = 0; kb < nkb; ++kb) {
        pipe_barrier<(kStages - 2) * kPer>();
        issue(kb + kStages - 1, fill);
        fill = fill + 1 == kStages ? 0 : fill + 1;
        const uint8_t* lw = lds + stage * kStageB;
        const uint8_t* lx = lw + kWB;
        const float* sx = (const float*)(lx + kXB);
        const float sw = sx[256 + ((wave >> 1) & 1)];
        stage = stage + 1 == kStages ? 0 : stage + 1;
        i32x8 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = frag(lw + (wr + 4 * i) * kBlk, wswz(wr + 4 * i), g);
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            const i32x8 b = frag(lx + (xr + 16 * m) * kBlk, xswz(xr + 16 * m), g);
            const float s = sx[xr + 16 * m] * sw;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 z = {0.f, 0.f, 0.f, 0.f};
                const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i], b, z, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][m][q] = __builtin_fmaf(d[q], s, acc[i][m][q]);
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");    // no load may reach LDS after the workgroup
    // a lane's 16 outputs of a row are neighbours: n = 16 g + 4 i + q
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
        const int r = xr + 16 * m, n = n0 + wn + 16 * g;
        if (r >= rows || n >= p.N) continue;        // N is a multiple of 32
        u32x4* y = (u32x4*)(p.y + (row0 + r) * p.N + n);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            y[h] = (u32x4){pack_bf16x2(acc[2 * h][m][0], acc[2 * h][m][1]), pack_bf16x2(acc[2 * h][m][2], acc[2 * h][m][3]),
                           pack_bf16x2(acc[2 * h + 1][m][0], acc[2 * h + 1][m][1]),
                           pack_bf16x2(acc[2 * h + 1][m][2], acc[2 * h + 1][m][3])};
    }
}

template <int kMT, int kStages>
void run(const BlockGemm& p, hipStream_t s) {
    constexpr int kBM = 32 * kMT;
    const int ntn = (p.N + kBN - 1) / kBN;
    const int64_t tiles = (p.rows + (int64_t)p.E * (kBM - 1)) / kBM * ntn;
    gemm_block_kernel<kMT, kStages><<<(unsigned)((tiles + 7) / 8 * 8), kThreads, 0, s>>>(p, ntn);
}

}  // namespace

hipError_t launch_gemm_block(const BlockGemm& p, hipStream_t s, const char* name) {
    if (p.rows == 0) return hipSuccess;
    TraceScope ts(name, s);
    const int64_t mean = p.rows / p.E;
#ifdef PROBE_MT
    const int v = getenv("MT") ? atoi(getenv("MT")) : 0;
    if (v == 8) run<8, 2>(p, s); else if (v == 4) run<4, 3>(p, s); else if (v == 2) run<2, 3>(p, s); else
#endif
    if (mean > 128) run<8, 2>(p, s);
    else if (mean > 32) run<4, 3>(p, s);
    else run<2, 3>(p, s);
    return hipGetLastError();
}

}  // namespace moe
