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
//   * Tile 256 columns (weights) x 256 rows, 8 waves, 4 along the weights: 64 x
//     128 outputs each.  An expert's last tile is 128 or 64 rows high where that
//     is enough (64 x 16 kMT outputs a wave).
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

constexpr int kBM = 256, kBN = 256, kThreads = 512;
constexpr uint32_t kOob = 0x80000000u;      // offset that reads zeros
constexpr int kWB = kBN * kBlk;             // a stage's weights

// Bits that swizzle a row's chunks: a fragment's reads take 16 rows of one
// chunk (weights: rows 16a + 4t + b for a fixed t), two per 256 bytes.
__device__ __forceinline__ int xswz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int wswz(int r) { return ((r >> 3) & 6) | ((r >> 1) & 1); }

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
    return (i32x8){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

__device__ __forceinline__ i32x8 frag(const uint8_t* row, int swz, int g) {
    return join(*(const u32x4*)(row + ((g ^ swz) << 4)), *(const u32x4*)(row + (((g + 4) ^ swz) << 4)));
}

// What a workgroup works on, the same for all its threads.
struct BlockTile {
    int e, n0, rows;        // expert, first column, rows of the tile
    int64_t row0;           // first grouped row
};

// LDS of a workgroup: kStages of weights, rows, scales of rows (1 KB) and weights.
constexpr int stage_bytes(int kMT) { return kWB + 32 * kMT * kBlk + 2048; }
constexpr int kLdsB = 3 * stage_bytes(4);
static_assert(kLdsB >= 2 * stage_bytes(8) && kLdsB >= 3 * stage_bytes(2), "stages of every height");

// One tile of at most 32 kMT rows.
template <int kMT, int kStages>
__device__ __forceinline__ void block_tile(const BlockGemm& p, const BlockTile& tl, uint8_t* lds) {
    constexpr int kBM = 32 * kMT, kXB = kBM * kBlk;
    constexpr int kStageB = stage_bytes(kMT);
    constexpr int kXI = kMT / 2;                    // row loads per wave and step
    constexpr int kPer = 4 + kXI + 1;               // loads per wave and step
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = tl.n0, rows = tl.rows;
    const int64_t row0 = tl.row0;
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
    const uint64_t wbase = (uint64_t)p.w.p[tl.e];
    const i32x4 rw = rsrc_at(wbase, 0x7fffffff), rx = rsrc_at((uint64_t)(p.x + xbase * p.K), 0x7fffffff);
    const uint64_t sbase = row_scales ? (uint64_t)(p.x_scale + xbase) : (uint64_t)p.w_scale.p[tl.e];
    const uint64_t sstep = row_scales ? (uint64_t)p.x_rows * 4u : (uint64_t)p.sk * 4u;
    const uint32_t l0 = lds_u32(lds);
    const int tail = p.K & (kBlk - 1);          // bytes of the last block, 0: all
    auto prep = [&](int kb) {                   // before the loads of step kb
        if (tail && kb == nkb - 1) {            // chunks past K
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((((lane & 7) ^ wswz((wave * 4 + j) * 8 + (lane >> 3))) << 4) >= tail) ow[j] = kOob;
#pragma unroll
            for (int j = 0; j < kXI; ++j)
                if ((((lane & 7) ^ xswz((wave * kXI + j) * 8 + (lane >> 3))) << 4) >= tail) ox[j] = kOob;
        }
    };
    auto part = [&](int kb, int stage, int j) { // load j of step kb
        const bool live = kb < nkb;
        const uint32_t base = l0 + stage * kStageB;
        Dma dw{rw, (uint32_t)(live ? kb * kBlk : 0)}, dx{rx, dw.soff};
        if (!live) dw.rs[2] = dx.rs[2] = 0;
        if (j < 4) dma16(dw, ow[j], base + (wave * 4 + j) * 1024);
        else if (j < 4 + kXI) dma16(dx, ox[j - 4], base + kWB + (wave * kXI + j - 4) * 1024);
        else {
            const i32x4 rs = rsrc_at(sbase + (live ? kb * sstep : 0), live ? 0x7fffffff : 0);
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                             base + kWB + kXB + (row_scales ? wave * 256 : 1024 + (wave - 4) * 256)),
                         "v"(os), "s"(rs)
                         : "memory");
        }
    };
    auto issue = [&](int kb, int stage) {
        prep(kb);
#pragma unroll
        for (int j = 0; j < kPer; ++j) part(kb, stage, j);
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
    f32x4 dp[4];
    float sp = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) dp[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int kb = 0; kb < nkb; ++kb) {
        pipe_barrier<(kStages - 2) * kPer>();
        prep(kb + kStages - 1);
        const int fl = fill;
        fill = fill + 1 == kStages ? 0 : fill + 1;
        const uint8_t* lw = lds + stage * kStageB;
        const uint8_t* lx = lw + kWB;
        const float* sx = (const float*)(lx + kXB);
        const float sw = sx[256 + ((wave >> 1) & 1)];
        stage = stage + 1 == kStages ? 0 : stage + 1;
        i32x8 a[4], b[2];
        float sb[2];
        b[0] = frag(lx + xr * kBlk, xswz(xr), g);
        sb[0] = sx[xr];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = frag(lw + (wr + 4 * i) * kBlk, wswz(wr + 4 * i), g);
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            if (m + 1 < kMT) {
                b[(m + 1) & 1] = frag(lx + (xr + 16 * (m + 1)) * kBlk, xswz(xr + 16 * (m + 1)), g);
                sb[(m + 1) & 1] = sx[xr + 16 * (m + 1)];
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j)      // two loads a fragment column, from the first on
                if ((j / 2 < kMT ? j / 2 : kMT - 1) == m) part(kb + kStages - 1, fl, j);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
            const float s = sb[m & 1] * sw;
            f32x4 d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 z = {0.f, 0.f, 0.f, 0.f};
                d[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i], b[m & 1], z, 0, 0, 0, 0, 0, 0);
                constexpr int kLast = kMT - 1;
                const int c = m > 0 ? m - 1 : kLast;
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][c][q] = __builtin_fmaf(dp[i][q], sp, acc[i][c][q]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) dp[i] = d[i];
            sp = s;
            __builtin_amdgcn_s_setprio(0);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][kMT - 1][q] = __builtin_fmaf(dp[i][q], sp, acc[i][kMT - 1][q]);
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

__global__ __launch_bounds__(kThreads, 2) void gemm_block_kernel(BlockGemm p, int ntn) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLdsB];
    __shared__ int sched[3][64];
    const int tid = threadIdx.x;
    if (tid < 64) {
        const int n = clamp_group_size(tid < p.E ? p.split[tid] : 0, p.rows);
        sched[0][tid] = wave_incl_scan((n + kBM - 1) / kBM);
        sched[1][tid] = wave_incl_scan(n) - n;
        sched[2][tid] = n;
    }
    __syncthreads();
    // XCD x (workgroups go round robin) takes a contiguous eighth of the tiles
    // that there are, in bands of at most 8 row tiles that share its L2
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
    BlockTile tl;
    tl.e = __builtin_amdgcn_readfirstlane(e);
    tl.n0 = __builtin_amdgcn_readfirstlane((tr / bm) * kBN);
    tl.rows = min(rows_e - m0, kBM);
    tl.row0 = __builtin_amdgcn_readfirstlane(sched[1][e]) + (int64_t)m0;
    if (tl.rows > 128) block_tile<8, 2>(p, tl, lds);
    else if (tl.rows > 64) block_tile<4, 3>(p, tl, lds);
    else block_tile<2, 3>(p, tl, lds);
}

// ---------------------------------------------------------------- few rows
// With a handful of rows per expert the weights' bytes are all that counts: a
// workgroup has 32 columns, its eight waves every eighth block of K each, and
// the fragments come straight from memory into registers.  Few registers, and
// so eight waves per SIMD, keep the memory busy: 16 rows over 8 experts of
// 28672 x 4096 138 us (6.8 TB/s); with the next block's loads in flight during
// the current one's products (78 registers for 52) 147, with two blocks at once
// 151, with streaming loads 166 (they also keep weights that would fit out of
// the last-level cache).  The waves' sums meet in LDS and are added in order.
//
// Taken up to 8 rows per expert on average; an expert with more than 16 goes
// in passes of 16.  us here / in tiles: 8 experts of 14336 x 4096, 64 rows
// 88 / 105, 128 rows 128 / 110; 64 experts of 2816 x 2048, 256 rows 63 / 74, 512 rows
// 70 / 77 (Zipf loads, where the tiles would win: 84 / 71), 1024 rows 102 / 78.
constexpr int kFewMean = 8;
constexpr int kFewN = 32, kFewWaves = 8, kFewThreads = 64 * kFewWaves, kFewRow = kFewN + 4;

// At most 16 rows of one expert.
__device__ __forceinline__ void few_rows(const BlockGemm& p, int e, int n0, int64_t row0, int rows, float* red) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int l16 = lane & 15, g = lane >> 4;
    const int nkb = (p.K + kBlk - 1) / kBlk;
    const int64_t xbase = p.src ? 0 : row0;
    const auto rw = __builtin_amdgcn_make_buffer_rsrc((void*)p.w.p[e], 0, 0x7fffffff, 0x00020000);
    const auto rx = __builtin_amdgcn_make_buffer_rsrc((void*)(p.x + xbase * p.K), 0, 0x7fffffff, 0x00020000);
    const float* sw = (const float*)p.w_scale.p[e] + (int64_t)(n0 / kBlk) * p.sn;
    uint32_t ow[2], ox = kOob, os = kOob;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int n = n0 + 16 * t + l16;
        ow[t] = n < p.N ? (uint32_t)n * (uint32_t)p.K + (g << 4) : kOob;
    }
    if (l16 < rows) {
        const int64_t s = p.src ? p.src[row0 + l16] : l16;
        if (!p.src || (s >= 0 && s < p.x_rows)) {
            ox = (uint32_t)(s * p.K) + (g << 4);
            os = (uint32_t)s * 4u;
        }
    }
    f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int kb = wave; kb < nkb; kb += kFewWaves) {
        const int left = p.K - kb * kBlk - (g << 4);            // bytes from the lane's first chunk on
        u32x4 w[2][2], x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t past = left > 64 * h ? 0u : kOob;
#pragma unroll
            for (int t = 0; t < 2; ++t) w[t][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, ow[t] | past, kb * kBlk + 64 * h, 0);
            x[h] = __builtin_amdgcn_raw_buffer_load_b128(rx, ox | past, kb * kBlk + 64 * h, 0);
        }
        const auto rs = __builtin_amdgcn_make_buffer_rsrc((void*)(p.x_scale + xbase + (int64_t)kb * p.x_rows), 0,
                                                          0x7fffffff, 0x00020000);
        const float s = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, os, 0, 0)) * sw[(int64_t)kb * p.sk];
        const i32x8 b = join(x[0], x[1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 z = {0.f, 0.f, 0.f, 0.f};
            const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w[t][0], w[t][1]), b, z, 0, 0, 0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[t][q] = __builtin_fmaf(d[q], s, acc[t][q]);
        }
    }
    // red[wave][row][32 columns]: a lane has columns 16 t + 4 g + q of row l16
#pragma unroll
    for (int t = 0; t < 2; ++t) *(f32x4*)(red + (wave * 16 + l16) * kFewRow + 16 * t + 4 * g) = acc[t];
    __syncthreads();
    if (threadIdx.x < 16 * (kFewN / 4)) {      // 4 columns each
        const int r = threadIdx.x / (kFewN / 4), n = threadIdx.x % (kFewN / 4) * 4;
        f32x4 v = *(const f32x4*)(red + r * kFewRow + n);
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += *(const f32x4*)(red + (w * 16 + r) * kFewRow + n);
        if (r < rows && n0 + n < p.N)
            *(u32x2*)(p.y + (row0 + r) * p.N + n0 + n) = (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
    __syncthreads();
}

__global__ __launch_bounds__(kFewThreads) void gemm_block_few_kernel(BlockGemm p, int ntn) {
    __shared__ __attribute__((aligned(16))) float red[kFewWaves * 16 * kFewRow];
    __shared__ int found[3];
    // workgroups of the q-th expert that has rows
    const int q = blockIdx.x / ntn;
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const int n = clamp_group_size(lane < p.E ? p.split[lane] : 0, p.rows);
        const int first = wave_incl_scan(n) - n;
        const uint64_t has = __ballot(n > 0);
        if (lane == 0) found[0] = -1;
        if (n > 0 && __popcll(has & lanemask_lt()) == q) {
            found[0] = lane;
            found[1] = first;
            found[2] = n;
        }
    }
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(found[0]);
    if (e < 0) return;
    int64_t row0 = __builtin_amdgcn_readfirstlane(found[1]);
    int rows = __builtin_amdgcn_readfirstlane(found[2]);
    const int n0 = (blockIdx.x % ntn) * kFewN;
    while (rows > 0) {
        const int n = min(rows, 16);
        few_rows(p, e, n0, row0, n, red);
        row0 += n;
        rows -= n;
    }
}

}  // namespace

hipError_t launch_gemm_block(const BlockGemm& p, hipStream_t s, const char* name) {
    if (p.rows == 0) return hipSuccess;
    TraceScope ts(name, s);
    if (p.rows <= kFewMean * p.E) {
        const int nt = (p.N + kFewN - 1) / kFewN;
        const int64_t experts = p.rows < p.E ? p.rows : p.E;
        gemm_block_few_kernel<<<(unsigned)(experts * nt), kFewThreads, 0, s>>>(p, nt);
        return hipGetLastError();
    }
    const int ntn = (p.N + kBN - 1) / kBN;
    const int64_t tiles = (p.rows + (int64_t)p.E * (kBM - 1)) / kBM * ntn;     // at most
    gemm_block_kernel<<<(unsigned)((tiles + 7) / 8 * 8), kThreads, 0, s>>>(p, ntn);
    return hipGetLastError();
}

}  // namespace moe
