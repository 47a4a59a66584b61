// Grouped product of 8-bit operands with an fp32 scale for each block of 128,
// for gfx950:
//
//   y[r, n] = sum_kb sx[kb, r] sw[n/128, kb] sum_{k in kb} qx[r, k] qw[n, k]
//
// The sum inside a block of 128 is one v_mfma_scale_f32_16x16x128_f8f6f4 (fp32);
// its 16 x 16 result is multiplied by the block's two scales and added to the
// accumulators by ordinary fma, in fp32.  (The instruction's own scale takes the
// power of two of the weights' scale: the product of both scales may leave fp32's
// range where the value does not.)  It sums its products in groups of 8 and drops
// what lies 13 bits and more below a group's largest: 2^-12 of a block's 2-norm at
// worst in 11 million outputs, under the rounding of y to bf16.
//
// What that costs: a matrix instruction takes 32 cycles of its SIMD and its
// four fma 16 of the vector unit, which runs beside it; on registers alone
// the pair reaches 3.6 PFLOP/s where the matrix instruction alone reaches 4.5
// (32 x 32 x 64: 3.4 and 4.1).  The accumulators have to be ordinary registers
// (the vector unit does not read accumulation registers), 128 of them, so a
// wave has 64 x 128 outputs and a SIMD two waves.
//
//   * Tile 256 columns (weights) x 256 rows, 8 waves, 4 along the weights: 64 x
//     128 outputs each.  An expert's last tile is 128 or 64 rows high where that
//     is enough (64 x 16 kMT outputs a wave).
//   * The weights are the instruction's first operand, the rows the second: a
//     lane holds outputs of one row per fragment and needs one row scale for
//     them.  A fragment's weight rows are picked such that the lane's outputs
//     of two fragments are 8 neighbours: y leaves without a pass through LDS.
//   * K steps of one block: 128 bytes per operand row are whole lines.  Both
//     operands and the scales reach LDS by direct loads, kStages - 1 steps
//     ahead, issued two per fragment column (all at the step's start: +5%,
//     one per column +4%); 16-byte chunks are XOR-swizzled by row bits.
//   * Any K order inside a block will do as long as both operands agree: lane
//     group g reads chunks g and g + 4 of a row.
//   * A fragment column's fma run under the next column's products (10% less
//     time than right behind their own).
//   * One workgroup per compute unit walks over tiles; its loads run on into
//     the next tile (5 to 10% less time than a workgroup per tile).
//   * Rows past the end, columns past N and bytes past K read zeros (offsets
//     past the buffer resource).
//
// Measured: 16384 rows over 8 experts of 28672 x 4096 1.80 to 1.92 ms (2.0 to 2.1
// PFLOP/s, matrix cores 49 to 50% busy), of 4096 x 14336 0.87 ms (2.2); a library product
// with one scale per tensor reaches 2.75 at 2048 x 28672 x 4096.  Bound by power: the
// shader clock falls to 1.5 GHz behind the first call after a rest and settles at 2.0 to
// 2.1 of 2.4 some 20 calls later, and each change that saved cycles cost clock.  Timing variants of an
// earlier step (2170 us): without loads 1690, without fma 1830; of a later one (1830)
// without stores 1700: y's 0.94 GB add their time at the memory's rate.  (The clock
// depends on what ran before: figures that are compared are of one run, side by side.)
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
// chunk (weights: rows 8a + b and a constant, a, b < 4), two per 256 bytes.
__device__ __forceinline__ int xswz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int wswz(int r) { return ((r >> 2) & 6) | ((r >> 1) & 1); }

// Sum over the lanes up to each one, cut at 2^32 - 1: shifts inside the rows of
// 16 lanes, then the rows' sums passed on (no LDS).
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t dpp_add_sat(uint32_t v) {
    return __builtin_elementwise_add_sat(
        v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xf, false));
}
__device__ __forceinline__ uint32_t scan(uint32_t v) {
    v = dpp_add_sat<0x111, 0xf>(v);     // row_shr:1, 2, 4, 8
    v = dpp_add_sat<0x112, 0xf>(v);
    v = dpp_add_sat<0x114, 0xf>(v);
    v = dpp_add_sat<0x118, 0xf>(v);
    v = dpp_add_sat<0x142, 0xa>(v);     // row_bcast:15 into rows 1 and 3
    return dpp_add_sat<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
}

// Rows of expert e (lane e of a full wave) and the first of them: a negative
// size counts as 0, and sizes whose running total passes `rows` are cut at it.
__device__ __forceinline__ int expert_rows(const BlockGemm& p, int& first) {
    const int lane = threadIdx.x & 63, n = lane < p.E ? p.split[lane] : 0;
    const uint32_t up = min(scan(n > 0 ? (uint32_t)n : 0u), (uint32_t)p.rows);
    const int before = __shfl_up((int)up, 1);
    first = lane ? before : 0;
    return (int)up - first;
}

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
    return (i32x8){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}


__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A block of weights' scale as fraction and power of two, s = f 2^(e - 127): the
// power goes into the matrix instruction as its operand's scale, so that f times
// the row's scale stays in fp32's normal range where the product of both scales
// leaves it.  A block's sum is 0 or 2^-18 .. 2^24.7, so with e - 127 from -108 to
// 102 it stays a normal number too, and every step up to the fma is what it is
// without the split (the same bits).  f is in [1, 2) but for scales out of that
// range (and 0, infinity and NaN, which it is then itself).  (8 x 2048 rows of
// 28672 x 4096 1757 -> 1803 us, of 4096 x 14336 850 -> 874, three quarters of it for the scaled
// form of the instruction.  Deciding by the product of the scales, per fragment
// column: the compiler spills 240 registers, 6500 us.)
struct BlkScale {
    float f;
    int e;
    __device__ __forceinline__ explicit BlkScale(float s) {
        const int t = min(max(__builtin_amdgcn_frexp_expf(s) - 1, -108), 102);
        f = __builtin_ldexpf(s, -t);
        e = t + 127;
    }
};
// The products of a block, scaled by the weights' power of two.
__device__ __forceinline__ f32x4 block_products(i32x8 w, i32x8 x, int we) {
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, z, 0, 0, 0, we, 0, 127);
}

// One tile, the same for all threads of its workgroup.
struct BlockTile {
    int e, n0, rows;        // expert, first column, rows of the tile (0: no tile)
    int64_t row0;           // first grouped row
};

// Fragment columns of 16 rows per wave that a tile of so many rows takes.
__device__ __forceinline__ int tile_height(int rows) { return rows > 128 ? 8 : rows > 64 ? 4 : 2; }

// LDS of a workgroup: kStages of weights, rows, scales of rows (1 KB) and weights.
constexpr int stage_bytes(int kMT) { return kWB + 32 * kMT * kBlk + 2048; }
constexpr int kLdsB = 3 * stage_bytes(4);
static_assert(kLdsB >= 2 * stage_bytes(8) && kLdsB >= 3 * stage_bytes(2), "stages of every height");

// The tiles of a launch, the high ones first, so that the low ones (the last
// rows of an expert) fill in where a workgroup has had one high tile less (in
// the experts' order the most loaded workgroup had 1.3 times the mean: 8 x 2048
// rows of 4096 x 14336 1027 -> 970 us, 1024 rows 150 -> 140; but the low tiles read
// their weights again, 8 x 2048 rows of 28672 x 4096 1883 -> 1905).  Of each
// height, XCD x (workgroups go round robin over the XCDs) takes a contiguous
// eighth, in bands of at most 8 row tiles that share its L2; its workgroups
// take its tiles in turn.
struct TileList {
    int (*sched)[64];       // [h][e]: row tiles of height 8, 4, 2 up to expert e; first row, rows
    int ntn, t, step, len[3];
    __device__ __forceinline__ void init(const BlockGemm& p, int ntn_, int (*sched_)[64]) {
        ntn = ntn_;
        sched = sched_;
        if (threadIdx.x < 64) {
            const int lane = threadIdx.x;
            int first;
            const int n = expert_rows(p, first), r = n % kBM;
            sched[0][lane] = (int)scan(n / kBM + (r > 128));
            sched[1][lane] = (int)scan(r > 64 && r <= 128);
            sched[2][lane] = (int)scan(r > 0 && r <= 64);
            sched[3][lane] = first;
            sched[4][lane] = n;
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 3; ++h) len[h] = max(min(total(h) - first(h), eighth(h)), 0);
        t = (int)(blockIdx.x >> 3);
        step = (int)(gridDim.x >> 3);
    }
    __device__ __forceinline__ int total(int h) const { return uniform(sched[h][63]) * ntn; }
    __device__ __forceinline__ int eighth(int h) const { return (total(h) + 7) >> 3; }
    __device__ __forceinline__ int first(int h) const { return (int)(blockIdx.x & 7) * eighth(h); }
    __device__ __forceinline__ BlockTile next() {
        BlockTile tl{0, 0, 0, 0};
        int h = 0, u = t;
        while (h < 3 && u >= len[h]) u -= len[h++];
        if (h == 3) return tl;
        t += step;
        u += first(h);
        // (experts past the last one hold the total)
        const int e = (int)__popcll(__ballot(sched[h][threadIdx.x & 63] * ntn <= u));
        const int before = e ? uniform(sched[h][e - 1]) : 0, n = uniform(sched[4][e]);
        u -= before * ntn;
        int m = n / kBM;
        if (h == 0) {
            const int mt = uniform(sched[0][e]) - before, band = u / (8 * ntn), b0 = band * 8, bm = min(mt - b0, 8);
            u -= band * 8 * ntn;
            m = b0 + u % bm;
            u /= bm;
        }
        tl.e = e;
        tl.n0 = u * kBN;
        tl.rows = min(n - m * kBM, kBM);
        tl.row0 = uniform(sched[3][e]) + (int64_t)m * kBM;
        return tl;
    }
};

// The lane, of which the compiler does not know that it never changes: what is
// computed from it once a tile takes no registers in between.
__device__ __forceinline__ int own_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// A wave's loads of a tile: instruction j covers 8 tile rows, 8 lanes each.  What
// changes from tile to tile is uniform (the resources, whose sizes also make
// columns past N read zeros) but for the rows of x, which come from a table.
template <int kMT>
struct BlockFeed {
    static constexpr int kXB = 32 * kMT * kBlk, kXI = kMT / 2;      // row loads per wave and step
    static constexpr int kPer = 4 + kXI + 1;                        // loads per wave and step
    uint32_t ow[4], ox[kXI], os;
    uint64_t wbase, xbase, sbase;       // of the step whose loads come next (scales), of the tile
    int wrec, xrec;                     // sizes; 0: everything reads zeros
    uint32_t soff;

    static __device__ __forceinline__ int wchunk(int j, int wave, int lane) {
        return ((lane & 7) ^ wswz((wave * 4 + j) * 8 + (lane >> 3))) << 4;
    }
    static __device__ __forceinline__ int xchunk(int j, int wave, int lane) {
        return ((lane & 7) ^ xswz((wave * kXI + j) * 8 + (lane >> 3))) << 4;
    }
    // rows[]: the row of x, from the buffer's base, of each tile row (-1: none)
    __device__ __forceinline__ void set(const BlockGemm& p, const BlockTile& tl, const int* rows, int wave) {
        const int lane = own_lane();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ow[j] = (uint32_t)((wave * 4 + j) * 8 + (lane >> 3)) * (uint32_t)p.K + wchunk(j, wave, lane);
#pragma unroll
        for (int j = 0; j < kXI; ++j) {
            const int s = rows[(wave * kXI + j) * 8 + (lane >> 3)];
            ox[j] = s < 0 ? kOob : (uint32_t)s * (uint32_t)p.K + xchunk(j, wave, lane);
        }
        const int64_t first = p.src ? 0 : tl.row0;
        wbase = (uint64_t)p.w.p[tl.e] + (uint64_t)tl.n0 * p.K;
        wrec = min(p.N - tl.n0, kBN) * p.K;
        xbase = (uint64_t)(p.x + first * p.K);
        xrec = 0x7fffffff;
        soff = 0;
        // waves 0 .. 3 load the rows' scales, the others the two of the weights
        if (wave < 4) {
            const int s = rows[wave * 64 + lane];
            os = s < 0 ? kOob : (uint32_t)s * 4u;
            sbase = (uint64_t)(p.x_scale + first);
        } else {
            const int nb = tl.n0 / kBlk + (lane & 1);
            os = nb * kBlk < p.N ? (uint32_t)(nb * p.sn) * 4u : kOob;
            sbase = (uint64_t)p.w_scale.p[tl.e];
        }
    }
    __device__ __forceinline__ void stop() { wrec = xrec = 0; }
    // Before the last step's loads: chunks from byte `tail` on are past K.
    __device__ __forceinline__ void cut(int tail, int wave) {
        const int lane = own_lane();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (wchunk(j, wave, lane) >= tail) ow[j] = kOob;
#pragma unroll
        for (int j = 0; j < kXI; ++j)
            if (xchunk(j, wave, lane) >= tail) ox[j] = kOob;
    }
    // Load j of the step into the stage at `base`; the last one moves on to the next step.
    __device__ __forceinline__ void load(uint64_t scale_step, uint32_t base, int j, int wave) {
        if (j < 4 + kXI) {
            const Dma d{j < 4 ? rsrc_at(wbase, wrec) : rsrc_at(xbase, xrec), (uint32_t)uniform(soff)};
            dma16(d, j < 4 ? ow[j] : ox[j - 4], base + (j < 4 ? (wave * 4 + j) * 1024 : kWB + (wave * kXI + j - 4) * 1024));
        } else {
            const i32x4 rs = rsrc_at(sbase, xrec);
            uint32_t to = base + kWB + kXB + wave * 256;
            asm volatile("" : "+v"(to));        // (or the sum is taken in a vector register that the load cannot use)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                             uniform(to)),
                         "v"(os), "s"(rs)
                         : "memory");
            sbase += scale_step;
            soff += kBlk;
        }
    }
};

// The row of x that tile row threadIdx.x takes, from the buffer's base (-1: none).
__device__ __forceinline__ int row_of_x(const BlockGemm& p, const BlockTile& tl) {
    const int r = threadIdx.x;
    if (r >= tl.rows) return -1;
    if (!p.src) return r;
    const int s = p.src[tl.row0 + r];
    return s < p.x_rows ? s : -1;
}

// y of a tile.  A lane's outputs of a row are n = 32 h + 8 g + 4 (i & 1) + q with
// h = i >> 1: 8 neighbours of each half, and the four lanes of a row write 64
// neighbouring bytes per store.
template <int kMT>
__device__ __forceinline__ void block_store(const BlockGemm& p, const BlockTile& tl, const f32x4 (&acc)[4][kMT], int wave) {
    const int lane = own_lane(), xr = (wave >> 2) * (16 * kMT) + (lane & 15);
    const int n = tl.n0 + (wave & 3) * 64 + 8 * (lane >> 4);
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
        const int r = xr + 16 * m;
        if (r >= tl.rows) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 a = acc[2 * h][m], b = acc[2 * h + 1][m];
            if (n + 32 * h < p.N)               // N is a multiple of 32
                *(u32x4*)(p.y + (tl.row0 + r) * p.N + n + 32 * h) =
                    (u32x4){pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
        }
    }
}

// Tiles of at most 32 kMT rows, from `tl` on until the next one has another
// height or there is none; returns that one.
template <int kMT, int kStages>
__device__ __forceinline__ BlockTile block_tiles(const BlockGemm& p, TileList& list, BlockTile tl, uint8_t* lds, int* rows) {
    constexpr int kXB = BlockFeed<kMT>::kXB, kPer = BlockFeed<kMT>::kPer;
    constexpr int kStageB = stage_bytes(kMT), kAhead = kStages - 1;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = (wave & 3) * 64, wm = (wave >> 2) * (16 * kMT), l16 = lane & 15, g = lane >> 4;
    // where a lane's fragments start in a stage: chunk g of its first row of the
    // weights and of x (chunk g + 4: the same with bit 6 changed; the next
    // fragment's row has the same swizzle), and the scale of its first row
    const int wr = wn + ((l16 >> 2) << 3) + (l16 & 3), xr = wm + l16;
    const int wat = wr * kBlk + ((g ^ wswz(wr)) << 4);
    const int xat = kWB + xr * kBlk + ((g ^ xswz(xr)) << 4), sat = kWB + kXB + xr * 4;
    const int nkb = (p.K + kBlk - 1) / kBlk;
    const int tail = p.K - (nkb - 1) * kBlk;                // bytes of the last block
    const uint32_t l0 = lds_u32(lds);

    if (tid < kBM) rows[tid] = row_of_x(p, tl);
    __syncthreads();
    const uint64_t scale_step = wave < 4 ? (uint64_t)p.x_rows * 4u : (uint64_t)p.sk * 4u;
    const int cut_at = tail < kBlk ? nkb - 1 : -1;
    BlockFeed<kMT> feed;
    feed.set(p, tl, rows, wave);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
        if (s == cut_at) feed.cut(tail, wave);
        if (s == nkb) feed.stop();
#pragma unroll
        for (int j = 0; j < kPer; ++j) feed.load(scale_step, l0 + s * kStageB, j, wave);
    }
    int stage = 0, fill = kAhead;
    BlockTile next;
    pipe_barrier<(kStages - 2) * kPer>();
    for (;;) {
        next = list.next();
        // the loads go on into the next tile without a pause
        const bool chain = next.rows > 0 && tile_height(next.rows) == kMT && nkb > kAhead + 1;
        const int ahead = chain && tid < kBM ? row_of_x(p, next) : -1;
        f32x4 acc[4][kMT], dp[4];
        float sp = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dp[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < kMT; ++m) acc[i][m] = dp[i];
        }
        for (int kb = 0; kb < nkb; ++kb) {
            if (kb == 1 && tid < kBM) rows[tid] = ahead;    // read from the next step on
            int kf = kb + kAhead;                           // the step whose loads go out now
            if (kf == nkb) {
                if (chain) feed.set(p, next, rows, wave);
                else feed.stop();
            }
            if (kf >= nkb) kf -= nkb;
            if (kf == cut_at) feed.cut(tail, wave);
            const uint32_t base = uniform(l0 + fill * kStageB);
            fill = fill + 1 == kStages ? 0 : fill + 1;
            const uint8_t* st = lds + stage * kStageB;
            stage = stage + 1 == kStages ? 0 : stage + 1;
            const uint8_t *w0 = st + wat, *w1 = st + (wat ^ 64), *x0 = st + xat, *x1 = st + (xat ^ 64), *sx = st + sat;
            const BlkScale sw(*(const float*)(st + kWB + kXB + 1024 + 4 * ((wave >> 1) & 1)));
            auto wfrag = [&](int i) {
                const int at = (32 * (i >> 1) + 4 * (i & 1)) * kBlk;
                return join(*(const u32x4*)(w0 + at), *(const u32x4*)(w1 + at));
            };
            auto xfrag = [&](int m) { return join(*(const u32x4*)(x0 + 16 * m * kBlk), *(const u32x4*)(x1 + 16 * m * kBlk)); };
            i32x8 a[4], b[2];
            float sb[2];
            b[0] = xfrag(0);
            sb[0] = *(const float*)sx;
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = wfrag(i);
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                if (m + 1 < kMT) {
                    b[(m + 1) & 1] = xfrag(m + 1);
                    sb[(m + 1) & 1] = *(const float*)(sx + 64 * (m + 1));
                }
#pragma unroll
                for (int j = 0; j < kPer; ++j)      // two loads a fragment column, from the first on
                    if ((j / 2 < kMT ? j / 2 : kMT - 1) == m) feed.load(scale_step, base, j, wave);
                __builtin_amdgcn_sched_barrier(0);
                const float s = sb[m & 1] * sw.f;
                f32x4 d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[i] = block_products(a[i], b[m & 1], sw.e);
                    const int c = m > 0 ? m - 1 : kMT - 1;  // the column before, of the step before at m = 0
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[i][c][q] = __builtin_fmaf(dp[i][q], sp, acc[i][c][q]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) dp[i] = d[i];
                sp = s;
            }
            // the next step's (or the next tile's first) loads have landed, and
            // all waves are done with this one's stage
            pipe_barrier<(kStages - 2) * kPer>();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][kMT - 1][q] = __builtin_fmaf(dp[i][q], sp, acc[i][kMT - 1][q]);
        block_store<kMT>(p, tl, acc, wave);    // these leave under the next tile's first products
        if (!chain) break;
        tl = next;
    }
    // (every load has landed before the stages get another meaning)
    pipe_barrier<0>();
    return next;
}

__global__ __launch_bounds__(kThreads, 2) void gemm_block_kernel(BlockGemm p, int ntn) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLdsB];
    __shared__ int sched[5][64], rows[kBM];
    TileList list;
    list.init(p, ntn, sched);
    BlockTile tl = list.next();
    while (tl.rows) {
        const int h = tile_height(tl.rows);
        if (h == 8) tl = block_tiles<8, 2>(p, list, tl, lds, rows);
        else if (h == 4) tl = block_tiles<4, 3>(p, list, tl, lds, rows);
        else tl = block_tiles<2, 3>(p, list, tl, lds, rows);
    }
}

// ---------------------------------------------------------------- few rows
// With a handful of rows per expert the weights' bytes are all that counts: a
// workgroup has 32 columns, its eight waves every eighth block of K each, and
// the fragments come straight from memory into registers.  Few registers, and
// so eight waves per SIMD, keep the memory busy: 16 rows over 8 experts of
// 28672 x 4096 158 us with other weights in every call (5.9 TB/s), 138 where the same
// come again; beside these 138, with the next block's loads in flight during
// the current one's products (78 registers for 52) 147, with two blocks at once
// 151, with streaming loads 166 (they also keep weights that would fit out of
// the last-level cache).  The waves' sums meet in LDS and are added in order.
//
// Taken up to 8 rows per expert on average; an expert with more than 16 goes
// in passes of 16, and its workgroups read its weights again in each.  The rule
// cannot see the loads, which are on the device.  us here / in tiles, other weights
// in every call:
//                                  even       Zipf 1.2   half on one  all on one
//   64 of 2816 x 2048, 512 rows    65 / 67    75 / 79     93 / 82     109 / 33
//                      256         62 / 66    52 / 54     69 / 80      56 / 32
//                      128         62 / 65    36 / 39     63 / 69      29 / 21
//   8 of 14336 x 4096, 64          86 / 111   93 / 106   103 / 111     49 / 26
//   8 of 28672 x 4096, 64         164 / 175  176 / 174   195 / 177     94 / 38
//                      32         158 / 174  136 / 158   172 / 175     51 / 36
// so it loses where most rows meet one expert, by 76 us at most here.  At 16 rows
// per expert on average the tiles are faster for even loads too (8 of 14336 x 4096,
// 128 rows 128 / 110, 64 of 2816 x 2048, 1024 rows 102 / 78).
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
        const BlkScale ws(sw[(int64_t)kb * p.sk]);
        const float s = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, os, 0, 0)) * ws.f;
        const i32x8 b = join(x[0], x[1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 d = block_products(join(w[t][0], w[t][1]), b, ws.e);
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

__global__ __launch_bounds__(kFewThreads) void gemm_block_few_kernel(BlockGemm p) {
    __shared__ __attribute__((aligned(16))) float red[kFewWaves * 16 * kFewRow];
    __shared__ int found[3];
    // workgroups of the q-th expert that has rows
    const int q = blockIdx.y;
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int first;
        const int n = expert_rows(p, first);
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
    const int n0 = blockIdx.x * kFewN;
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
        const int experts = (int)(p.rows < p.E ? p.rows : p.E);
        gemm_block_few_kernel<<<dim3((unsigned)nt, (unsigned)experts), kFewThreads, 0, s>>>(p);
        return hipGetLastError();
    }
    const int ntn = (p.N + kBN - 1) / kBN;
    const int64_t tiles = (p.rows + (int64_t)p.E * (kBM - 1)) / kBM * ntn;     // at most
    gemm_block_kernel<<<tiles < 256 ? (unsigned)((tiles + 7) / 8 * 8) : 256u, kThreads, 0, s>>>(p, ntn);
    return hipGetLastError();
}

}  // namespace moe
