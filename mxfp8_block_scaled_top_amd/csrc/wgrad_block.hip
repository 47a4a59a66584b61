// Weight gradients of the products in 8-bit blocks, for gfx950:
//
//   dW_e[n, k] = sum_{r of expert e} dy[r, n] x[r, k]       (bf16 operands)
//
// A tile of 256 x 256 outputs has rows / 32 K steps, a dozen or two for usual
// loads, so what stands at its ends counts beside its products: 128 KB of
// writes, and the wait for its first loads.  One workgroup per compute unit
// therefore walks over tiles as over one long row of K steps: the loads of step
// s + 4 go out during step s, whichever tile they belong to, the fragments of
// step s + 1 are read during step s, and the writes of a tile leave while the
// next one's loads are already there.
//
//   * 4 waves of 128 x 128 outputs, which fill a wave's 256 accumulation
//     registers; two sets of fragments in turn.  (8 waves of 128 x 64: 96 KB of
//     LDS reads a step for 64; 1360 cycles a step where these take 1180 and the
//     matrix instructions alone 1024.)
//   * With one wave per SIMD a vector instruction right before a read that needs
//     it, or scalar work before the barrier, leaves the matrix pipe empty: the
//     addresses of the next step's reads and the resources of its loads are
//     made under the step's last products (1500 -> 1180 cycles).
//   * Both operands have their columns in memory order: rows of 512 bytes go to
//     LDS by direct loads (16-byte chunks XOR-swizzled by the row) and come
//     back through transposing reads.
//   * x is the instruction's first operand: a lane holds 4 neighbouring outputs
//     of a row per fragment; one exchange between rows of lanes makes them 8 of
//     one of two fragments, and four lanes write 64 neighbouring bytes.
//   * Experts in decreasing order of rows.  The workgroups take neighbouring
//     tiles at a time, 32 (8 x 4: their operands fit the L2) an XCD, every
//     second time in reverse; tiles that take longer than a workgroup's mean
//     share have a workgroup each (32771 Zipf rows over 64 experts of 2048 x 1408
//     366 -> 289 us).
//
// Against a workgroup per tile (gemm.hip), with the rows' decoding, us: 4099 uneven
// rows over 8 experts of 4096 x 14336 604 -> 577, 16384 rows 1660 -> 1620, of 28672 x 4096
// 2897 -> 2855 (1.35 PFLOP/s); 64 experts of 2816 x 2048, 512 rows each, 563 -> 441.
// (Side by side; at the settled clock of 60 calls in a row 4099 rows take 518, the
// 64 experts 439.)  Bound by power for long tiles and by that and the gradients'
// writes for short ones: without the writes 4099 rows take 365 of these 518, and neither
// streaming writes (672 for 577) nor waits that let them finish later (580) make up for
// any of it.
#include "common.hpp"
#include "dma.hpp"
#include "kernels.hpp"
#include "trace.hpp"

#include <type_traits>

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short i16x4;
typedef __attribute__((ext_vector_type(8))) short i16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4_t;

constexpr int kTile = 256, kThreads = 256, kStep = 32, kStages = 4;
constexpr int kRowB = kTile * 2;                // an operand's row of a tile
constexpr int kOpB = kStep * kRowB, kStageB = 2 * kOpB;
constexpr int kTileCost = 8;                    // what a tile costs besides its steps, in steps
constexpr int kPer = 8;                         // loads per wave and step
constexpr uint32_t kOob = 0x80000000u;          // offset that reads zeros, and is not written

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
    return (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)(uint32_t)v);
}

// A transposing read takes 32 bytes of rows k..k+3 and of rows 8 below in one go:
// the four rows in different quarters of 256 bytes, the two sets in different
// halves of a quarter.
__device__ __forceinline__ int swz(int k) { return ((k & 3) << 2) ^ ((k >> 2) & 2); }

struct WgradList {
    int (*sched)[64];       // experts in order: which, first row, rows
    int total, per, mt, round, pos, width, own;
    __device__ __forceinline__ bool next(int& e, int& m0, int& n0, int& rows, int64_t& row0) {
        // the first `own` workgroups have a tile each, the others the rest in turns
        const int w = width - own, at = pos - own;
        const int u = at < 0 ? (round ? total : pos) : own + round * w + (round & 1 ? w - 1 - at : at);
        ++round;
        if (pos < 0 || u >= total) return false;
        const int q = u / per, t = u - q * per, nt = per / mt;
        const int band = t / (8 * nt), bm = min(mt - band * 8, 8), v = t - band * 8 * nt;
        m0 = (band * 8 + v % bm) * kTile;
        n0 = v / bm * kTile;
        e = uniform(sched[0][q]);
        row0 = uniform(sched[1][q]);
        rows = uniform(sched[2][q]);
        return true;
    }
};

// A wave's loads: instruction j of an operand covers rows 8 wave + 2 j, + 1 of the
// step.  Rows past the expert's last read zeros by the resource's size, columns
// past the matrix by their offset.
struct WgradFeed {
    uint32_t oa[4], ob[4];
    uint64_t a, b;
    int left;
    Dma da, db;
    __device__ __forceinline__ void set(const WgradBlock& p, int m0, int n0, int rows, int64_t row0, int wave) {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));      // (nothing of it is kept from tile to tile)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = wave * 8 + j * 2 + (lane >> 5), c = (lane & 31) ^ swz(k);
            oa[j] = m0 + c * 8 < p.N ? (uint32_t)(k * p.N * 2 + c * 16) : kOob;
            ob[j] = n0 + c * 8 < p.K ? (uint32_t)(k * p.K * 2 + c * 16) : kOob;
        }
        a = uniform((uint64_t)(p.dy + row0 * p.N + m0));
        b = uniform((uint64_t)(p.x + row0 * p.K + n0));
        left = uniform(rows);
    }
    // The resources of the next loads: 32 rows, or what is left.  (Where nothing is
    // left they are not used: the next tile's come first.)
    __device__ __forceinline__ void ready(const WgradBlock& p) {
        const int rows = uniform(min(left, kStep));
        da = {rsrc_at(a, rows * p.N * 2), 0};
        db = {rsrc_at(b, rows * p.K * 2), 0};
    }
    __device__ __forceinline__ void move(const WgradBlock& p) {
        a = uniform(a + (uint64_t)(kStep * 2) * p.N);
        b = uniform(b + (uint64_t)(kStep * 2) * p.K);
        left = uniform(left - kStep);
    }
};

struct WgradFrags { bf16x8_t x[8], d[8]; };

__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void wgrad_block_kernel(WgradBlock p, int mt, int nt) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages * kStageB];
    __shared__ int sched[3][64], count, large;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int per = mt * nt, grid = (int)gridDim.x;
    if (tid < 64) {
        const int n = clamp_group_size(lane < p.E ? p.split[lane] : 0, p.rows);
        const int first = wave_incl_scan(n) - n;
        int rank = 0;
        for (int j = 0; j < p.E; ++j) {
            const int m = __shfl(n, j);
            rank += m > n || (m == n && j < lane) ? 1 : 0;
        }
        if (lane < p.E) {
            sched[0][rank] = lane;
            sched[1][rank] = first;
            sched[2][rank] = n;
        }
        const int used = (int)__popcll(__ballot(n > 0));
        // (a float sum of at most 64 counts; an expert more or less changes times alone)
        const float cost = n > 0 ? (float)((n - 1) / kStep + 1 + kTileCost) : 0.f;
        const int width = min(grid, (used * per + 7) & ~7);
        const int big = (int)__popcll(__ballot(cost * (float)width > wave_sum(cost) * (float)per));
        if (lane == 0) {
            count = used;
            large = min(big * per, width - 1);
        }
    }
    __syncthreads();
    const int used = uniform(count);

    // experts without rows: zeros
    for (int u = blockIdx.x; u < (p.E - used) * per; u += grid) {
        const int e = uniform(sched[0][used + u / per]), t = u % per;
        const int col = (t / mt) * kTile + (tid & 31) * 8, m0 = (t % mt) * kTile, end = min(p.N, m0 + kTile);
        if (col >= p.K) continue;
        bf16_t* c = (bf16_t*)p.dw.p[e] + col;
        for (int m = m0 + (tid >> 5); m < end; m += kThreads / 32)
            __builtin_nontemporal_store((u32x4){0u, 0u, 0u, 0u}, (u32x4*)(c + (int64_t)m * p.K));
    }

    WgradList list;
    list.sched = sched;
    list.total = used * per;
    list.per = per;
    list.mt = mt;
    list.round = 0;
    list.own = uniform(large);
    list.width = min(grid, (list.total + 7) & ~7);
    const int slot = (int)(blockIdx.x >> 3);
    list.pos = slot < list.width / 8 ? (int)(blockIdx.x & 7) * (list.width / 8) + slot : -1;
    WgradList ahead = list;
    int e, m0, n0, rows;
    int64_t row0;
    if (!list.next(e, m0, n0, rows, row0)) return;

    const uint32_t l0 = lds_u32(lds);
    WgradFeed feed;
    feed.left = 0;
    for (int j = 0; j < 4; ++j) feed.oa[j] = feed.ob[j] = kOob;
    feed.a = feed.b = 0;
    auto turn = [&]() {                 // to the tile of the step whose loads come next
        if (feed.left > 0) return;
        feed.left = 0;
        int fe, fm, fn, fr;
        int64_t f0;
        if (ahead.next(fe, fm, fn, fr, f0)) feed.set(p, fm, fn, fr, f0, wave);
        feed.ready(p);
    };
    const int wx = (wave & 1) * 128, wd = (wave >> 1) * 128;
    // a lane's transposing reads of a fragment: rows kb and kb + 4, which have the
    // same swizzle
    const int kb = 8 * (lane >> 4) + ((lane & 15) >> 2), q4 = 4 * (lane & 3);
    const int at0 = kb * kRowB + ((q4 & 7) << 1), sz = swz(kb);
    uint32_t lane_at[8];                // of fragment f, from the wave's first column
#pragma unroll
    for (int f = 0; f < 8; ++f) lane_at[f] = at0 + (((2 * f + (q4 >> 3)) ^ sz) << 4);
    auto frag = [&](uint32_t at) {
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)at);
        const i16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(at + 4 * kRowB));
        const i16x8 v = {lo[0], lo[1], lo[2], lo[3], up[0], up[1], up[2], up[3]};
        return __builtin_bit_cast(bf16x8_t, v);
    };
    WgradFrags F0, F1;
    int stage = 0;                      // of the loads that come next
    uint32_t to = uniform((int)l0 + wave * 4096);
    // fragment n of 16 of a stage, in the order in which a step uses them
    // (x's first, dy's, the other ones of x); where they start, from the stage on
    uint32_t ad[16];
    auto address = [&](uint32_t st, int n) {
        ad[n] = st + (n == 0 || n > 8 ? kOpB + wx * 2 + lane_at[n ? n - 8 : 0] : wd * 2 + lane_at[n ? n - 1 : 0]);
        asm volatile("" : "+v"(ad[n]));
    };
    auto read = [&](WgradFrags& f, int n) {
        if (n == 0 || n > 8) f.x[n ? n - 8 : 0] = frag(ad[n]);
        else f.d[n - 1] = frag(ad[n]);
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
        turn();
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            dma16(j < 4 ? feed.da : feed.db, j < 4 ? feed.oa[j & 3] : feed.ob[j & 3],
                  uniform((int)l0 + s * kStageB + (j >> 2) * kOpB + wave * 4096 + (j & 3) * 1024));
        feed.move(p);
        feed.ready(p);
    }
    pipe_barrier<(kStages - 1) * kPer>();
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        address(l0, n);
        read(F0, n);
        address(l0 + kStageB, n);
    }

    f32x4 acc[8][8];
    auto settle = [&]() {               // between products and other instructions on their registers
        asm volatile("s_nop 15\n\ts_nop 3" ::: "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
    // The step of fragments `f`, whose stage is free once all waves are here: reads
    // the next step's fragments and loads the step 4 ahead.
    auto step = [&](auto First, WgradFrags& f, WgradFrags& g) {
        turn();
        __builtin_amdgcn_sched_barrier(0);
        pipe_barrier<(kStages - 2) * kPer>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // (the DMA's address goes to M0 before the product, which gives it the
                // wait state that the DMA needs)
                if ((j == 2 && i < 7) || (j == 6 && i == 0)) {
                    const int n = i ? i + 1 : j == 6, at = n < 4 ? n * 1024 : kOpB + (n - 4) * 1024;
                    const Dma& d = n < 4 ? feed.da : feed.db;
                    const uint32_t vo = n < 4 ? feed.oa[n & 3] : feed.ob[n & 3];
                    if constexpr (decltype(First)::value)
                        asm volatile("s_add_u32 m0, %3, %4\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, 0\n\t"
                                     "buffer_load_dwordx4 %5, %6, %7 offen lds"
                                     : "=a"(acc[i][j]) : "v"(f.x[i]), "v"(f.d[j]), "s"(to), "i"(at), "v"(vo), "s"(d.rs), "s"(d.soff)
                                     : "memory", "scc");
                    else
                        asm volatile("s_add_u32 m0, %3, %4\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\t"
                                     "buffer_load_dwordx4 %5, %6, %7 offen lds"
                                     : "+a"(acc[i][j]) : "v"(f.x[i]), "v"(f.d[j]), "s"(to), "i"(at), "v"(vo), "s"(d.rs), "s"(d.soff)
                                     : "memory", "scc");
                } else if constexpr (decltype(First)::value) {
                    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "=a"(acc[i][j]) : "v"(f.x[i]), "v"(f.d[j]));
                } else {
                    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(f.x[i]), "v"(f.d[j]));
                }
                __builtin_amdgcn_sched_barrier(0);
                // 16 fragments over the first 28 pairs of products
                const int at = i * 4 + j / 2;
                if ((j & 1) && at < 28 && (at + 1) * 16 / 28 != at * 16 / 28) read(g, at * 16 / 28);
                if (i == 7) {       // under the last products: what the next step starts with
                    if (j == 0) {
                        stage = uniform((stage + 1) & (kStages - 1));
                        feed.move(p);
                    }
                    if (j == 1) feed.ready(p);
                    if (j == 2) to = uniform((int)l0 + stage * kStageB + wave * 4096);
                    const uint32_t st = uniform((int)(l0 + ((stage + 1) & (kStages - 1)) * kStageB));
                    address(st, 2 * j);
                    address(st, 2 * j + 1);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    using First = std::true_type;
    using Next = std::false_type;
    for (;;) {
        const int nk = (rows - 1) / kStep + 1;
        step(First{}, F0, F1);
        int k = 1;
        for (; k + 2 <= nk; k += 2) {
            step(Next{}, F1, F0);
            step(Next{}, F0, F1);
        }
        if (k < nk) step(Next{}, F1, F0);
        else F0 = F1;
        __builtin_amdgcn_sched_barrier(0);
        settle();
        // a lane has columns 4 g .. + 3 of fragment i in row l16 of j; the exchange
        // gives it 8 columns of one of two fragments
        int l = threadIdx.x & 63;
        asm volatile("" : "+v"(l));
        const int g = l >> 4;
        const auto out = __builtin_amdgcn_make_buffer_rsrc((void*)p.dw.p[e], 0, p.N * p.K * 2, 0x00020000);
        const int col = n0 + wx + 16 * (g & 1) + 8 * (g >> 1);
        const uint32_t at = (uint32_t)(m0 + wd + (l & 15)) * (uint32_t)p.K;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const f32x4 a = acc[i][j], b = acc[i + 1][j];
                const auto u0 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[0], a[1]), pack_bf16x2(b[0], b[1]), false, false);
                const auto u1 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[2], a[3]), pack_bf16x2(b[2], b[3]), false, false);
                const int c = col + 16 * i;
                const uint32_t o = c < p.K ? (at + 16u * j * (uint32_t)p.K + (uint32_t)c) * 2u : kOob;
                __builtin_amdgcn_raw_buffer_store_b128((u32x4){u0[0], u1[0], u0[1], u1[1]}, out, o, 0, 0);
            }
        if (!list.next(e, m0, n0, rows, row0)) break;
    }
    pipe_barrier<0>();      // every load has landed before the workgroup ends
}

}  // namespace

hipError_t launch_wgrad_block(const WgradBlock& p, hipStream_t s, const char* name) {
    TraceScope ts(name, s);
    const int mt = (p.N + kTile - 1) / kTile, nt = (p.K + kTile - 1) / kTile;
    const int64_t tiles = (int64_t)p.E * mt * nt;
    wgrad_block_kernel<<<tiles < 256 ? (unsigned)((tiles + 7) / 8 * 8) : 256u, kThreads, 0, s>>>(p, mt, nt);
    return hipGetLastError();
}

}  // namespace moe
