// bf16 grouped products for few rows per expert, for gfx950: the four products
// of the expert MLP that read weights, with the epilogues of the 8-bit-A1 form.
//
//   gate_up   A1 = x W1^T, then A2 = p silu(g) u and A1's MXFP8 rows
//   down      y = A2 W2^T
//   dgrads    dA2 = dy W2 with the SwiGLU backward,  dx = dA1 W1
//   wgrads    dW2 = dy^T A2,  dW1 = dA1^T x
//
// With few rows the weights' bytes bound them: each weight should be read (or
// written) once, by as many compute units as there are.  The 256 x 256 tiles
// of the large products do neither: a tile spends its whole matrix time on a
// few rows, and a narrow weight gives few tiles (N = 2816 and 5 experts: 55).
//   * A workgroup has 64 weight columns (32 gate and 32 up ones for gate_up)
//     of one expert and up to 16 kMs of its rows; its waves split K, so a
//     narrow weight still has 64 x E workgroups at N = 4096.
//   * Weights go from memory to registers to the matrix cores, with the next
//     unit's loads in flight during this one's; nothing is shared by the waves
//     until their fp32 sums meet in LDS, where they are added in wave order.
//   * The products are 16 x 16 x 32 with the weights as first operand: a lane
//     ends up with 4 neighbouring columns of one row.
//   * K-contiguous weights (forward): a lane loads 32 neighbouring bytes of
//     one weight row, the four lanes of a row a whole 128-byte line, and both
//     operands take the K values in that order.
//   * N-contiguous weights (dgrads): a lane loads 4 neighbouring columns of 8 K
//     rows and turns the 8 x 4 block in registers (16 byte permutes).
//   * Tiles of the same weight columns go to the same XCD (round-robin
//     dispatch), so an expert with several row tiles rereads weights from L2.
//   * Weight gradients: a wave has a 64 x 64 piece of dW in registers, both
//     operands turned as in the dgrads, and writes 128-byte lines straight
//     from the accumulators: no LDS, several waves per SIMD whose reads, products and
//     writes overlap, where a 256 x 256 tile has the CU to itself.
// Measured, 8 experts of 2048 x 1408 with 4 rows each (138 MB of weights):
// forward 33 us, backward 52 us (the weights' bytes alone, at a large copy's
// rate: 27 and 53 us); 256 x 256 tiles 73 and 117 us.
#include "common.hpp"
#include "kernels.hpp"
#include "mlp.hpp"
#include "trace.hpp"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kFewN = 64;            // weight columns of a workgroup
constexpr int kPitch = kFewN + 4;    // floats per row of a wave's partial sums in LDS

struct FewTile {
    int e;
    int valid;       // rows of the tile
    int64_t row0;    // its first row
    int nt;          // column tile
};

// The workgroup's expert, rows and columns; false when it has none (the same
// for the whole workgroup).  Column tiles vary fastest, padded to a multiple
// of 8 so that a column tile stays on one XCD.
template <int kMs>
__device__ __forceinline__ bool few_tile(const GemmArgs& g, int ntiles, int* lds, FewTile& t) {
    constexpr int kM = 16 * kMs;
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const int n = clamp_group_size(lane < g.E ? g.split[lane] : 0, g.rows);
        lds[lane] = n;
        lds[64 + lane] = wave_incl_scan(n);
        lds[128 + lane] = wave_incl_scan((n + kM - 1) / kM);
    }
    __syncthreads();
    const int pad = (ntiles + 7) / 8 * 8;
    const int slot = blockIdx.x / pad;
    t.nt = blockIdx.x - slot * pad;
    int e = 0;
    while (e < g.E && lds[128 + e] <= slot) ++e;
    if (e >= g.E || t.nt >= ntiles) return false;
    const int m0 = (slot - (e ? lds[127 + e] : 0)) * kM;
    t.e = __builtin_amdgcn_readfirstlane(e);
    t.row0 = __builtin_amdgcn_readfirstlane((e ? lds[63 + e] : 0) + m0);
    t.valid = __builtin_amdgcn_readfirstlane(min(kM, lds[e] - m0));
    return true;
}

// Adds the waves' partial sums: `part` holds [wave][row][kPitch]; the 4 columns
// 4q.. of row m.
template <int kMs, int kWaves>
__device__ __forceinline__ f32x4 few_sum(const float* part, int m, int q) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        s += *(const f32x4*)(part + (w * 16 * kMs + m) * kPitch + 4 * q);
    return s;
}

__device__ __forceinline__ float sigmoid_few(float x) {
    return __builtin_amdgcn_rcpf(1.f + __expf(-x));
}

__device__ __forceinline__ u32x2 pack4(const f32x4& v) {
    return (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// MXFP8 of 4 values per lane, 8 neighbouring lanes a block of 32 (all active
// or none).
__device__ __forceinline__ void mx_store4(const f32x4& x, uint8_t* codes, uint8_t* scale, bool first) {
    float m = quad_max(fmaxf(fmaxf(__builtin_fabsf(x[0]), __builtin_fabsf(x[1])),
                             fmaxf(__builtin_fabsf(x[2]), __builtin_fabsf(x[3]))));
    m = fmaxf(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0x141, 0xf, 0xf, true)));
    const uint32_t S = mx_scale_byte(m);
    *(uint32_t*)codes = mx_encode4(x[0], x[1], x[2], x[3], S);
    if (first) *scale = (uint8_t)S;
}

// ---------------------------------------------------------------- K-contiguous weights
// gate_up (kSwiglu) and down.
template <int kMs, int kWaves, bool kSwiglu>
__global__ __launch_bounds__(64 * kWaves) void few_fwd_kernel(GemmArgs g, int ntiles) {
    __shared__ int sched[192];
    __shared__ __attribute__((aligned(16))) float part[kWaves * 16 * kMs * kPitch];
    FewTile t;
    if (!few_tile<kMs>(g, ntiles, sched, t)) return;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63, r = lane & 15, kg = lane >> 4;
    const int ms = (t.valid + 15) / 16;          // 16-row pieces that have rows
    const bf16_t* W = (const bf16_t*)g.b.p[t.e];
    const bf16_t* wp[4];
    const bf16_t* xp[kMs];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int n = kSwiglu ? (s >> 1) * g.I + t.nt * 32 + (s & 1) * 16 + r : t.nt * 64 + s * 16 + r;
        wp[s] = W + (int64_t)n * g.ldb + kg * 16;
    }
#pragma unroll
    for (int i = 0; i < kMs; ++i) {
        const int m = min(i * 16 + r, t.valid - 1);      // rows past the tile's repeat its last
        xp[i] = (const bf16_t*)g.a + (t.row0 + m) * g.lda + kg * 16;
    }
    f32x4 acc[4][kMs];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < kMs; ++i) acc[s][i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const int units = g.K / 64;                  // of 64 K values; K is a multiple of 128
    u32x4 w[4][2], x[kMs][2];
    auto load = [&](int u) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[s][h] = *(const u32x4*)(wp[s] + (int64_t)u * 64 + 8 * h);
#pragma unroll
        for (int i = 0; i < kMs; ++i)
            if (i < ms)
#pragma unroll
                for (int h = 0; h < 2; ++h) x[i][h] = *(const u32x4*)(xp[i] + (int64_t)u * 64 + 8 * h);
    };
    if (wave < units) load(wave);
    for (int u = wave; u < units; u += kWaves) {
        u32x4 cw[4][2], cx[kMs][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int s = 0; s < 4; ++s) cw[s][h] = w[s][h];
#pragma unroll
            for (int i = 0; i < kMs; ++i) cx[i][h] = x[i][h];
        }
        if (u + kWaves < units) load(u + kWaves);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kMs; ++i)
                if (i < ms)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        acc[s][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, cw[s][h]),
                            __builtin_bit_cast(bf16x8_t, cx[i][h]), acc[s][i], 0, 0, 0);
    }
    // lane: row r of piece i, columns 16 s + 4 kg ..
#pragma unroll
    for (int i = 0; i < kMs; ++i)
        if (i < ms)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                *(f32x4*)(part + (wave * 16 * kMs + i * 16 + r) * kPitch + 16 * s + 4 * kg) = acc[s][i];
    __syncthreads();
    if constexpr (kSwiglu) {
        const int q = threadIdx.x & 7;           // 8 threads per row, 4 j each
        for (int m = threadIdx.x >> 3; m < t.valid; m += 8 * kWaves) {
            const int64_t I = g.I, gr = t.row0 + m, j = t.nt * 32 + 4 * q;
            const f32x4 gt = few_sum<kMs, kWaves>(part, m, q);
            const f32x4 up = few_sum<kMs, kWaves>(part, m, 8 + q);
            const float p = g.prob[gr];
            f32x4 a2;
#pragma unroll
            for (int k = 0; k < 4; ++k) a2[k] = p * (gt[k] * sigmoid_few(gt[k])) * up[k];
            *(u32x2*)(g.act + gr * I + j) = pack4(a2);
            const int64_t at = gr * 2 * I + j;
            mx_store4(gt, g.a1_codes + at, g.a1_scales + at / 32, q == 0);
            mx_store4(up, g.a1_codes + at + I, g.a1_scales + (at + I) / 32, q == 0);
        }
    } else {
        const int q = threadIdx.x & 15;
        for (int m = threadIdx.x >> 4; m < t.valid; m += 4 * kWaves)
            *(u32x2*)((bf16_t*)g.c + (t.row0 + m) * g.ldc + t.nt * 64 + 4 * q) =
                pack4(few_sum<kMs, kWaves>(part, m, q));
    }
}

// ---------------------------------------------------------------- N-contiguous weights
// The down dgrad with the SwiGLU backward (kSwiglu) and the gate_up dgrad.
template <int kMs, int kWaves, bool kSwiglu>
__global__ __launch_bounds__(64 * kWaves) void few_dgrad_kernel(GemmArgs g, int ntiles) {
    __shared__ int sched[192];
    __shared__ __attribute__((aligned(16))) float part[kWaves * 16 * kMs * kPitch];
    FewTile t;
    if (!few_tile<kMs>(g, ntiles, sched, t)) return;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63, r = lane & 15, kg = lane >> 4;
    const int ms = (t.valid + 15) / 16;
    // lane: columns 4 r .. of the K rows 8 kg .. of a unit of 32
    const bf16_t* wp = (const bf16_t*)g.b.p[t.e] + (int64_t)kg * 8 * g.ldb + t.nt * 64 + 4 * r;
    const bf16_t* xp[kMs];
#pragma unroll
    for (int i = 0; i < kMs; ++i) {
        const int m = min(i * 16 + r, t.valid - 1);
        xp[i] = (const bf16_t*)g.a + (t.row0 + m) * g.lda + kg * 8;
    }
    f32x4 acc[4][kMs];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < kMs; ++i) acc[s][i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const int units = g.K / 32;
    u32x2 w[8];
    u32x4 x[kMs];
    auto load = [&](int u) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = *(const u32x2*)(wp + ((int64_t)u * 32 + k) * g.ldb);
#pragma unroll
        for (int i = 0; i < kMs; ++i)
            if (i < ms) x[i] = *(const u32x4*)(xp[i] + (int64_t)u * 32);
    };
    if (wave < units) load(wave);
    for (int u = wave; u < units; u += kWaves) {
        u32x4 f[4], cx[kMs];        // f[s]: column 4 r + s, its 8 K values
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                f[s][k] = __builtin_amdgcn_perm(w[2 * k + 1][s >> 1], w[2 * k][s >> 1],
                                                s & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int i = 0; i < kMs; ++i) cx[i] = x[i];
        if (u + kWaves < units) load(u + kWaves);
#pragma unroll
        for (int i = 0; i < kMs; ++i)
            if (i < ms)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    acc[s][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8_t, f[s]), __builtin_bit_cast(bf16x8_t, cx[i]),
                        acc[s][i], 0, 0, 0);
    }
    // acc[s][i][q]: row r of piece i, column 4 (4 kg + q) + s
#pragma unroll
    for (int i = 0; i < kMs; ++i)
        if (i < ms)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(f32x4*)(part + (wave * 16 * kMs + i * 16 + r) * kPitch + 16 * kg + 4 * q) =
                    (f32x4){acc[0][i][q], acc[1][i][q], acc[2][i][q], acc[3][i][q]};
    __syncthreads();
    const int q = threadIdx.x & 15;
    for (int m = threadIdx.x >> 4; m < t.valid; m += 4 * kWaves) {
        const f32x4 d = few_sum<kMs, kWaves>(part, m, q);
        const int64_t gr = t.row0 + m;
        const int64_t n = t.nt * 64 + 4 * q;
        if constexpr (kSwiglu) {
            const int64_t I = g.I, at = gr * 2 * I + n;
            const float p = g.prob[gr];
            float gt[4], up[4];
            const uint32_t cg = *(const uint32_t*)(g.a1_codes + at);
            const uint32_t cu = *(const uint32_t*)(g.a1_codes + at + I);
            const uint32_t Sg = g.a1_scales[at / 32], Su = g.a1_scales[(at + I) / 32];
            mx_decode4(cg, Sg, gt);
            mx_decode4(cu, Su, up);
            f32x4 dg, du;
            float dp = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float sg = sigmoid_few(gt[k]), sl = gt[k] * sg, dk = d[k] * p;
                dg[k] = dk * up[k] * sg * (1.f + gt[k] * (1.f - sg));
                du[k] = dk * sl;
                dp += d[k] * sl * up[k];
            }
            *(u32x2*)(g.act + at) = pack4(dg);
            *(u32x2*)(g.act + at + I) = pack4(du);
            dp = group_sum<16>(dp);              // the tile's 64 columns of the row
            if (q == 0) g.dprob_part[gr * ntiles + t.nt] = dp;
        } else {
            *(u32x2*)((bf16_t*)g.c + gr * g.ldc + n) = pack4(d);
        }
    }
}

// ---------------------------------------------------------------- weight gradients
// dW_e [128 mt, 128 nt] = A_e^T B_e over the expert's rows.
struct FewWgrad {
    const bf16_t* a;
    const bf16_t* b;
    int64_t lda, ldb;
    int mt, nt;
    MatTable dw;
};
// Both weight gradients and the sums of dprob in one launch: none of them fills
// the chip to its end, and a launch costs about 2 us.  Workgroups: E x the
// gate_up tiles, E x the down tiles, then those of dprob (a wave has a row).
struct FewGrads {
    FewWgrad gate_up, down;
    const int32_t* split;
    int E;
    int64_t rows;
    const float* part;      // [rows][ntiles]
    int ntiles;
    float* dprob;
};

__global__ __launch_bounds__(256) void few_grads_kernel(FewGrads g) {
    const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    // the experts' rows (every wave for itself)
    const int n = clamp_group_size(lane < g.E ? g.split[lane] : 0, g.rows);
    const int incl = wave_incl_scan(n);
    int b = blockIdx.x;
    const int n1 = g.E * g.gate_up.mt * g.gate_up.nt, n2 = g.E * g.down.mt * g.down.nt;
    if (b >= n1 + n2) {
        const int64_t r = (int64_t)(b - n1 - n2) * 4 + wave;
        if (r >= __builtin_amdgcn_readlane(incl, 63)) return;    // rows of no expert
        float s = 0.f;
        for (int t = lane; t < g.ntiles; t += 64) s += g.part[r * g.ntiles + t];
        s = wave_sum(s);
        if (lane == 0) g.dprob[r] = s;
        return;
    }
    const bool up = b < n1;
    if (!up) b -= n1;
    const FewWgrad& w = up ? g.gate_up : g.down;
    const int64_t lda = w.lda, ldb = w.ldb, ldc = (int64_t)w.nt * 128;
    const int per = w.mt * w.nt;                // 128 x 128 tiles of an expert
    const int e = b / per, tile = b - e * per;
    const int m0 = tile / w.nt * 128 + (wave >> 1) * 64, n0 = tile % w.nt * 128 + (wave & 1) * 64;
    const int rows = __builtin_amdgcn_readlane(n, e);
    const int64_t row0 = __builtin_amdgcn_readlane(incl, e) - rows;
    const bf16_t* A = w.a + row0 * lda + m0 + 4 * c;
    const bf16_t* B = w.b + row0 * ldb + n0 + 4 * c;
    bf16_t* dw = (bf16_t*)w.dw.p[e];
    f32x4 acc[4][4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[s][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < rows; r0 += 32) {     // lane: 4 columns of rows r0 + 8 kg ..
        u32x2 a[8], bv[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = r0 + 8 * kg + k;
            a[k] = bv[k] = (u32x2){0u, 0u};
            if (r < rows) {
                a[k] = *(const u32x2*)(A + (int64_t)r * lda);
                bv[k] = *(const u32x2*)(B + (int64_t)r * ldb);
            }
        }
        u32x4 fa[4], fb[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t sel = s & 1 ? 0x07060302u : 0x05040100u;
                fa[s][k] = __builtin_amdgcn_perm(a[2 * k + 1][s >> 1], a[2 * k][s >> 1], sel);
                fb[s][k] = __builtin_amdgcn_perm(bv[2 * k + 1][s >> 1], bv[2 * k][s >> 1], sel);
            }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                acc[s][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8_t, fa[s]), __builtin_bit_cast(bf16x8_t, fb[t]),
                    acc[s][t], 0, 0, 0);
    }
    // acc[s][t][q]: row 4 (4 kg + q) + s, column 4 c + t
    bf16_t* C = dw + (int64_t)(m0 + 16 * kg) * ldc + n0 + 4 * c;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int s = 0; s < 4; ++s)
            __builtin_nontemporal_store(
                pack4((f32x4){acc[s][0][q], acc[s][1][q], acc[s][2][q], acc[s][3][q]}),
                (u32x2*)(C + (int64_t)(4 * q + s) * ldc));
}

}  // namespace

// The rule, from times of both forms with the rows spread evenly (forward /
// backward, us, few against 256 x 256 tiles).  Up to 64 rows per expert the
// weights' bytes lead:
//   H, I, E           rows per expert
//   4096, 14336, 8    16: 513 / 1077 against 720 / 1230;  64: 684 / 1490 against 795 / 1411
//                     128 (not taken): 1253 / 2337 against 824 / 1557
//   2048, 1408, 64    16: 280 / 507 against 295 / 697;  64: 349 / 697 against 311 / 785
//                     128 (not taken): 577 / 1032 against 326 / 853
// Further up to 256 while the experts have so few 256-wide tiles that these
// leave most compute units idle (rows I <= 2^21):
//   2048, 1408, 8     64: 51 / 77 against 77 / 128;  128: 84 / 120 against 78 / 136
//                     186: 110 / 178 against 77 / 140;  256 (not taken): 140 / 202 against 78 / 152
//   1024, 4096, 2     256: 71 / 100 against 101 / 192
//   512, 1024, 8      256: 38 / 53 against 49 / 88
// Near its upper ends it gives back what it wins below.  The host does not know
// how the rows are spread.  Uneven ones cost this form more, since every 64 (16)
// rows of an expert read its weights again, from L2; Zipf loads (exponent 1.2),
// and all rows at one expert:
//   4096, 14336, 8    64: 868 / 1766 against 746 / 1367;  one: 610 / 1280 against 344 / 1084
//   2048, 1408, 64    64: 416 / 762 against 350 / 778;  one: 309 / 547 against 91 / 362
//   2048, 1408, 64    16: 317 / 516 against 293 / 695;  one: 221 / 348 against 80 / 284
//   2048, 1408, 8     64: 70 / 91 against 77 / 127;  one: 48 / 83 against 75 / 133
// Wider weights than 65536 stay with the tiles (the grids here are bounded for
// those that are not).  Both conditions hold up to some count of rows: the rule
// is its larger one (-1: none).
int64_t most_few_rows(int E, int H, int I) {
    if (H > (1 << 16) || I > (1 << 16)) return -1;
    const int64_t mean64 = 64 * (int64_t)E, mean256 = 256 * (int64_t)E;
    const int64_t narrow = I > 0 ? (1 << 21) / I : mean256;
    const int64_t few_tiled = narrow < mean256 ? narrow : mean256;
    return mean64 > few_tiled ? mean64 : few_tiled;
}

bool use_few_rows(int64_t rows, int E, int H, int I) { return rows <= most_few_rows(E, H, I); }

int few_tiles(int N) { return N / kFewN; }

hipError_t launch_few(int use, const GemmArgs& g, hipStream_t s) {
    TraceScope ts(g.name ? g.name : "gemm_few", s);
    const bool fwd = use == U_GATEUP_FWD || use == U_DOWN_FWD;
    const bool swiglu = use == U_GATEUP_FWD || use == U_DOWN_DGRAD;
    const int ntiles = use == U_GATEUP_FWD ? g.I / 32 : few_tiles(g.N);
    // up to 16 rows on average: 16-row tiles of 8 waves (an expert with more
    // rows has several); above, 64-row tiles, of 4 waves so that two fit a CU
    // (2048 x 1408, 64 experts of 32 rows: forward 277 us, with 8 waves 372)
    const bool wide = g.rows > 16 * (int64_t)g.E;
    const int64_t kM = wide ? 64 : 16;
    const int64_t slots = (g.rows + g.E * (kM - 1)) / kM;
    const unsigned grid = (unsigned)(slots * ((ntiles + 7) / 8 * 8));
#define FEW_CASE(KERNEL, SW)                                         \
    do {                                                             \
        if (wide) KERNEL<4, 4, SW><<<grid, 256, 0, s>>>(g, ntiles);  \
        else KERNEL<1, 8, SW><<<grid, 512, 0, s>>>(g, ntiles);       \
    } while (0)
    if (fwd && swiglu) FEW_CASE(few_fwd_kernel, true);
    else if (fwd) FEW_CASE(few_fwd_kernel, false);
    else if (swiglu) FEW_CASE(few_dgrad_kernel, true);
    else FEW_CASE(few_dgrad_kernel, false);
#undef FEW_CASE
    return hipGetLastError();
}

hipError_t launch_few_grads(const GemmArgs& gate_up, const GemmArgs& down, const float* part,
                            int ntiles, float* dprob, hipStream_t s) {
    auto wgrad = [](const GemmArgs& w) {
        return FewWgrad{(const bf16_t*)w.a, (const bf16_t*)w.b.p[0], w.lda, w.ldb,
                        w.M / 128, w.N / 128, w.c_tab};
    };
    const FewGrads g{wgrad(gate_up), wgrad(down), gate_up.split, gate_up.E, gate_up.rows,
                     part, ntiles, dprob};
    const int64_t grid = (int64_t)g.E * (g.gate_up.mt * g.gate_up.nt + g.down.mt * g.down.nt) +
                         (g.rows + 3) / 4;
    TraceScope ts("gemm_bf16_wgrads_dprob", s);
    few_grads_kernel<<<(unsigned)grid, 256, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace moe
