// The 128-block 8-bit formats (block8.hpp) for gfx950: rows in 1 x 128 blocks,
// weights in 128 x 128 blocks (with a transposed copy on request, the operand of
// the data gradient), and rows back to bf16.
//
// All three are bound by HBM bytes: 8192 x 4096 rows 19 to 21 us (4.9 to 5.2 TB/s, a copy
// of 1 GiB 5.1), 64 matrices of 2816 x 2048 in both orders 266 us (5.5), 4099 rows of
// 14336 decoded 33 us (5.5).
#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"
#include "norm.hpp"
#include "trace.hpp"

namespace moe {

namespace {

// The chunks of a thread: every gridDim.x * 256-th of `per` a row, as row and
// place in it.  (One division a thread.  With one of 64 bits for every chunk, whole calls,
// us: 8192 x 4096 20.8 for 20.2, 300000 x 64 20.7 for 19.7, 4099 x 14336 36.6 for 35.4.)
struct Chunks {
    int64_t r, dr;
    uint32_t c, dc, per;
    __device__ __forceinline__ Chunks(uint32_t per_) : per(per_) {
        const uint32_t i = blockIdx.x * 256u + threadIdx.x, step = gridDim.x * 256u;    // below 2^22
        r = i / per;
        c = i % per;
        dr = step / per;
        dc = step % per;
    }
    __device__ __forceinline__ void next() {
        r += dr;
        c += dc;
        if (c >= per) {
            c -= per;
            ++r;
        }
    }
};

// Rows: 16 lanes have a block, 8 neighbouring values each, of the rows padded to
// whole blocks.
__global__ __launch_bounds__(256) void quant_rows128_kernel(const bf16_t* __restrict__ x, int64_t rows,
                                                            int cols, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
    const int nc = cols / 8;
    for (Chunks at((uint32_t)blocks_of(cols) * 16); at.r < rows; at.next()) {
        const int64_t r = at.r;
        const int c = (int)at.c;
        Raw8<false> w{};
        if (c < nc) w = load_raw<false>(x, r * cols + c * 8);
        float v[8], scale;
        unpack<false>(w, v);
        const u32x2 q = blk_encode8(v, scale);      // 16 chunks a block: whole blocks are active
        if (c < nc) {
            __builtin_nontemporal_store(q, (u32x2*)(codes + r * cols + c * 8));
            if ((c & 15) == 0) scales[(int64_t)(c >> 4) * rows + r] = scale;
        }
    }
}

struct QuantW {
    MatTable w, codes, scales, codes_t;
    int N, K;
    int with_t;
};

// 8 words of 8 codes (row i: columns 0..7) to 8 words of 8 codes (column j: rows 0..7).
__device__ __forceinline__ void transpose8x8(u32x2 (&m)[8]) {
    u32x2 o[8];
#pragma unroll
    for (int h = 0; h < 2; ++h)             // columns 4h..4h+3
#pragma unroll
        for (int g = 0; g < 2; ++g) {       // rows 4g..4g+3
            const uint32_t a = m[4 * g][h], b = m[4 * g + 1][h], c = m[4 * g + 2][h], d = m[4 * g + 3][h];
            // byte i of __builtin_amdgcn_perm(hi, lo, sel): 0..3 from lo, 4..7 from hi
            const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602);
            const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602);
            o[4 * h][g] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100);
            o[4 * h + 1][g] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302);
            o[4 * h + 2][g] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100);
            o[4 * h + 3][g] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302);
        }
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = o[j];
}

// One 128 x 128 block per workgroup.  Thread (rg, c) has rows 8 rg .. + 7 of
// columns 8 c .. + 7: a row's 16 threads read 256 and write 128 neighbouring
// bytes, and the transposed copy is an 8 x 8 transposition in registers and
// one pass through LDS, after which it too leaves as 128 neighbouring bytes.
__global__ __launch_bounds__(256) void quant_weights128_kernel(QuantW a) {
    __shared__ uint32_t red[4];
    __shared__ u32x2 tile[128][17];             // [column][8 rows]; 17: banks
    const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
    const int c = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int k = kb * kBlk + c * 8, n0 = nb * kBlk + rg * 8;
    const bf16_t* w = (const bf16_t*)a.w.p[e];
    Raw8<false> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        raw[i] = Raw8<false>{};
        if (k < a.K && n0 + i < a.N) raw[i] = load_raw<false>(w, (int64_t)(n0 + i) * a.K + k);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        unpack<false>(raw[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = m > abs_bits(v[j]) ? m : abs_bits(v[j]);
    }
    m = row16_umax(m);
    uint32_t o = __shfl_xor(m, 16);
    m = m > o ? m : o;
    o = __shfl_xor(m, 32);
    m = m > o ? m : o;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) m = m > red[i] ? m : red[i];
    const float scale = blk_scale(m);
    const BlkDiv d(scale);
    if (threadIdx.x == 0)
        ((float*)a.scales.p[e])[(int64_t)nb * blocks_of(a.K) + kb] = scale;
    u32x2 q[8];
    uint8_t* codes = (uint8_t*)a.codes.p[e];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        unpack<false>(raw[i], v);
        q[i] = (u32x2){e4m3x4(d(v[0]), d(v[1]), d(v[2]), d(v[3])),
                       e4m3x4(d(v[4]), d(v[5]), d(v[6]), d(v[7]))};
        if (k < a.K && n0 + i < a.N)
            __builtin_nontemporal_store(q[i], (u32x2*)(codes + (int64_t)(n0 + i) * a.K + k));
    }
    if (!a.with_t) return;
    transpose8x8(q);
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[c * 8 + j][rg] = q[j];
    __syncthreads();
    uint8_t* t = (uint8_t*)a.codes_t.p[e];
#pragma unroll
    for (int i = 0; i < 8; ++i) {               // 16 columns of the matrix at a time, 128 rows each
        const int col = i * 16 + rg, n = nb * kBlk + c * 8;
        if (kb * kBlk + col < a.K && n < a.N)   // N is a multiple of 8
            __builtin_nontemporal_store(tile[col][c], (u32x2*)(t + (int64_t)(kb * kBlk + col) * a.N + n));
    }
}

// Row r of the output is row src[r] (or r) of the codes, in bf16; zeros where
// src[r] is not a row.
__global__ __launch_bounds__(256) void dequant_rows128_kernel(const uint8_t* __restrict__ codes,
                                                              const float* __restrict__ scales,
                                                              const int32_t* __restrict__ src, int64_t x_rows,
                                                              int64_t rows, int cols, bf16_t* __restrict__ out) {
    for (Chunks at((uint32_t)cols / 8); at.r < rows; at.next()) {
        const int64_t r = at.r;
        const int c = (int)at.c;
        const int64_t from = src ? src[r] : r;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
        if (from >= 0 && from < x_rows) {
            const u32x2 w = *(const u32x2*)(codes + from * cols + c * 8);
            const float s = scales[(int64_t)(c >> 4) * x_rows + from];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
                const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
                v[4 * h] = lo[0] * s;
                v[4 * h + 1] = lo[1] * s;
                v[4 * h + 2] = hi[0] * s;
                v[4 * h + 3] = hi[1] * s;
            }
        }
        store8<false>(out, r * cols + c * 8, v);
    }
}

unsigned grid_for(int64_t items, int most) {
    const int64_t n = (items + 255) / 256;
    return (unsigned)(n < most ? n : most);
}

}  // namespace

hipError_t launch_quant_rows128(const bf16_t* x, int64_t rows, int cols, uint8_t* codes, float* scales,
                                hipStream_t s, const char* name) {
    if (rows == 0) return hipSuccess;
    TraceScope ts(name, s);
    quant_rows128_kernel<<<grid_for(rows * blocks_of(cols) * 16, 4096), 256, 0, s>>>(x, rows, cols, codes, scales);
    return hipGetLastError();
}

hipError_t launch_quant_weights128(const MatTable& w, int nmat, int N, int K, const MatTable& codes,
                                   const MatTable& scales, const MatTable* codes_t, hipStream_t s) {
    QuantW a{w, codes, scales, codes_t ? *codes_t : MatTable{}, N, K, codes_t ? 1 : 0};
    TraceScope ts("quant_weights128", s);
    quant_weights128_kernel<<<dim3((unsigned)blocks_of(K), (unsigned)blocks_of(N), (unsigned)nmat), 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_dequant_rows128(const uint8_t* codes, const float* scales, const int32_t* src, int64_t x_rows,
                                  int64_t rows, int cols, bf16_t* out, hipStream_t s, const char* name) {
    if (rows == 0) return hipSuccess;
    TraceScope ts(name, s);
    dequant_rows128_kernel<<<grid_for(rows * (cols / 8), 8192), 256, 0, s>>>(codes, scales, src, x_rows, rows, cols, out);
    return hipGetLastError();
}

}  // namespace moe
