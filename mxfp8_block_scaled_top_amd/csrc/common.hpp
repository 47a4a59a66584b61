// Device helpers shared by the gfx950 kernels of libmoe_mi355x.
//
// MXFP8 encoding follows the block rule of the BioNeMo MoE recipe page
// (section on MXFP8 and the fused MLP): one scale for every 32 consecutive
// values.  Element format E4M3 (bias 7, 3 mantissa bits, largest finite 448,
// no infinities), scale format E8M0 (power of two, bias 127).  The scale of a
// block is the smallest power of two X with amax <= 448 X, so no element is
// clamped; elements round to nearest, ties to even.  All of it is integer /
// exact arithmetic: the codes do not depend on any floating-point rounding
// mode or on the order of operations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kWave = 64;
constexpr int kMxBlock = 32;

typedef uint16_t bf16_t;  // bfloat16 bit pattern

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

__device__ __forceinline__ float bf16_to_f32(uint32_t b) {
    return __uint_as_float(b << 16);
}

typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_v;

// Round to nearest even (gfx950's v_cvt_pk_bf16_f32, two values per
// instruction; denormals kept, overflow to infinity); NaN stays a quiet NaN.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){lo, hi}, bf16x2_v));
}

__device__ __forceinline__ uint32_t f32_to_bf16(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// E8M0 scale byte of a block from its max magnitude (amax >= 0, finite):
// smallest s with amax <= 448 * 2^s, i.e. 448 = 1.75 * 2^8 compared with the
// significand of amax; S = s + 127 clamped to [0, 254]; amax = 0 gives 0.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
    uint32_t b = __float_as_uint(amax);
    int eb = (int)((b >> 23) & 0xffu);
    int up = (b & 0x7fffffu) > 0x600000u ? 1 : 0;
    int s = eb - 8 + up;
    s = s < 0 ? 0 : (s > 254 ? 254 : s);
    return b == 0u ? 0u : (uint32_t)s;
}

// Exact multiply by 2^(127 - S) for the magnitudes that matter: results at or
// above 2^-126 are exact; smaller ones all encode to zero anyway.
__device__ __forceinline__ float mx_unscale(float v, uint32_t S) {
    return __builtin_ldexpf(v, 127 - (int)S);
}

// E4M3 code of v / 2^(S-127): sign bit kept, magnitude rounded to nearest
// even on the E4M3 grid.  |v| / X <= 448 is guaranteed by the scale choice.
__device__ __forceinline__ uint32_t mx_encode(float v, uint32_t S) {
    uint32_t sign = (__float_as_uint(v) >> 24) & 0x80u;
    float y = mx_unscale(__builtin_fabsf(v), S);
    uint32_t b = __float_as_uint(y);
    uint32_t mag;
    if (b < 0x3c800000u) {
        // below 2^-6: subnormal steps of 2^-9 (exact product), rint = half-even
        mag = (uint32_t)__builtin_rintf(y * 512.0f);
    } else {
        uint32_t e = (b >> 23) - 120u;       // E4M3 exponent field (bias 7)
        uint32_t m = b & 0x7fffffu;
        uint32_t keep = m >> 20;             // top 3 mantissa bits
        uint32_t rest = m & 0xfffffu;
        uint32_t up = (rest > 0x80000u) || (rest == 0x80000u && (keep & 1u));
        mag = ((e << 3) | keep) + up;        // a carry moves into the exponent
    }
    return sign | mag;
}

// Four E4M3 codes of v0..v3 / 2^(S-127), packed little-endian in a word, by
// gfx950's scaled conversion (v_cvt_scalef32_pk_fp8_f32 divides by the given
// power of two and rounds to nearest even, keeping the sign): two values per
// instruction and no separate unscale.  It gives the same bytes as mx_encode
// for every value a block's scale admits (checked exhaustively over all bf16
// inputs and scales, rounding ties and subnormal midpoints), and the same
// bytes as an exact ldexp unscale followed by v_cvt_pk_fp8_f32 for fp32
// inputs with arbitrary low mantissa bits (8.4 M value pairs on the GPU).
typedef __attribute__((ext_vector_type(2))) short s16x2_t;

__device__ __forceinline__ uint32_t mx_encode4(float v0, float v1, float v2, float v3,
                                               uint32_t S) {
    const float scale = __builtin_ldexpf(1.f, (int)S - 127);     // exact, S in [0, 254]
    const s16x2_t z = {0, 0};
    const s16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, v0, v1, scale, false);
    const s16x2_t w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v2, v3, scale, true);
    return __builtin_bit_cast(uint32_t, w);
}

// Value of an E4M3 code times 2^(S-127), exact in fp32.
__device__ __forceinline__ float mx_decode(uint32_t code, uint32_t S) {
    uint32_t e = (code >> 3) & 15u, m = code & 7u;
    float mag = e == 0u ? (float)m * 0.001953125f                // m * 2^-9
                        : __builtin_ldexpf((float)(8u + m), (int)e - 10);
    float v = __builtin_ldexpf(mag, (int)S - 127);
    return (code & 0x80u) ? -v : v;
}

// v plus the value that the DPP control brings (0 where it brings none).
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, kRows, 0xf,
                                                          false));
}

// Sum over the 64 lanes, the same for all of them: shifts inside the rows of
// 16 lanes, then the rows' sums passed on (six dependent adds and no LDS; the
// order is fixed).
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x111, 0xf>(v);     // row_shr:1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);     // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xc>(v);     // row_bcast:31 into rows 2 and 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum over each 16 (or 32) neighbouring lanes, the same for all of them.
template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
    static_assert(kLanes == 16 || kLanes == 32, "part of a wave");
    v = dpp_add<0xB1, 0xf>(v);      // quad_perm: lane ^ 1, lane ^ 2
    v = dpp_add<0x4E, 0xf>(v);
    v = dpp_add<0x141, 0xf>(v);     // row_half_mirror, row_mirror
    v = dpp_add<0x140, 0xf>(v);
    if (kLanes == 32) v += __shfl_xor(v, 16);
    return v;
}

// Largest of the four lanes 4q..4q+3 (quad permutes; no LDS).
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xf, 0xf, true)));
    return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xf, 0xf, true)));
}

// MXFP8 of 8 neighbouring values per lane: the four lanes 4q..4q+3 hold a
// block of 32 (all four active or none).  Each stores its 8 codes; the first
// stores the scale byte.
__device__ __forceinline__ void mx_store8(const float (&x)[8], uint8_t* codes, uint8_t* scale) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, __builtin_fabsf(x[k]));
    const uint32_t S = mx_scale_byte(quad_max(m));
    const u32x2 w = {mx_encode4(x[0], x[1], x[2], x[3], S), mx_encode4(x[4], x[5], x[6], x[7], S)};
    __builtin_nontemporal_store(w, (u32x2*)codes);
    if ((threadIdx.x & 3) == 0) *scale = (uint8_t)S;
}

// The values of 4 codes of one block.
__device__ __forceinline__ void mx_decode4(uint32_t w, uint32_t S, float (&x)[4]) {
    const float scale = __builtin_ldexpf(1.f, (int)S - 127);
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
    x[3] = b[1];
}

// The values of 8 neighbouring codes of one block.
__device__ __forceinline__ void mx_decode8(u32x2 w, uint32_t S, float (&x)[8]) {
    const float scale = __builtin_ldexpf(1.f, (int)S - 127);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], scale, false);
        const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], scale, true);
        x[4 * h] = a[0];
        x[4 * h + 1] = a[1];
        x[4 * h + 2] = b[0];
        x[4 * h + 3] = b[1];
    }
}

__device__ __forceinline__ void mx_load8(const uint8_t* codes, const uint8_t* scale,
                                         float (&x)[8]) {
    const u32x2 w = __builtin_nontemporal_load((const u32x2*)codes);
    mx_decode8(w, *scale, x);
}

// Row-pair layout of the 8-bit GEMM operands: rows 2p and 2p+1 of a matrix
// with K bytes per row share 128-byte lines, one line per 64 K-bytes, so that
// one K step (64 bytes) of a tile's row pair is one whole line:
//   byte (r, k) at (r >> 1) * p2_stride(K) + (k >> 6) * 128 + (r & 1) * 64 + (k & 63)
// The matrix occupies ceil(R / 2) * p2_stride(K) bytes; bytes of K-steps past
// K (when K is not a multiple of 64) are padding that no kernel reads.
__host__ __device__ inline int64_t p2_stride(int64_t K) { return ((K + 63) / 64) * 128; }
__host__ __device__ inline int64_t p2_off(int64_t r, int64_t k, int64_t ps) {
    return (r >> 1) * ps + (k >> 6) * 128 + (r & 1) * 64 + (k & 63);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

__device__ __forceinline__ int wave_incl_scan(int v) {
    int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        int t = __shfl_up(v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// A group's size as the kernels use it, from the size the caller gave (lane
// g of a full wave holds group g's): a negative size counts as 0, and sizes
// whose running total passes `rows` are cut at it.  Sizes that are >= 0 and
// sum to rows come through unchanged; any others still keep every group
// inside the rows the buffers hold.  (The running total is taken in 64 bits:
// raw sizes may sum past 2^31.)
__device__ __forceinline__ int clamp_group_size(int n, int64_t rows) {
    const int lane = threadIdx.x & 63;
    const int64_t v = n > 0 ? n : 0;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t t = __shfl_up(incl, o);
        if (lane >= o) incl += t;
    }
    const int64_t excl = incl - v;
    return (int)((incl < rows ? incl : rows) - (excl < rows ? excl : rows));
}

// Rows that the groups hold in all (every lane of a full wave gets it).
__device__ __forceinline__ int grouped_rows(const int32_t* split, int E, int64_t rows) {
    const int lane = threadIdx.x & 63;
    const int n = clamp_group_size(lane < E ? split[lane] : 0, rows);
    return __builtin_amdgcn_readlane(wave_incl_scan(n), 63);
}

__device__ __forceinline__ uint64_t lanemask_lt() {
    int lane = threadIdx.x & 63;
    return lane == 0 ? 0ull : (~0ull >> (64 - lane));
}

}  // namespace moe
