// 8-bit blocks of 128: E4M3 codes with one fp32 scale per 128 consecutive
// values of a row (weights: per 128 x 128 values).
//
//   s = max(amax, 448 * 2^-126) / 448,   code = E4M3(v / s)
//
// Both quotients are the correctly rounded fp32 ones; the code is the E4M3
// value nearest to the second (ties to even).  |v| / s rounds to at most 448,
// so nothing is clamped, and the bound from below keeps s a normal number (an
// all-zero block has codes 0).  A block with an infinity or a NaN has s = inf
// or NaN, and every value of it decodes to NaN.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kBlk = 128;

__host__ __device__ inline int64_t blocks_of(int64_t n) { return (n + kBlk - 1) / kBlk; }

// bits of 448 * 2^-126
constexpr uint32_t kLeastAmax = 0x04e00000u;

// Largest magnitude's bits (as integers they order like the magnitudes, with
// infinity and NaN on top) over each row of 16 lanes, the same for all of them.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t m) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kCtrl, 0xf, 0xf, false);
    return m > o ? m : o;
}
__device__ __forceinline__ uint32_t row16_umax(uint32_t m) {
    m = dpp_umax<0xB1>(m);      // quad_perm: lane ^ 1, lane ^ 2
    m = dpp_umax<0x4E>(m);
    m = dpp_umax<0x141>(m);     // row_half_mirror, row_mirror
    return dpp_umax<0x140>(m);
}

// The scale of a block from its largest magnitude's bits.
__device__ __forceinline__ float blk_scale(uint32_t amax_bits) {
    return __uint_as_float(amax_bits > kLeastAmax ? amax_bits : kLeastAmax) / 448.f;
}

// v / s, correctly rounded, for many v of one block: a product with the
// rounded inverse, then its residual (exact in one fma) times the inverse
// added [P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990].  The residual must not underflow: blocks of
// tiny values are moved up by an exact 2^64 first.
struct BlkDiv {
    float s, inv, up;
    __device__ __forceinline__ explicit BlkDiv(float scale) {
        up = scale < 0x1p-60f ? 0x1p64f : 1.f;
        s = scale * up;
        inv = 1.f / s;
    }
    __device__ __forceinline__ float operator()(float v) const {
        v *= up;
        const float q = v * inv;
        return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, v), inv, q), v);    // -0 stays
    }
};

// Four E4M3 codes, packed little-endian.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The codes of 8 neighbouring values per lane, the 16 lanes of a row of lanes
// holding a block (zeros past the end of the data); all of them active.
__device__ __forceinline__ u32x2 blk_encode8(const float (&v)[8], float& scale) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = m > abs_bits(v[k]) ? m : abs_bits(v[k]);
    scale = blk_scale(row16_umax(m));
    const BlkDiv d(scale);
    return (u32x2){e4m3x4(d(v[0]), d(v[1]), d(v[2]), d(v[3])),
                   e4m3x4(d(v[4]), d(v[5]), d(v[6]), d(v[7]))};
}

}  // namespace moe
