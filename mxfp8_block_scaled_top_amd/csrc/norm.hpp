// Rows of a norm (layer norm, RMS norm) over the lanes of a workgroup: loads and
// stores of 8 values per lane, sums over a row, the kernels' shapes by width.
#pragma once

#include "common.hpp"

namespace moe {

// 8 neighbouring values of a row of bf16 or fp32, as loaded
template <bool F32>
struct Raw8 {
    u32x4 w[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw(const void* p, int64_t i) {
    Raw8<F32> r;
    const u32x4* q = (const u32x4*)((const char*)p + i * (F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) r.w[k] = __builtin_nontemporal_load(q + k);
    return r;
}

template <bool F32>
__device__ __forceinline__ void unpack(const Raw8<F32>& r, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (F32) {
            v[k] = __uint_as_float(r.w[0][k]);
            v[4 + k] = __uint_as_float(r.w[1][k]);
        } else {
            v[2 * k] = lo_bf16(r.w[0][k]);
            v[2 * k + 1] = hi_bf16(r.w[0][k]);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
    if constexpr (F32) {
        u32x4 a, b;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(v[k]);
            b[k] = __float_as_uint(v[4 + k]);
        }
        __builtin_nontemporal_store(a, (u32x4*)((float*)p + i));
        __builtin_nontemporal_store(b, (u32x4*)((float*)p + i) + 1);
    } else {
        u32x4 a;
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
        __builtin_nontemporal_store(a, (u32x4*)((bf16_t*)p + i));
    }
}

// 8 weights (gamma or beta) of either type; `fill` where there are none
__device__ __forceinline__ void load_w8(const void* p, int f32, int64_t i, float fill,
                                        float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fill;
    } else if (f32) {
        Raw8<true> r;
        r.w[0] = ((const u32x4*)((const float*)p + i))[0];
        r.w[1] = ((const u32x4*)((const float*)p + i))[1];
        unpack<true>(r, v);
    } else {
        Raw8<false> r;
        r.w[0] = *(const u32x4*)((const bf16_t*)p + i);
        unpack<false>(r, v);
    }
}

// A kernel's shape: kRows rows side by side in a workgroup, on each kWpr waves
// or, where a row is short, kLanes lanes of a wave; kV steps of 8 values per
// lane.
template <int kLanes_, int kWpr_, int kV_, int kRows_>
struct Shape {
    static constexpr int kLanes = kLanes_, kWpr = kWpr_, kV = kV_, kRows = kRows_;
    static_assert(kLanes == 64 || kWpr == 1, "whole waves on a long row");
    static constexpr int kPer = kLanes * kWpr;         // lanes on a row
    static constexpr int kThreads = kPer * kRows;
    // Rows so wide (above 16384) that gamma and a prefetched row no longer fit
    // beside the row: gamma and beta are read again for every row (from L2),
    // and nothing is prefetched.
    static constexpr bool kLean = kV * kWpr > 32;

    // The thread's row in the workgroup, the same for a whole wave when a row
    // has one, and its place on it.
    static __device__ __forceinline__ int row() {
        if (kLanes < 64) return (int)threadIdx.x / kPer;
        return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) / kWpr;
    }
    static __device__ __forceinline__ int place() { return (int)threadIdx.x % kPer; }
};

// Sum of N values over the lanes of a row; every lane gets it.  `red` holds
// the partial sums of the workgroup's waves; two calls in a row use different
// ones, so one barrier per call is enough.
template <class S, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[N]) {
    if constexpr (S::kLanes < 64) {
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = group_sum<S::kLanes>(v[n]);
        return;
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
        if constexpr (S::kWpr > 1) {
            const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int n = 0; n < N; ++n) red[wave][n] = v[n];
            __syncthreads();
#pragma unroll
            for (int n = 0; n < N; ++n) {
                v[n] = 0.f;
#pragma unroll
                for (int w = 0; w < S::kWpr; ++w) v[n] += red[S::row() * S::kWpr + w][n];
            }
        }
    }
}

// v^-1/2 to half an ulp: the hardware's estimate and one Newton step with the
// product's rounding error carried along (the ends of the range go through
// the division).
__device__ __forceinline__ float inv_sqrt(float v) {
    if (!(v >= 1.17549435e-38f && v <= 3.0e38f)) return 1.f / sqrtf(v);
    const float y = __builtin_amdgcn_rsqf(v);
    const float h = v * y;
    const float e = __builtin_fmaf(-h, y, 1.f) - __builtin_fmaf(v, y, -h) * y;
    return __builtin_fmaf(0.5f * e, y, y);
}

// Hides from the compiler that the words are those it has seen: it would keep
// the unpacked values of the first use, instead of the words, for the second.
__device__ __forceinline__ void forget(u32x4& w) { asm volatile("" : "+v"(w)); }
__device__ __forceinline__ void forget(u32x2& w) { asm volatile("" : "+v"(w)); }
template <bool F32>
__device__ __forceinline__ void forget(Raw8<F32>& r) {
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) forget(r.w[k]);
}

// The forward's shapes by width: few waves on a row and 2 steps.
template <class F>
void with_fwd_shape(int H, F&& f) {
    if (H <= 128) f(Shape<16, 1, 1, 16>{});
    else if (H <= 256) f(Shape<32, 1, 1, 16>{});
    else if (H <= 512) f(Shape<64, 1, 1, 8>{});
    else if (H <= 1024) f(Shape<64, 1, 2, 8>{});
    else if (H <= 2048) f(Shape<64, 2, 2, 4>{});
    else if (H <= 4096) f(Shape<64, 4, 2, 2>{});
    else if (H <= 8192) f(Shape<64, 8, 2, 1>{});
    else if (H <= 16384) f(Shape<64, 16, 2, 1>{});
    else f(Shape<64, 16, 4, 1>{});
}

// Workgroups: enough to fill the chip's waves once (each walks over rows).
template <class S>
unsigned groups_of(int64_t T, int per_cu) {
    const int64_t need = (T + S::kRows - 1) / S::kRows, cap = 256 * per_cu;
    return (unsigned)(need < cap ? need : cap);
}
template <class S>
unsigned fwd_groups(int64_t T) {
    return groups_of<S>(T, S::kThreads >= 1024 ? 1 : S::kThreads >= 512 ? 2 : 4);
}
}  // namespace moe
