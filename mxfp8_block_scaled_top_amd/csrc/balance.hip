// Balance loss and z loss of the router's logits, per-expert counts, and the
// logits' gradient, for gfx950.
//
//   p = softmax(logits of a token),  lse = log sum exp,  n = tokens that count,
//   c_e = their picks of expert e,   f_e = c_e / (n k),  P_e = sum_t p_te / n
//   loss = a E sum_e f_e P_e + z sum_t lse_t^2 / n
//   dlogits_te = dloss [ a E / n p_te (f_e - sum_j f_j p_tj) + 2 z / n lse_t p_te ]
//
// Bound by launches for usual sizes (4 MB of logits at 16384 x 64), by HBM bytes
// beyond.  A token has 2^j lanes with 4 experts each, so its maximum and sums are
// lane shifts, and each lane adds up its own experts' probabilities over the
// tokens it walks.  (Rows of other than multiples of 4 experts start anywhere:
// loads and stores of 16 bytes need 4-byte alignment alone.  One expert a lane takes
// three times as long, 131072 x 60 129 us both ways, so 45.)  Sums are taken in a fixed order: a workgroup's partial
// rows, which a second kernel adds (in one launch where one workgroup has all
// tokens); counts are integers.  No float atomics.
//
// Measured: 256 x 4 4.9 us and 2.2 for the gradient; 16384 x 64, 8 picks, 5.8 + 4.3 and 5.5;
// a million tokens of 64 180 us both ways (5 TB/s).
#include "common.hpp"
#include "kernels.hpp"
#include "trace.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
// Workgroups of the forward: each has a pass over 256 lanes' tokens, from 256 on as
// many as have 16 passes.  us both ways with 256 / 512 / 1024: 16384 x 64 (1024 passes)
// 13.4 / 13.9 / 16.6, 131072 x 8 (1024) 13.7 / 14.7 / 19.0, a million x 8 (7813) 42 / 34 / 34, 131072 x 64
// (8192) 44 / 36 / 35, a million x 64 (62500) 326 / 219 / 180.
constexpr int kParts = 256, kPasses = 16, kMaxParts = 1024;

// Largest or sum over each G neighbouring lanes, the same for all of them.
struct Max { static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); } };
struct Sum { static __device__ __forceinline__ float of(float a, float b) { return a + b; } };
template <class Op, int kCtrl>
__device__ __forceinline__ float dpp_op(float v) {
    return Op::of(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xf, 0xf, true)));
}
template <int G, class Op>
__device__ __forceinline__ float over(float v) {
    if (G >= 2) v = dpp_op<Op, 0xB1>(v);        // quad_perm: lane ^ 1, lane ^ 2
    if (G >= 4) v = dpp_op<Op, 0x4E>(v);
    if (G >= 8) v = dpp_op<Op, 0x141>(v);       // row_half_mirror, row_mirror
    if (G >= 16) v = dpp_op<Op, 0x140>(v);
    return v;
}

struct BalArgs {
    const float* logits;
    const int32_t* topk;
    const uint8_t* mask;        // NULL: every token counts
    int64_t T;
    int E, k;
    float coef, zcoef;
};

constexpr int V = 4;        // experts of a lane

// A token's logits in its lanes' registers (V experts each, -inf past E) to
// probabilities, and its log sum exp.  A token without a finite or infinite
// logit above -inf has no softmax: p = 0, lse = 0.
template <int G>
__device__ __forceinline__ void softmax(float (&x)[V], float& lse) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
    m = over<G, Max>(m);
    const float top = m == -INFINITY ? 0.f : m;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = expf(x[i] - top);
        t += x[i];
    }
    t = over<G, Sum>(t);
    const float inv = t == 0.f ? 0.f : 1.f / t;
    lse = t == 0.f ? 0.f : top + logf(t);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] *= inv;
}

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// Four of a row's E values from e0 on; `none` past the end.
__device__ __forceinline__ void load_row4(const float* row, int e0, int E, float none, float (&x)[4]) {
    if (e0 + 4 <= E) {
        const f32x4u w = *(const f32x4u*)(row + e0);
        x[0] = w[0]; x[1] = w[1]; x[2] = w[2]; x[3] = w[3];
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = e0 + i < E ? row[e0 + i] : none;
}
__device__ __forceinline__ void store_row4(float* row, int e0, int E, const float (&x)[4]) {
    if (e0 + 4 <= E) {
        *(f32x4u*)(row + e0) = (f32x4u){x[0], x[1], x[2], x[3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (e0 + i < E) row[e0 + i] = x[i];
}

// What the sums become: losses [total, balance, z], counts [E], the number of
// tokens, mean probabilities.  The thread of expert e has its
// sums; one wave.
__device__ void finish(const BalArgs& a, int e, double prob, int count, double z, int tokens,
                       float* loss, int32_t* counts, int32_t* ntok, float* mean_prob) {
    const double n = tokens > 0 ? tokens : 1;
    const float pe = (float)(prob / n);
    double b = e < a.E ? (double)pe * (count / (n * a.k)) : 0.0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) b += __shfl_xor(b, o);
    if (e < a.E) {
        counts[e] = count;
        if (mean_prob) mean_prob[e] = pe;
    }
    if (e == 0) {
        *ntok = tokens;
        const double lb = (double)a.coef * a.E * b, lz = (double)a.zcoef * z / n;
        loss[0] = (float)(lb + lz);
        loss[1] = (float)lb;
        loss[2] = (float)lz;
    }
}

// Partial sums of a workgroup: [kMaxParts][E] probabilities, [kMaxParts] of
// lse^2, then as integers [kMaxParts][E] counts and [kMaxParts] tokens.  With
// one workgroup they are the sums, and it writes the outputs.
template <int G>
__global__ __launch_bounds__(kThreads) void balance_fwd_kernel(BalArgs a, float* part, float* loss,
                                                               int32_t* counts, int32_t* ntok, float* mean_prob) {
    constexpr int kSlots = kThreads / G;            // tokens at once
    __shared__ float sp[kThreads / 64][64], sz[kThreads / 64];
    __shared__ int sc[64], sn;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid < 64) sc[tid] = 0;
    if (tid == 0) sn = 0;
    __syncthreads();
    const int e0 = (tid % G) * V;
    float prob[V];
#pragma unroll
    for (int i = 0; i < V; ++i) prob[i] = 0.f;
    float z = 0.f;
    int n = 0;
    for (int64_t t = (int64_t)blockIdx.x * kSlots + tid / G; t < a.T; t += (int64_t)gridDim.x * kSlots) {
        if (a.mask && !a.mask[t]) continue;         // the same for the token's lanes
        float x[V], lse;
        load_row4(a.logits + t * a.E, e0, a.E, -INFINITY, x);
        for (int j = tid % G; j < a.k; j += G) {
            const int e = a.topk[t * a.k + j];
            if ((unsigned)e < (unsigned)a.E) atomicAdd(&sc[e], 1);
        }
        softmax<G>(x, lse);
#pragma unroll
        for (int i = 0; i < V; ++i) prob[i] += x[i];
        if (tid % G == 0) {
            if (a.zcoef != 0.f) z += lse * lse;     // a row of the lowest logits: past fp32's range
            ++n;
        }
    }
    // the tokens of a wave, then the waves in order
#pragma unroll
    for (int o = G; o < 64; o <<= 1)
#pragma unroll
        for (int i = 0; i < V; ++i) prob[i] += __shfl_xor(prob[i], o);
    z = wave_sum(z);
    if (n) atomicAdd(&sn, n);
    if (lane < G)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e0 + i < 64) sp[wave][e0 + i] = prob[i];
    if (lane == 0) sz[wave] = z;
    __syncthreads();
    if (tid >= 64) return;
    const float p = tid < a.E ? (sp[0][tid] + sp[1][tid]) + (sp[2][tid] + sp[3][tid]) : 0.f;
    const float zz = (sz[0] + sz[1]) + (sz[2] + sz[3]);
    if (gridDim.x == 1) {
        finish(a, tid, p, sc[tid], zz, sn, loss, counts, ntok, mean_prob);
        return;
    }
    const int b = blockIdx.x;
    int32_t* ci = (int32_t*)(part + kMaxParts * (a.E + 1));
    if (tid < a.E) {
        part[b * a.E + tid] = p;
        ci[b * a.E + tid] = sc[tid];
    }
    if (tid == 0) {
        part[kMaxParts * a.E + b] = zz;
        ci[kMaxParts * a.E + b] = sn;
    }
}

// The np partial sums added: thread (q, e) takes every 16th of expert e's.
__global__ __launch_bounds__(1024) void balance_sum_kernel(BalArgs a, const float* __restrict__ part, int np,
                                                           float* loss, int32_t* counts,
                                                           int32_t* ntok, float* mean_prob) {
    __shared__ double sp[16][64], sz[16];
    __shared__ int sc[16][64], sn[16];
    const int e = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int32_t* ci = (const int32_t*)(part + kMaxParts * (a.E + 1));
    double p = 0, z = 0;
    int c = 0, n = 0;
    if (e < a.E)
#pragma unroll 8
        for (int b = q; b < np; b += 16) {
            p += part[b * a.E + e];
            c += ci[b * a.E + e];
        }
    for (int b = q + 16 * e; b < np; b += 1024) {       // lane e's: all in one step
        z += part[kMaxParts * a.E + b];
        n += ci[kMaxParts * a.E + b];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        z += __shfl_xor(z, o);
        n += __shfl_xor(n, o);
    }
    sp[q][e] = p;
    sc[q][e] = c;
    if (e == 0) {
        sz[q] = z;
        sn[q] = n;
    }
    __syncthreads();
    if (q) return;
    p = z = 0;
    c = n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        p += sp[w][e];
        c += sc[w][e];
        z += sz[w];
        n += sn[w];
    }
    finish(a, e, p, c, z, n, loss, counts, ntok, mean_prob);
}

template <int G>
__global__ __launch_bounds__(kThreads) void balance_bwd_kernel(BalArgs a, const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ ntok,
                                                               const float* __restrict__ dloss,
                                                               const float* add, float* dlogits) {
    constexpr int kSlots = kThreads / G;
    const int e0 = (threadIdx.x % G) * V;
    const int tokens = *ntok;
    const float n = tokens > 0 ? (float)tokens : 1.f;
    const float up = dloss ? dloss[0] : 1.f;
    const float cb = up * (a.coef * (float)a.E / n), cz = up * (2.f * a.zcoef / n);
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = e0 + i < a.E ? (float)counts[e0 + i] / (n * (float)a.k) : 0.f;
    for (int64_t t = (int64_t)blockIdx.x * kSlots + threadIdx.x / G; t < a.T;
         t += (int64_t)gridDim.x * kSlots) {
        float d[V], x[V];
        const bool live = !(a.mask && !a.mask[t]);      // the same for the token's lanes
        float old[V];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = old[i] = 0.f;
        if (add) load_row4(add + t * a.E, e0, a.E, 0.f, old);
        if (live) {
            float lse, s = 0.f;
            load_row4(a.logits + t * a.E, e0, a.E, -INFINITY, x);
            softmax<G>(x, lse);
#pragma unroll
            for (int i = 0; i < V; ++i) s += x[i] * f[i];
            s = over<G, Sum>(s);
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = x[i] * (cb * (f[i] - s) + cz * lse);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] += old[i];
        store_row4(dlogits + t * a.E, e0, a.E, d);
    }
}

template <int N> struct Num { static constexpr int v = N; };
// Lanes of a token.
template <class F>
void with_lanes(int E, F&& f) {
    if (E <= 4) f(Num<1>{});
    else if (E <= 8) f(Num<2>{});
    else if (E <= 16) f(Num<4>{});
    else if (E <= 32) f(Num<8>{});
    else f(Num<16>{});
}

int64_t passes(int64_t T, int lanes) { return (T + kThreads / lanes - 1) / (kThreads / lanes); }
unsigned parts(int64_t n) {
    const int64_t most = n / kPasses < kParts ? kParts : n / kPasses < kMaxParts ? n / kPasses : kMaxParts;
    return (unsigned)(n < 1 ? 1 : n < most ? n : most);
}

}  // namespace

size_t balance_workspace_bytes(int E) { return (size_t)kMaxParts * 2 * (E + 1) * sizeof(float); }

hipError_t launch_balance_fwd(const float* logits, int64_t T, int E, int k, const int32_t* topk,
                              const uint8_t* mask, float coef, float zcoef, float* loss, int32_t* counts,
                              int32_t* ntok, float* mean_prob, void* ws, hipStream_t s) {
    const BalArgs a{logits, topk, mask, T, E, k, coef, zcoef};
    unsigned np = 1;
    {
        TraceScope ts("balance_fwd", s);
        with_lanes(E, [&](auto g) {
            np = parts(passes(T, decltype(g)::v));
            balance_fwd_kernel<decltype(g)::v>
                <<<np, kThreads, 0, s>>>(a, (float*)ws, loss, counts, ntok, mean_prob);
        });
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || np == 1) return e;
    TraceScope ts("balance_sum", s);
    balance_sum_kernel<<<1, 1024, 0, s>>>(a, (const float*)ws, (int)np, loss, counts, ntok, mean_prob);
    return hipGetLastError();
}

hipError_t launch_balance_bwd(const float* logits, int64_t T, int E, int k, const uint8_t* mask, float coef,
                              float zcoef, const int32_t* counts, const int32_t* ntok, const float* dloss,
                              const float* add, float* dlogits, hipStream_t s) {
    if (T == 0) return hipSuccess;
    const BalArgs a{logits, nullptr, mask, T, E, k, coef, zcoef};
    TraceScope ts("balance_bwd", s);
    with_lanes(E, [&](auto g) {
        const int64_t n = passes(T, decltype(g)::v);
        balance_bwd_kernel<decltype(g)::v>
            <<<(unsigned)(n < 2048 ? n : 2048), kThreads, 0, s>>>(a, counts, ntok, dloss, add, dlogits);
    });
    return hipGetLastError();
}

}  // namespace moe
