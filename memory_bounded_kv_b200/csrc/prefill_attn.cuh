// Retention-gated attention over packed prompts ("Cache What Lasts" section 2.1: the weight of key
// j for query i is proportional to exp(q_i . k_j + (i - j) log beta_j)), with an optional tanh cap
// of the scores and an optional prefix whose tokens see each other, and its gradients.
//
// Documents are rows [cu[n], cu[n + 1]) of the packed tensors; row i of a document sees the keys
// j < max(i + 1, prefix_n) of the same document, at the distance max(i - j, 0). A key at distance 0
// has no bias, whatever its log beta (so beta = 0 leaves a token visible to itself alone).
#pragma once

#include "prefill_units.cuh"

namespace kvb {

// ---- one warp per row: the plainest form -------------------------------------

template <int D>
__device__ __forceinline__ void row_load(float (&x)[D / 32], const uint16_t* row, int lane) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x[e] = bf16_lo(row[lane + 32 * e]);
}
template <int D>
__device__ __forceinline__ float row_dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) s = fmaf(a[e], b[e], s);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(kFull, s, m);
    return s;
}
template <int D>
__device__ __forceinline__ void row_store(uint16_t* row, const float (&x)[D / 32], float f, int lane) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) row[lane + 32 * e] = __bfloat16_as_ushort(__float2bfloat16_rn(x[e] * f));
}

__device__ __forceinline__ int prefill_prefix(const PrefillParams& p, int n, int len) {
    return p.prefix == nullptr ? 0 : min(max(p.prefix[n], 0), len);
}

// logit of (i, j) from the dot product, and the derivative of the capped score
__device__ __forceinline__ float prefill_logit(const PrefillParams& p, float dot, int i, int j, int s, int g, float& slope) {
    float x = dot * p.scale;
    slope = 1.f;
    if (p.softcap > 0.f) {
        const float t = tanhf(x / p.softcap);
        x = p.softcap * t;
        slope = 1.f - t * t;
    }
    if (p.lb != nullptr && i > j) x += (float)(i - j) * p.lb[(long long)(s + j) * p.lb_st + g * p.lb_sh];
    return x;
}

// grid: (documents, heads, blocks of rows); 8 rows per block step
// dq and delta, one warp per query row
template <int D>
__global__ void __launch_bounds__(256) prefill_dq_rows_kernel(const __grid_constant__ PrefillParams p) {
    griddep_wait();
    if (!prefill_docs_ok(p.cu, p.N, p.T)) return;
    const int s = p.cu[blockIdx.x], e = p.cu[blockIdx.x + 1];
    const int h = blockIdx.y, g = h / p.G, lane = threadIdx.x & 31, len = e - s;
    const int pre = prefill_prefix(p, blockIdx.x, len);
    for (int i = blockIdx.z * 8 + (threadIdx.x >> 5); i < len; i += gridDim.z * 8) {
        const size_t row = (size_t)(s + i) * p.Hq + h;
        float q[D / 32], dq[D / 32] = {}, k[D / 32], v[D / 32], go[D / 32];
        row_load<D>(q, p.q + (long long)(s + i) * p.q_st + h * p.q_sh, lane);
        row_load<D>(go, p.d_o + row * D, lane);
        const float lse = p.lse[row];
        float delta = 0.f, slope;
        for (int pass = 0; pass < 2; ++pass) {
            for (int j = 0; j < max(i + 1, pre); ++j) {
                row_load<D>(k, p.k + (long long)(s + j) * p.kv_st + g * p.kv_sh, lane);
                row_load<D>(v, p.v + (long long)(s + j) * p.kv_st + g * p.kv_sh, lane);
                const float w = expf(prefill_logit(p, row_dot<D>(q, k), i, j, s, g, slope) - lse);
                const float dp = row_dot<D>(go, v);
                if (pass == 0) {
                    delta = fmaf(w, dp, delta);
                } else {
                    const float ds = w * (dp - delta) * slope;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) dq[c] = fmaf(ds, k[c], dq[c]);
                }
            }
            if (pass == 0 && p.d_lse != nullptr) delta -= p.d_lse[row];
        }
        row_store<D>(p.dq + row * D, dq, p.scale, lane);
        if (lane == 0) p.delta[row] = delta;
    }
}

// dk, dv and dlog_beta, one warp per key row
template <int D>
__global__ void __launch_bounds__(256) prefill_dkv_rows_kernel(const __grid_constant__ PrefillParams p) {
    griddep_wait();
    if (!prefill_docs_ok(p.cu, p.N, p.T)) return;
    const int s = p.cu[blockIdx.x], e = p.cu[blockIdx.x + 1];
    const int g = blockIdx.y, lane = threadIdx.x & 31, len = e - s;
    const int pre = prefill_prefix(p, blockIdx.x, len);
    for (int j = blockIdx.z * 8 + (threadIdx.x >> 5); j < len; j += gridDim.z * 8) {
        float q[D / 32], k[D / 32], v[D / 32], go[D / 32], dk[D / 32] = {}, dv[D / 32] = {};
        row_load<D>(k, p.k + (long long)(s + j) * p.kv_st + g * p.kv_sh, lane);
        row_load<D>(v, p.v + (long long)(s + j) * p.kv_st + g * p.kv_sh, lane);
        float dlb = 0.f, slope;
        for (int i = j < pre ? 0 : j; i < len; ++i)
            for (int h = g * p.G; h < (g + 1) * p.G; ++h) {
                const size_t row = (size_t)(s + i) * p.Hq + h;
                row_load<D>(q, p.q + (long long)(s + i) * p.q_st + h * p.q_sh, lane);
                row_load<D>(go, p.d_o + row * D, lane);
                const float w = expf(prefill_logit(p, row_dot<D>(q, k), i, j, s, g, slope) - p.lse[row]);
                float ds = w * (row_dot<D>(go, v) - p.delta[row]);
                dlb = fmaf(ds, (float)max(i - j, 0), dlb);
                ds *= slope;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    dv[c] = fmaf(w, go[c], dv[c]);
                    dk[c] = fmaf(ds, q[c], dk[c]);
                }
            }
        const size_t row = (size_t)(s + j) * p.Hkv + g;
        row_store<D>(p.dk + row * D, dk, p.scale, lane);
        row_store<D>(p.dv + row * D, dv, 1.f, lane);
        if (lane == 0 && p.dlb != nullptr) p.dlb[row] = dlb;
    }
}

}  // namespace kvb
