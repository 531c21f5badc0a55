// route.cuh -- top-k routing: k largest router logits, then softmax over those k.
//
// The MXFP4 experts take routing data -- expert ids plus routing weights -- rather
// than a dispatch of expert ids (transformers PR #49431 "Restore GPT-OSS's
// router-masked expert-parallel plan").  Selection order: value descending, ties
// to the lower expert index.  Weights: exp(l_j - l_max) / sum_i exp(l_i - l_max)
// over the k chosen logits, in fp32.
//
// One warp per token; each lane holds VPL logits (expert lane + 32 v) in
// registers, k rounds of a warp-wide arg-max with the (value desc, index asc) rule.
// NaN logits are never chosen; a token with fewer than k other logits gets id -1
// and weight 0 in its remaining slots and raises MOE_DEVERR_BAD_LOGIT.
#pragma once
#include "common.cuh"

namespace moe {

template <int VPL>
__global__ void __launch_bounds__(256) route_topk_kernel(const float *__restrict__ logits,
                                                         int64_t T, int E, int k,
                                                         int32_t *__restrict__ ids,
                                                         float *__restrict__ weights) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= T) return;
    const float *row = logits + t * E;
    float v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        v[i] = (e < E) ? __ldg(row + e) : -INFINITY;
    }
    uint32_t taken = 0;  // bit i: slot i of this lane already chosen (or absent)
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i >= E) taken |= 1u << i;

    float sel_v[8];
    int sel_i[8];
    for (int j = 0; j < k; ++j) {
        float bv = -INFINITY;
        int bi = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i;
            const bool ok = !((taken >> i) & 1u);
            if (ok && (v[i] > bv || (v[i] == bv && e < bi))) {
                bv = v[i];
                bi = e;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float ov = __shfl_xor_sync(0xFFFFFFFFu, bv, off);
            const int oi = __shfl_xor_sync(0xFFFFFFFFu, bi, off);
            if (ov > bv || (ov == bv && oi < bi)) {
                bv = ov;
                bi = oi;
            }
        }
        // bi == E-or-more only when every remaining logit is NaN (a NaN never wins a
        // comparison): the slot stays empty
        if (bi < E && (bi & 31) == lane) taken |= 1u << (bi >> 5);
        sel_v[j] = bv;
        sel_i[j] = bi;
    }
    if (lane == 0) {
        // empty slots (fewer than k non-NaN logits) get id -1 and weight 0 and flag
        // the device error word; the softmax runs over the chosen logits only
        const float m = sel_v[0];
        float ex[8], sum = 0.0f;
        for (int j = 0; j < k; ++j) {
            ex[j] = sel_i[j] < E ? expf(sel_v[j] - m) : 0.0f;
            sum += ex[j];
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        for (int j = 0; j < k; ++j) {
            const bool valid = sel_i[j] < E;
            if (!valid) raise_device_error(MOE_DEVERR_BAD_LOGIT);
            ids[t * k + j] = valid ? sel_i[j] : -1;
            weights[t * k + j] = ex[j] * inv;
        }
    }
}

// Gradient of the routing weights with respect to the logits.  w = softmax over the k
// chosen logits, so dlogits[t, ids[t, j]] = w_j (dw_j - sum_i w_i dw_i), and the logits
// that were not chosen do not move the weights: 0.  Empty slots (id -1) give nothing; an
// expert named by two slots of a token gets both, in slot order.  Bound by the stores of
// the dense [T, E] gradient.  A block builds the rows of `tokens` tokens in shared memory
// (one thread per token and its k pairs) and stores them as one contiguous run of 16-byte
// words: per word one shared load and one store, whatever k is.  Measured: 65536 tokens, k = 8
// of 128 experts 10.3 us, 59% of the copy rate (a block's load, clear and store follow each
// other; a thread per word that reads all k pairs took 24 us); 4096 tokens of 32 experts 2.4 us.
constexpr int kRouteGradFloats = 4096;     // of gradient per block (16 KB)
__host__ __device__ constexpr int route_grad_tokens(int E) {
    return kRouteGradFloats / E < 256 ? kRouteGradFloats / E / 4 * 4 : 256;
}

template <bool kWide>    // dlogits 16-byte aligned
__global__ void __launch_bounds__(256) route_backward_kernel(const float *__restrict__ dweights,
                                                             const int32_t *__restrict__ ids,
                                                             const float *__restrict__ weights, int64_t T, int E,
                                                             int k, float *__restrict__ dlogits) {
    __shared__ __align__(16) float grad[kRouteGradFloats];
    const int tokens = route_grad_tokens(E), tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, T - t0) * E;
    pdl_wait();
    pdl_trigger();
    const bool mine = tid < tokens && t0 + tid < T;
    float w[8], g[8];
    int id[8];
    if (mine) {
        const int64_t p = (t0 + tid) * k;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            id[j] = j < k ? __ldg(ids + p + j) : -1;
            w[j] = j < k ? __ldg(weights + p + j) : 0.0f;
            g[j] = j < k ? __ldg(dweights + p + j) : 0.0f;
        }
    }
    for (int i = tid; i < (n + 3) / 4; i += 256) reinterpret_cast<float4 *>(grad)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    if (mine) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool used = id[j] >= 0 && id[j] < E;
            if (!used && id[j] != -1) raise_device_error(MOE_DEVERR_BAD_EXPERT_ID);
            if (!used) id[j] = -1;
            if (used) s = fmaf(w[j], g[j], s);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (id[j] >= 0) grad[tid * E + id[j]] += w[j] * (g[j] - s);
    }
    __syncthreads();
    float *dst = dlogits + t0 * E;       // tokens is a multiple of 4: 16-byte aligned if dlogits is
    if constexpr (kWide) {
        for (int i = tid; i < n / 4; i += 256) reinterpret_cast<float4 *>(dst)[i] = reinterpret_cast<const float4 *>(grad)[i];
        if (tid < n % 4) dst[n / 4 * 4 + tid] = grad[n / 4 * 4 + tid];
    } else {
        for (int i = tid; i < n; i += 256) dst[i] = grad[i];
    }
}

}  // namespace moe
