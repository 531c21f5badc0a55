// matvec.cuh -- products of a few rows with 4-bit weights (MXFP4 or NVFP4).
//
//   y[r, n] = s2 * sum_k W[e, n, k] x[r / rows_per_x, k] + bias[e, n],   e = row_ids[r]
// with W = E2M1(code) * scale(block); kSwiGlu: outputs 2i (gate) and 2i+1 (up) become the
// clamped SwiGLU of the expert layer.  One warp per output (pair): a lane takes eight
// codes of a row at a time, products and sums in fp32.
#pragma once
#include "common.cuh"
#include "dequant.cuh"
#include "pair_rows.cuh"

namespace moe {

struct MatvecParams {
    const void *x;
    int64_t x_stride;
    int rows_per_x;
    int R, N, K, E;
    const int32_t *row_ids;     // [R] or null (matrix 0)
    const uint8_t *blocks;      // [E, N, K/2]
    const uint8_t *scales;      // [E, N, K/32] E8M0 or [E, N, K/16] E4M3
    const float *scale2;        // NVFP4: [E], or [E, 2] with SwiGLU, or null
    const float *bias;          // [E, N] or null
    float alpha, limit;
    void *out;                  // [R, N] or [R, N/2]
};

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const float mag = m < 2u ? 0.5f * (float)m : __uint_as_float((((m >> 1) + 126u) << 23) | ((m & 1u) << 22));
    return (c & 8u) ? -mag : mag;
}

// Clamped SwiGLU with the library exponential: the result may be kept in fp32.
__device__ __forceinline__ float clamped_swiglu_f32(float gate, float up, float alpha, float limit) {
    const float g = fminf(gate, limit);
    const float u = fminf(fmaxf(up, -limit), limit);
    return (u + 1.0f) * (g / (1.0f + expf(-alpha * g)));
}

template <class X, class Out, bool kNv, bool kSwiGlu>
__global__ void __launch_bounds__(256) matvec_kernel(MatvecParams q) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int n_out = kSwiGlu ? q.N / 2 : q.N;
    const int o = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int r = blockIdx.y;
    if (o >= n_out) return;
    const int e = q.row_ids ? __ldg(q.row_ids + r) : 0;
    if (e < 0 || e >= q.E) {
        raise_device_error(MOE_DEVERR_BAD_EXPERT_ID);
        return;
    }
    const X *x = static_cast<const X *>(q.x) + (r / q.rows_per_x) * q.x_stride;
    float y[kSwiGlu ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (kSwiGlu ? 2 : 1); ++h) {
        const int64_t n = kSwiGlu ? 2 * o + h : o;
        const int64_t row = (int64_t)e * q.N + n;
        const uint32_t *w = reinterpret_cast<const uint32_t *>(q.blocks + row * (q.K / 2));
        const uint8_t *sc = q.scales + row * (q.K / (kNv ? 16 : 32));
        float acc = 0.0f;
        for (int c = lane; c < q.K / 8; c += 32) {
            const uint32_t codes = __ldg(w + c);
            const uint32_t sb = __ldg(sc + c / (kNv ? 2 : 4));
            if (kNv ? (sb & 0x7Fu) == 0x7Fu : sb == 255u) raise_device_error(MOE_DEVERR_BAD_SCALE);
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part = fmaf(e2m1_value((codes >> (4 * i)) & 15u), elem_to_f32(x[c * 8 + i]), part);
            acc = fmaf(part, kNv ? e4m3_byte_value(sb) : e8m0_to_f32(sb), acc);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, d);
        if (kNv && q.scale2) acc *= __ldg(q.scale2 + (kSwiGlu ? 2 * e + h : e));
        if (q.bias) acc += __ldg(q.bias + row);
        y[h] = acc;
    }
    if (lane == 0) {
        float v = y[0];
        if constexpr (kSwiGlu) v = clamped_swiglu_f32(y[0], y[1], q.alpha, q.limit);
        static_cast<Out *>(q.out)[(int64_t)r * n_out + o] = f32_to_elem<Out>(v);
    }
}

}  // namespace moe
