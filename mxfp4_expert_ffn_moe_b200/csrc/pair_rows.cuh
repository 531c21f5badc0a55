// pair_rows.cuh -- token rows to expert rows and back, with the routing weights applied,
// and the gradients of both directions.
//
// Pair p = t*k + j of token t has the expert row r(p) = pair_rows[p] (permute.cuh; -1 for
// a dropped pair, p itself without pair_rows) and the weight s_p (1 without weights).
//   spread:  rows[r(p)] = s_p a[t]         dots: dw_p = <a[t], src[r(p)]>
//   sum:     out[t] = sum_j s_p rows[r(p)]  dots: dw_p = <a[t], rows[r(p)]>
// The two are transposes of each other, so the spread is the forward pass of the dispatch
// and the gradient of the combine, and the sum is the combine and the gradient of the
// dispatch; the dots are the gradient of the weights.  Sums and dots run in fp32 in a
// fixed order (slots ascending; a thread's chunks ascending, then a shuffle tree over
// lanes and warps), each result is rounded once: the same call gives the same bits.
//
// Bound by HBM: every token row and every expert row crosses it once.  Both walk the
// tokens, not the expert rows: a token's row is then read (written) once instead of k
// times, and its k expert rows are whole contiguous runs wherever they lie.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

constexpr int kPairThreads = 256;

// ---- VE elements of a row as fp32 --------------------------------------------------
__device__ __forceinline__ float elem_to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem_to_f32(float v) { return v; }
template <class T>
__device__ __forceinline__ T f32_to_elem(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 f32_to_elem<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half f32_to_elem<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float f32_to_elem<float>(float v) { return v; }

// VE consecutive elements as they lie in memory: one 16-byte word (8 two-byte elements),
// two (8 floats), or one word of 2 or 1 elements.
template <class T, int VE>
struct Chunk {
    static constexpr int kBytes = VE * (int)sizeof(T);
    static constexpr int kWord = kBytes >= 16 ? 16 : kBytes;
    static constexpr int kWords = kBytes / kWord;
    struct alignas(kWord) Word {
        T e[kWord / sizeof(T)];
    };
    Word w[kWords];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (kWord == 16) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[i] = *reinterpret_cast<const Word *>(&v);
            } else {
                w[i] = reinterpret_cast<const Word *>(p)[i];
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<Word *>(p)[i] = w[i];
    }
    __device__ __forceinline__ float get(int i) const {
        constexpr int n = kWord / sizeof(T);
        return elem_to_f32(w[i / n].e[i % n]);
    }
    __device__ __forceinline__ void set(int i, float v) {
        constexpr int n = kWord / sizeof(T);
        w[i / n].e[i % n] = f32_to_elem<T>(v);
    }
};

// What both kernels take.  Strides are in elements.
struct PairRows {
    int64_t T, H, R;
    int k;
    int group;                  // threads per token: 32 .. 256, a power of two
    const int32_t *pair_rows;   // [T*k] or null
    const float *weights;       // [T*k] or null
    float *dots;                // [T*k] (kDot)
};

// The expert rows and weights of one token; a dropped pair gets row -1.  A row past the
// R rows of the buffer is dropped too and flagged.
template <int KM>
__device__ __forceinline__ void load_pairs(const PairRows &q, int64_t t, int (&row)[KM], float (&s)[KM]) {
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        row[j] = -1;
        s[j] = 1.0f;
        if (j < q.k) {
            const int64_t p = t * q.k + j;
            const int64_t r = q.pair_rows ? (int64_t)__ldg(q.pair_rows + p) : p;
            if (r >= q.R)
                raise_device_error(MOE_DEVERR_OUT_OF_BOUNDS);
            else
                row[j] = r < 0 ? -1 : (int)r;
            if (q.weights) s[j] = __ldg(q.weights + p);
        }
    }
}

// Sum of each dot over the token's `group` threads, written by its first thread.  Called
// by all threads of the block.
template <int KM>
__device__ __forceinline__ void write_dots(const PairRows &q, int64_t t, bool live, float (&dot)[KM]) {
    __shared__ float part[kPairThreads / 32][KM];
#pragma unroll
    for (int j = 0; j < KM; ++j)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int j = 0; j < KM; ++j) part[warp][j] = dot[j];
    __syncthreads();
    const int local = threadIdx.x & (q.group - 1);
    if (live && local < q.k) {
        float v = 0.0f;
        for (int w = 0; w < q.group / 32; ++w) v += part[warp + w][local];   // local < 32: warp is the group's first
        q.dots[t * q.k + local] = v;
    }
}

template <class Tok, class Row, int VE, int KM, bool kDot>
__global__ void __launch_bounds__(kPairThreads) spread_rows_kernel(PairRows q, const Tok *__restrict__ a,
                                                                   int64_t a_stride, const Row *__restrict__ src,
                                                                   int64_t src_stride, Row *__restrict__ rows,
                                                                   int64_t rows_stride) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = (int64_t)blockIdx.x * (kPairThreads / q.group) + threadIdx.x / q.group;
    const int local = threadIdx.x & (q.group - 1);
    const bool live = t < q.T;
    float dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
    if (live) {
        int row[KM];
        float s[KM];
        load_pairs<KM>(q, t, row, s);
        const int64_t chunks = q.H / VE;
        const Tok *at = a + t * a_stride;
        constexpr int U = kDot ? 2 : 4;
        for (int64_t c0 = local; c0 < chunks; c0 += U * q.group) {
            Chunk<Tok, VE> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * q.group < chunks) v[u].load(at + (c0 + u * q.group) * VE);
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                if (row[j] < 0) continue;
                Chunk<Row, VE> y[U];
                if constexpr (kDot) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (c0 + u * q.group < chunks) y[u].load(src + row[j] * src_stride + (c0 + u * q.group) * VE);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c0 + u * q.group >= chunks) continue;
                    Chunk<Row, VE> o;
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        const float x = v[u].get(i);
                        if constexpr (kDot) dot[j] = fmaf(x, y[u].get(i), dot[j]);
                        o.set(i, x * s[j]);
                    }
                    o.store(rows + row[j] * rows_stride + (c0 + u * q.group) * VE);
                }
            }
        }
    }
    if constexpr (kDot) write_dots<KM>(q, t, live, dot);
}

template <class Tok, class Row, int VE, int KM, bool kDot>
__global__ void __launch_bounds__(kPairThreads) sum_rows_kernel(PairRows q, const Row *__restrict__ rows,
                                                                int64_t rows_stride, const Tok *__restrict__ a,
                                                                int64_t a_stride, Tok *__restrict__ out,
                                                                int64_t out_stride) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = (int64_t)blockIdx.x * (kPairThreads / q.group) + threadIdx.x / q.group;
    const int local = threadIdx.x & (q.group - 1);
    const bool live = t < q.T;
    float dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
    if (live) {
        int row[KM];
        float s[KM];
        load_pairs<KM>(q, t, row, s);
        const int64_t chunks = q.H / VE;
        for (int64_t c = local; c < chunks; c += q.group) {
            Chunk<Row, VE> y[KM];
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (row[j] >= 0) y[j].load(rows + row[j] * rows_stride + c * VE);
            Chunk<Tok, VE> x;
            if constexpr (kDot) x.load(a + t * a_stride + c * VE);
            float acc[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) acc[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                if (row[j] < 0) continue;
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float y_i = y[j].get(i);
                    if constexpr (kDot) dot[j] = fmaf(x.get(i), y_i, dot[j]);
                    acc[i] = fmaf(s[j], y_i, acc[i]);
                }
            }
            Chunk<Tok, VE> o;
#pragma unroll
            for (int i = 0; i < VE; ++i) o.set(i, acc[i]);
            o.store(out + t * out_stride + c * VE);
        }
    }
    if constexpr (kDot) write_dots<KM>(q, t, live, dot);
}

}  // namespace moe
