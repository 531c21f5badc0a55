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
//
// Two kernels for each.  Rows of 16-byte words (the usual case) come through shared memory
// by bulk asynchronous copies, a copy per row, issued by a warp of their own a token or two
// ahead: what is in flight is then a matter of shared memory, not of registers and warps.
// Any other rows are read directly, two elements or one at a time.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

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
    __device__ __forceinline__ void load_shared(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const Word *>(p)[i];
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

// Chunks of a row that a thread has in flight at once, with KM expert rows each, and the
// blocks of 256 threads that keep an SM supplied with them: registers are capped to let
// kPairBlocks blocks on an SM.
__host__ __device__ constexpr int pair_unroll(int VE, int KM) { return VE == 8 ? 1 : (VE == 2 ? 16 : 32) / KM; }
constexpr int pair_blocks(int KM) { return KM == 4 ? 4 : 2; }

template <class Tok, class Row, int VE, int KM, bool kDot>
__global__ void __launch_bounds__(kPairThreads, pair_blocks(KM)) spread_rows_kernel(PairRows q, const Tok *__restrict__ a,
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
        const int chunks = (int)(q.H / VE);
        const Tok *at = a + t * a_stride;
        constexpr int U = kDot ? pair_unroll(VE, KM) : 4;
        for (int c0 = local; c0 < chunks; c0 += U * q.group) {
            // every load of the step before its first use
            Chunk<Tok, VE> v[U];
            Chunk<Row, VE> y[kDot ? U : 1][kDot ? KM : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * q.group;
                if (c >= chunks) continue;
                v[u].load(at + (int64_t)c * VE);
                if constexpr (kDot) {
#pragma unroll
                    for (int j = 0; j < KM; ++j)
                        if (row[j] >= 0) y[u][j].load(src + row[j] * src_stride + (int64_t)c * VE);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * q.group;
                if (c >= chunks) continue;
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (row[j] < 0) continue;
                    Chunk<Row, VE> o;
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        const float x = v[u].get(i);
                        if constexpr (kDot) dot[j] = fmaf(x, y[u][j].get(i), dot[j]);
                        o.set(i, x * s[j]);
                    }
                    o.store(rows + row[j] * rows_stride + (int64_t)c * VE);
                }
            }
        }
    }
    if constexpr (kDot) write_dots<KM>(q, t, live, dot);
}

template <class Tok, class Row, int VE, int KM, bool kDot>
__global__ void __launch_bounds__(kPairThreads, pair_blocks(KM)) sum_rows_kernel(PairRows q, const Row *__restrict__ rows,
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
        const int chunks = (int)(q.H / VE);
        constexpr int U = pair_unroll(VE, KM);
        for (int c0 = local; c0 < chunks; c0 += U * q.group) {
            Chunk<Row, VE> y[U][KM];
            Chunk<Tok, VE> x[kDot ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * q.group;
                if (c >= chunks) continue;
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    if (row[j] >= 0) y[u][j].load(rows + row[j] * rows_stride + (int64_t)c * VE);
                if constexpr (kDot) x[u].load(a + t * a_stride + (int64_t)c * VE);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * q.group;
                if (c >= chunks) continue;
                float acc[VE];
#pragma unroll
                for (int i = 0; i < VE; ++i) acc[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (row[j] < 0) continue;
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        const float y_i = y[u][j].get(i);
                        if constexpr (kDot) dot[j] = fmaf(x[u].get(i), y_i, dot[j]);
                        acc[i] = fmaf(s[j], y_i, acc[i]);
                    }
                }
                Chunk<Tok, VE> o;
#pragma unroll
                for (int i = 0; i < VE; ++i) o.set(i, acc[i]);
                o.store(out + t * out_stride + (int64_t)c * VE);
            }
        }
    }
    if constexpr (kDot) write_dots<KM>(q, t, live, dot);
}

// ---- rows of 16-byte words --------------------------------------------------------------
constexpr int kBulkWarps = 4;                          // computing warps; one more issues the copies
constexpr int kBulkThreads = 32 * (kBulkWarps + 1);
constexpr int kBulkStages = 4;

// The operands; a stage holds `seg` elements of the token's row (a, if it is read) and of
// each of its k expert rows (rows_in, if they are read).
struct PairBulk {
    const void *a, *rows_in;
    void *out;                    // sum: [T, H] of the token type; spread: [R, H] of the row type
    int64_t a_stride, rows_stride, out_stride;
    int seg, stages, stage_bytes;
};

template <class Tok, class Row, int KM, bool kSum, bool kDot>
__global__ void __launch_bounds__(kBulkThreads) pair_bulk_kernel(const __grid_constant__ PairRows q,
                                                                 const __grid_constant__ PairBulk b) {
    constexpr bool kReadsA = !kSum || kDot, kReadsRows = kSum || kDot;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kBulkStages], empty[kBulkStages];
    __shared__ int row_s[kBulkStages][8];
    __shared__ float weight_s[kBulkStages][8];
    __shared__ float part[2][kBulkWarps][KM];
    __shared__ int failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < b.stages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&empty[i]), kBulkWarps);
        }
        ptx::fence_mbarrier_init();
        failed = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const auto wait = [&](uint64_t &bar, uint32_t parity) {      // after one wait gave up, none waits again
        const uint32_t a = ptx::smem_u32(&bar);
        if (ptx::mbar_test_wait(a, parity) || *reinterpret_cast<volatile int *>(&failed)) return;
        if (!ptx::mbar_wait(a, parity)) *reinterpret_cast<volatile int *>(&failed) = 1;
    };
    const int H = (int)q.H, segs = (H + b.seg - 1) / b.seg;
    const int a_bytes = kReadsA ? b.seg * (int)sizeof(Tok) : 0, row_bytes = b.seg * (int)sizeof(Row);
    int stage = 0;
    uint32_t phase = 0;

    if (warp == kBulkWarps) {
        // lane j < k: pair j of the token, read one token ahead
        const auto pair = [&](int64_t t, int &r, float &w) {
            r = -1;
            w = 1.0f;
            if (t >= q.T || lane >= q.k) return;
            const int64_t p = t * q.k + lane, row = q.pair_rows ? (int64_t)__ldg(q.pair_rows + p) : p;
            if (q.weights) w = __ldg(q.weights + p);
            if (row >= q.R)
                raise_device_error(MOE_DEVERR_OUT_OF_BOUNDS);
            else
                r = row < 0 ? -1 : (int)row;
        };
        int r, next_r;
        float w, next_w;
        pair(blockIdx.x, r, w);
        for (int64_t t = blockIdx.x; t < q.T; t += gridDim.x) {
            pair(t + gridDim.x, next_r, next_w);
            const int used = __popc(__ballot_sync(0xFFFFFFFFu, r >= 0));
            for (int s = 0; s < segs; ++s) {
                const int h0 = s * b.seg, n = min(b.seg, H - h0);
                wait(empty[stage], phase ^ 1u);
                __syncwarp();
                if (lane < 8) {
                    row_s[stage][lane] = r;
                    weight_s[stage][lane] = w;
                }
                __syncwarp();
                const uint32_t bar = ptx::smem_u32(&full[stage]), dst = ptx::smem_u32(ring + stage * b.stage_bytes);
                if (lane == 0)
                    ptx::mbar_arrive_expect_tx(bar, (kReadsRows ? used * n * (int)sizeof(Row) : 0) +
                                                        (kReadsA ? n * (int)sizeof(Tok) : 0));
                __syncwarp();
                if (kReadsRows && r >= 0)
                    ptx::bulk_load(dst + a_bytes + lane * row_bytes,
                                   static_cast<const Row *>(b.rows_in) + r * b.rows_stride + h0, n * (int)sizeof(Row), bar);
                if (kReadsA && lane == 8)
                    ptx::bulk_load(dst, static_cast<const Tok *>(b.a) + t * b.a_stride + h0, n * (int)sizeof(Tok), bar);
                if (++stage == b.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            r = next_r;
            w = next_w;
        }
        return;
    }

    int turn = 0;
    for (int64_t t = blockIdx.x; t < q.T; t += gridDim.x, turn ^= 1) {
        float dot[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
        for (int s = 0; s < segs; ++s) {
            const int h0 = s * b.seg, n = min(b.seg, H - h0);
            wait(full[stage], phase);
            const uint8_t *sa = ring + stage * b.stage_bytes, *sr = sa + a_bytes;
            int row[KM];
            float w[KM];
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                row[j] = row_s[stage][j];
                w[j] = weight_s[stage][j];
            }
            for (int c = tid * 8; c < n; c += 32 * kBulkWarps * 8) {
                Chunk<Tok, 8> x, o;
                if constexpr (kReadsA) x.load_shared(reinterpret_cast<const Tok *>(sa) + c);
                float acc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (row[j] < 0) continue;
                    Chunk<Row, 8> y, z;
                    if constexpr (kReadsRows) y.load_shared(reinterpret_cast<const Row *>(sr + j * row_bytes) + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (kDot) dot[j] = fmaf(x.get(i), y.get(i), dot[j]);
                        if constexpr (kSum) acc[i] = fmaf(w[j], y.get(i), acc[i]);
                        if constexpr (!kSum) z.set(i, x.get(i) * w[j]);
                    }
                    if constexpr (!kSum) z.store(static_cast<Row *>(b.out) + row[j] * b.out_stride + h0 + c);
                }
                if constexpr (kSum) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) o.set(i, acc[i]);
                    o.store(static_cast<Tok *>(b.out) + t * b.out_stride + h0 + c);
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&empty[stage]));
            if (++stage == b.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if constexpr (kDot) {
            // over the lanes, then the warps in order; `part` of the token before last is read by now
#pragma unroll
            for (int j = 0; j < KM; ++j)
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < KM; ++j) part[turn][warp][j] = dot[j];
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kBulkWarps) : "memory");
            if (tid < q.k) {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < kBulkWarps; ++i) v += part[turn][i][tid];
                q.dots[t * q.k + tid] = v;
            }
        }
    }
    if (failed) {                 // a wait gave up: the copies still under way, once more with a limit
        for (int i = 0; i < b.stages; ++i) ptx::mbar_wait(ptx::smem_u32(&full[i]), i < stage ? phase : phase ^ 1u);
    }
}

}  // namespace moe
