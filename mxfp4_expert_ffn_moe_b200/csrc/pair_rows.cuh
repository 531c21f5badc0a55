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
// Rows come through shared memory by bulk asynchronous copies, a copy per row, issued by a
// warp of their own a token or two ahead: what is in flight is then a matter of shared
// memory, not of registers and warps.  Rows that do not lie on 16-byte words come as the
// 16-byte granules that hold them and are taken apart element by element; the granules at
// the two ends of a tensor, which may not be its own, are read with plain loads.
//
// Measured (device time; share of the 6.55 TB/s copy rate): combine's gradient with the dots,
// 8192 tokens x 4 x 2880 bf16, 76 us, 85%; combine, 4096 x 4 x 2880 bf16, 21 us, 84%; dispatch's
// gradient with the dots, same sizes, 27 us, 79%; combine of fp32 rows 35 us, 92%; 4096 x 4 rows
// of 1001 bf16: combine 11 us, 55%, dispatch 14 us, 45%, their gradients 18 and 15 us.  With direct
// loads (four 16-byte ones in flight a thread) the first five took 85, 23, 32, 35 and 18 us.  The
// spread without dots writes four times what it reads: 8192 tokens 45 us, 80%, by copies where no
// weight is applied, 48 us, 75%, by stores.
#pragma once
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "ring.cuh"
#include "sm100_ptx.cuh"

namespace moe {

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
// two (8 floats), or a single element.
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

// What the kernels take.
struct PairRows {
    int64_t T, H, R;
    int k;
    const int32_t *pair_rows;   // [T*k] or null
    const float *weights;       // [T*k] or null
    float *dots;                // [T*k] (kDot)
};

constexpr int kBulkWarps = 4;                          // computing warps; one more issues the copies
constexpr int kBulkThreads = 32 * (kBulkWarps + 1);
constexpr int kBulkStages = 4;
constexpr uint32_t kGaveUp = 1u << 31;                 // beside a stage's bytes: a reader gave up

// The operands, strides in elements; a stage holds `seg` elements of the token's row (a, if
// it is read) and of each of its k expert rows (rows_in, if they are read).
struct PairBulk {
    const void *a, *rows_in;
    void *out;                    // sum: [T, H] of the token type; spread: [R, H] of the row type
    int64_t a_stride, rows_stride, out_stride;
    int seg, stages;
    int a_slot, row_slot, stage_bytes;      // room for the token's row, an expert row, all of them
    int zero_blocks, zero_room;             // spread: blocks that zero rows, and the rows they can mark at once
};

// Lane j < k of a warp: the expert row of pair j of token t (-1: dropped) and its weight.
// A row past the R rows of the buffer is dropped too and flagged.
__device__ __forceinline__ void load_pair(const PairRows &q, int64_t t, int lane, int &r, float &w) {
    r = -1;
    w = 1.0f;
    if (t >= q.T || lane >= q.k) return;
    const int64_t p = t * q.k + lane, row = q.pair_rows ? (int64_t)__ldg(q.pair_rows + p) : p;
    if (q.weights) w = __ldg(q.weights + p);
    if (row >= q.R)
        raise_device_error(MOE_DEVERR_OUT_OF_BOUNDS);
    else
        r = row < 0 ? -1 : (int)row;
}

// Zeros in the rows of a spread's buffer that no pair names, by blocks of their own (the
// first of the grid) beside those that write the others.  Such a block has a share of the
// rows: it reads all of pair_rows, marks its rows that are named in shared memory, a byte
// each (`marks`, room for `room`), and zeroes the rest.  A row is stored by units: 16-byte
// words or elements.
// They read while the others write, so what they cost shows only where a call is shorter than
// their reading of many pairs (without / with them): dispatch of 4096 x 8 rows of 64 bf16
// 5.9 / 14 us, 4000 x 4 of 512 fp16 5.6 / 7.4; 8192 x 4 of 2880 44.2 / 44.6, combine's gradient
// there 75.4 / 76.2.  Marks as bits, set by shared atomics, took up to 85 us; a fill of the whole
// buffer 30 us there.  Calls of more pairs launch unnamed_rows.cuh's kernel instead.
template <class Unit>
__device__ __forceinline__ void zero_unnamed(const PairRows &q, Unit *rows, int64_t stride, int64_t units, int share, int shares,
                                             uint8_t *marks, int room, int threads) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = (int)q.T * q.k, R = (int)q.R;
    const int lo = (int)((int64_t)R * share / shares), hi = (int)((int64_t)R * (share + 1) / shares);
    const bool wide = (reinterpret_cast<uintptr_t>(q.pair_rows) & 15u) == 0;
    for (int base = lo; base < hi; base += min(room, hi - base)) {
        const int n = min(room, hi - base);
        const auto mark = [&](int r) {
            const unsigned at = (unsigned)r - (unsigned)base;      // past n for negative entries too
            if (at < (unsigned)n) marks[at] = 1;
        };
        __syncthreads();
        for (int i = tid; i < n; i += threads) marks[i] = !q.pair_rows && i < P - base;     // no pair_rows: pair p has row p
        __syncthreads();
        if (q.pair_rows) {
            constexpr int kWords = 8;                      // 16-byte words in flight a thread
            const int words = wide ? P / 4 : 0;
            for (int i = tid; i < words; i += kWords * threads) {
                int4 v[kWords];
#pragma unroll
                for (int u = 0; u < kWords; ++u)
                    v[u] = i + u * threads < words ? __ldg(reinterpret_cast<const int4 *>(q.pair_rows) + i + u * threads)
                                                   : make_int4(-1, -1, -1, -1);
#pragma unroll
                for (int u = 0; u < kWords; ++u) {
                    mark(v[u].x);
                    mark(v[u].y);
                    mark(v[u].z);
                    mark(v[u].w);
                }
            }
            for (int i = 4 * words + tid; i < P; i += min(threads, P - i)) mark(__ldg(q.pair_rows + i));
        }
        __syncthreads();
        for (int i = 32 * warp; i < n; i += threads) {
            unsigned left = __ballot_sync(0xFFFFFFFFu, i + lane < n && !marks[i + lane]);
            for (; left; left &= left - 1) {
                Unit *row = rows + (int64_t)(base + i + __ffs(left) - 1) * stride;
                for (int64_t c = lane; c < units; c += 32) row[c] = Unit{};
            }
        }
    }
}

// The 16-byte granules of [p, p + n * sizeof(T)) inside the tensor [base, end): what a bulk
// copy brings (`lo`, `bytes`); elements in a granule that is not wholly the tensor's are
// stored to `dst` (the shared address of the first granule) by this thread.  A later copy
// into the same stage writes there through the async proxy, hence the fence.
template <class T>
__device__ __forceinline__ void granules(const T *p, int n, const T *base, const T *end, uint8_t *dst, uintptr_t &lo,
                                         uint32_t &bytes) {
    const uintptr_t first = reinterpret_cast<uintptr_t>(p), last = reinterpret_cast<uintptr_t>(p + n);
    const uintptr_t start = first & ~uintptr_t(15);
    uintptr_t hi = (last + 15) & ~uintptr_t(15);
    lo = start;
    const auto plain = [&](uintptr_t from, uintptr_t to) {
        for (uintptr_t i = from; i < to; i += sizeof(T))
            *reinterpret_cast<T *>(dst + (i - start)) = *reinterpret_cast<const T *>(i);
        ptx::fence_proxy_async_smem();
    };
    if (lo < reinterpret_cast<uintptr_t>(base)) {
        lo += 16;
        plain(first, min(lo, last));
    }
    if (hi > reinterpret_cast<uintptr_t>(end) && hi > lo) {
        hi -= 16;
        plain(max(hi, max(first, lo)), last);
    }
    bytes = hi > lo ? (uint32_t)(hi - lo) : 0u;
}

// kWords: every row and segment of every operand lies on 16-byte words.  The spreads' registers
// are bounded to eight blocks an SM, five with the dots: left to the compiler they spill beside
// the zeroing blocks' (combine's gradient of 8192 x 4 x 2880 78 us for 76), and five blocks of the
// plain spread are too few for short rows (131072 x 8 of 64 144 us for 115).  The sums are best
// left alone.
template <class Tok, class Row, int KM, bool kSum, bool kDot, bool kWords>
__global__ void __launch_bounds__(kBulkThreads, kSum ? 0 : kDot ? 5 : 8)
    pair_bulk_kernel(const __grid_constant__ PairRows q, const __grid_constant__ PairBulk b) {
    constexpr bool kReadsA = !kSum || kDot, kReadsRows = kSum || kDot;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kBulkStages], empty[kBulkStages];
    __shared__ int row_s[kBulkStages][8];
    __shared__ float weight_s[kBulkStages][8];
    __shared__ float part[2][kBulkWarps][KM];
    __shared__ int failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int zero_blocks = kSum ? 0 : b.zero_blocks, block = (int)blockIdx.x - zero_blocks, blocks = (int)gridDim.x - zero_blocks;
    if (block < 0) {
        pdl_wait();
        pdl_trigger();
        using Unit = std::conditional_t<kWords, uint4, std::conditional_t<sizeof(Row) == 4, uint32_t, uint16_t>>;
        constexpr int per = sizeof(Unit) / sizeof(Row);
        zero_unnamed(q, static_cast<Unit *>(b.out), b.out_stride / per, q.H / per, blockIdx.x, zero_blocks,
                     ring, b.zero_room, kBulkThreads);
        return;
    }
    if (tid < kBulkStages * 8) row_s[tid / 8][tid % 8] = -1;      // at all times a row of the buffer or none
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
    const int H = (int)q.H, segs = (H + b.seg - 1) / b.seg;
    int stage = 0;
    uint32_t phase = 0;

    if (warp == kBulkWarps) {
        // lane j < k: the row of pair j, read one token ahead; lane 8: the token's row
        const Tok *const a0 = static_cast<const Tok *>(b.a), *const a1 = a0 + (q.T - 1) * b.a_stride + q.H;
        const Row *const r0 = static_cast<const Row *>(b.rows_in), *const r1 = r0 + (q.R - 1) * b.rows_stride + q.H;
        int r, next_r;
        float w, next_w;
        load_pair(q, block, lane, r, w);
        bool ok = true;
        for (int64_t t = block; t < q.T && ok; t += blocks) {
            load_pair(q, t + blocks, lane, next_r, next_w);
            for (int s = 0; s < segs; ++s) {
                const int h0 = s * b.seg, n = min(b.seg, H - h0);
                ok = __all_sync(0xFFFFFFFFu, wait_or_fail(failed, empty[stage], phase ^ 1u));
                if (!ok) break;
                const int gave_up = *static_cast<volatile int *>(&failed);      // tested below, behind its latency
                if (lane < 8) {
                    row_s[stage][lane] = r;
                    weight_s[stage][lane] = w;
                }
                uint8_t *dst = ring + stage * b.stage_bytes;
                uintptr_t src = 0;
                uint32_t bytes = 0;
                if (kReadsRows && r >= 0) {
                    dst += b.a_slot + lane * b.row_slot;
                    const Row *p = r0 + r * b.rows_stride + h0;
                    if constexpr (kWords) {
                        src = reinterpret_cast<uintptr_t>(p);
                        bytes = n * (int)sizeof(Row);
                    } else {
                        granules(p, n, r0, r1, dst, src, bytes);
                        dst += src - (reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
                    }
                } else if (kReadsA && lane == 8) {
                    const Tok *p = a0 + t * b.a_stride + h0;
                    if constexpr (kWords) {
                        src = reinterpret_cast<uintptr_t>(p);
                        bytes = n * (int)sizeof(Tok);
                    } else {
                        granules(p, n, a0, a1, dst, src, bytes);
                        dst += src - (reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
                    }
                }
                const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, lane == 0 && gave_up ? bytes | kGaveUp : bytes);
                const uint32_t bar = ptx::smem_u32(&full[stage]);
                ok = total < kGaveUp;
                if (!ok) break;
                __syncwarp();           // the plain stores above come before the arrival
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, total);
                __syncwarp();
                if (bytes) ptx::bulk_load(ptx::smem_u32(dst), reinterpret_cast<const void *>(src), bytes, bar);
                if (++stage == b.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            r = next_r;
            w = next_w;
        }
        wait_for_fills(full, b.stages, stage, phase);
        return;
    }

    int turn = 0;
    for (int64_t t = block; t < q.T; t += blocks, turn ^= 1) {
        float dot[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
        for (int s = 0; s < segs; ++s) {
            const int h0 = s * b.seg, n = min(b.seg, H - h0);
            wait_or_fail(failed, full[stage], phase);
            const uint8_t *sa = ring + stage * b.stage_bytes;
            int row[KM];
            float w[KM];
            const Row *y_s[KM];
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                row[j] = row_s[stage][j];
                w[j] = weight_s[stage][j];
                const uint8_t *at = sa + b.a_slot + j * b.row_slot;
                if (!kWords && kReadsRows)
                    at += reinterpret_cast<uintptr_t>(static_cast<const Row *>(b.rows_in) + row[j] * b.rows_stride + h0) & 15u;
                y_s[j] = reinterpret_cast<const Row *>(at);
            }
            if (!kWords && kReadsA) sa += reinterpret_cast<uintptr_t>(static_cast<const Tok *>(b.a) + t * b.a_stride + h0) & 15u;
            const Tok *x_s = reinterpret_cast<const Tok *>(sa);
            constexpr int VE = kWords ? 8 : 1;
#pragma unroll(kWords ? 1 : 2)
            for (int c = tid * VE; c < n; c += 32 * kBulkWarps * VE) {
                Chunk<Tok, VE> x, o;
                if constexpr (kReadsA) x.load(x_s + c);
                float acc[VE];
#pragma unroll
                for (int i = 0; i < VE; ++i) acc[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (row[j] < 0) continue;
                    Chunk<Row, VE> y, z;
                    if constexpr (kReadsRows) y.load(y_s[j] + c);
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        if constexpr (kDot) dot[j] = fmaf(x.get(i), y.get(i), dot[j]);
                        if constexpr (kSum) acc[i] = fmaf(w[j], y.get(i), acc[i]);
                        if constexpr (!kSum) z.set(i, x.get(i) * w[j]);
                    }
                    if constexpr (!kSum) z.store(static_cast<Row *>(b.out) + row[j] * b.out_stride + h0 + c);
                }
                if constexpr (kSum) {
#pragma unroll
                    for (int i = 0; i < VE; ++i) o.set(i, acc[i]);
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
}

// The spread of unweighted rows of one type, on 16-byte words: rows[r(p)] = a[t] bit for bit,
// so nothing but copies.  One warp a block: a bulk copy brings a segment of a token's row
// to shared memory, lanes j < k each send it on to their expert row.  Blocks that zero rows
// work with all of kCopyThreads (the launch has 32 where there are none).
constexpr int kCopyStages = 4;
constexpr int kCopyThreads = 128;

__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(const __grid_constant__ PairRows q, const __grid_constant__ PairBulk b,
                                                       int elem) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kCopyStages];
    const int block = (int)blockIdx.x - b.zero_blocks, blocks = (int)gridDim.x - b.zero_blocks;
    if (block < 0) {
        pdl_wait();
        pdl_trigger();
        zero_unnamed(q, static_cast<uint4 *>(b.out), b.out_stride * elem / 16, q.H * elem / 16, blockIdx.x, b.zero_blocks,
                     ring, b.zero_room, kCopyThreads);
        return;
    }
    const int lane = threadIdx.x, segs = (int)((q.H + b.seg - 1) / b.seg);
    if (lane >= 32) return;
    if (lane == 0) {
        for (int i = 0; i < kCopyStages; ++i) ptx::mbar_init(ptx::smem_u32(&full[i]), 1);
        ptx::fence_mbarrier_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    // the next segment to fetch, its stage and that stage's parity; lane 0 issues the copy
    int64_t ft = block;
    int fs = 0, fstage = 0;
    uint32_t fphase = 0;
    const auto bytes_of = [&](int seg) { return (uint32_t)(min(b.seg, (int)q.H - seg * b.seg) * elem); };
    const auto fetch = [&]() {
        if (ft >= q.T) return;
        if (lane == 0) {
            const uint32_t bar = ptx::smem_u32(&full[fstage]), bytes = bytes_of(fs);
            ptx::mbar_arrive_expect_tx(bar, bytes);
            ptx::bulk_load(ptx::smem_u32(ring + fstage * b.stage_bytes),
                           static_cast<const uint8_t *>(b.a) + (ft * b.a_stride + (int64_t)fs * b.seg) * elem, bytes, bar);
        }
        fstage = (fstage + 1) % kCopyStages;
        if (fstage == 0) fphase ^= 1u;
        if (++fs == segs) {
            fs = 0;
            ft += blocks;
        }
    };
    for (int i = 0; i < kCopyStages - 1; ++i) fetch();
    int r, next_r, stage = 0;
    uint32_t phase = 0;
    float w;
    bool ok = true;
    load_pair(q, block, lane, r, w);
    for (int64_t t = block; t < q.T && ok; t += blocks, r = next_r) {
        load_pair(q, t + blocks, lane, next_r, w);
        for (int s = 0; s < segs && ok; ++s) {
            ok = __all_sync(0xFFFFFFFFu, ring_wait(full[stage], phase));
            if (ok && r >= 0)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                 static_cast<uint8_t *>(b.out) + (r * b.out_stride + (int64_t)s * b.seg) * elem),
                             "r"(ptx::smem_u32(ring + stage * b.stage_bytes)), "r"(bytes_of(s))
                             : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            // the next fetch takes the previous segment's stage: that one is read when one group is left
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
            if (ok) fetch();
            stage = (stage + 1) % kCopyStages;
            if (stage == 0) phase ^= 1u;
        }
    }
    if (!ok) wait_for_fills(full, kCopyStages, fstage, fphase);      // a wait gave up, up to three fetches behind the last
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace moe
