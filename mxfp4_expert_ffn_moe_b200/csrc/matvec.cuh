// matvec.cuh -- products of a few rows with 4-bit weights (MXFP4 or NVFP4).
//
//   y[r, n] = s2 * sum_k W[e, n, k] x[r / rows_per_x, k] + bias[e, n],   e = row_ids[r]
// with W = E2M1(code) * scale(block); kSwiGlu: outputs 2i (gate) and 2i+1 (up) become the
// clamped SwiGLU of the expert layer.
//
// Bound by HBM: a weight is half a byte and serves the few rows of its expert.  At 6.5 TB/s
// an SM has to take 44 weights per clock, so the work per weight decides:
//  * Codes are decoded by cvt.rn.f16x2.e2m1x2 (two per instruction, measured at over 400
//    weights per clock and SM; prmt tables with sign bits reach 170) and multiplied on the
//    tensor cores by mma.sync m16n8k16 (f16 in, fp32 sums): 16 weight rows x 16 k against
//    up to 8 rows of x, so 1 to 8 rows cost the same (measured with the decode: 77
//    weights per clock and SM).  tcgen05 would need the decoded weights in shared memory
//    first, which costs more than the product at these sizes.
//  * f16 holds every E2M1 value, and every E2M1 * E4M3 product (at most 6 significant bits,
//    2^-10 .. 2688), exactly.  bf16 x is brought to f16 by a power of two per row of x
//    (its largest finite value to 2^14 .. 2^15): bf16's 8 bits stay exact down to 2^-31 of
//    the row's largest value and are rounded to 2^-39 of it below, far under the 2^-24 of
//    the fp32 sum.  Products are then exact, the sums are fp32, the result is rounded once.
//  * NVFP4 scales multiply the weights in f16 (exact).  E8M0 scales do not fit f16; they
//    multiply the fp32 sums of their 32-element block, relative to a scale of the warp's
//    slice of the row, so that no intermediate overflows before the result does (blocks
//    2^-126 below that scale drop out).  Each warp turns the scale bytes of its blocks into
//    factors once per stage, a row to a lane, instead of in each of the lanes that use them.
//  * Weights arrive as TMA boxes of 128 bytes x the item's rows, 128-byte swizzled (the 8
//    rows x 4 words of a fragment load then fall into 32 different banks), into a ring of
//    stages filled by a ninth warp.  An item's scale bytes are one contiguous run that
//    starts anywhere: one bulk copy of the 16-byte granules that hold it.
// An item is kRows weight rows x K against one tile of at most 8 rows of x of one expert;
// CTAs take contiguous runs of items (expert by expert), so the rows of x are staged once
// per expert a CTA meets.  kSplit warps share a group of rows, each with 4 blocks of 32
// elements of every stage; their sums are joined in warp order, so the same call gives
// the same bits.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "dequant.cuh"
#include "pair_rows.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace mv {

constexpr int kTok = 8;                // rows of x of an item (mma N)
constexpr int kMaxStages = 4;
constexpr int kMaxExperts = 256;
constexpr int kWarpBlocks = 4;         // 32-element blocks of a warp in one stage

// kWarps computing warps (one more issues the copies), kSplit of them over the K of each
// group of 16 * kTiles weight rows; kBlocksPerSm such blocks on an SM.
template <int kWarps_, int kSplit_, int kTiles_, int kBlocksPerSm_>
struct Tile {
    static constexpr int kWarps = kWarps_, kSplit = kSplit_, kTiles = kTiles_, kBlocksPerSm = kBlocksPerSm_;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kGroups = kWarps / kSplit;
    static constexpr int kGroupRows = 16 * kTiles;
    static constexpr int kRows = kGroups * kGroupRows;           // weight rows of an item
    static constexpr int kStageK = kSplit * kWarpBlocks * 32;    // their elements in a stage
    static constexpr int kBoxBytes = kRows * 128;                // 256 elements of every row
    static constexpr int kStageBytes = kStageK / 256 * kBoxBytes;
    static constexpr int kRedBytes = kWarps * kGroupRows * kTok * 4;
    static constexpr int kFactorBytes = kWarps * kWarpBlocks * kGroupRows * 4;   // twice that for NVFP4
};
#ifndef MOE_WIDE
#define MOE_WIDE 16, 4, 2, 1
#endif
using WideTile = Tile<MOE_WIDE>;        // 128 rows x 512 elements a stage
using NarrowTile = Tile<8, 8, 1, 2>;    // 16 rows x 1024 elements a stage

// Shared-memory layout of a call (host-computed; offsets and strides in bytes from a
// 1024-byte boundary).
struct Layout {
    int nt;                // rows of x per tile, at most kTok
    int stages;            // of the weight ring, which starts at 0
    int scale_bufs;        // items whose scales are held
    int scale_bytes;       // of one item
    int xs;                // stride of a row of x
    int x, scales, red, factors, total;
};

struct Params {
    const void *x;
    int64_t x_stride;
    int rows_per_x;
    int R, N, K, E;
    const int32_t *row_ids;     // [R] or null (matrix 0)
    const uint8_t *scales;      // [E, N, K/32] E8M0 or [E, N, K/16] E4M3
    const float *scale2;        // NVFP4: [E], or [E, 2] with SwiGLU, or null
    const float *bias;          // [E, N] or null
    float alpha, limit;
    void *out;                  // [R, N] or [R, N/2]
    Layout L;
};

// A row of x is 64 bytes past a multiple of 128, so the two rows of a quarter-warp's
// 16-byte loads fall into different banks.
__host__ __device__ constexpr int x_row_stride(int K) { return 2 * K + ((64 - 2 * K) & 127); }

// Clamped SwiGLU with the library exponential and a full division: the result may be kept
// in fp32.
__device__ __forceinline__ float clamped_swiglu_f32(float gate, float up, float alpha, float limit) {
    const float g = fminf(gate, limit);
    const float u = fminf(fmaxf(up, -limit), limit);
    return (u + 1.0f) * (g / (1.0f + expf(-alpha * g)));
}

// Eight E2M1 codes (element 2j in the low nibble of byte j) -> four f16x2 words.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t q, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
    uint32_t h;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(pair));
    return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// d = A B (kNew) or d += A B, A 16 x 16 (weights), B 16 x 8 (x), f16 in, fp32 sums.
template <bool kNew>
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    if constexpr (kNew)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Loads of shared memory in program order with the barriers around them, but free to move
// past arithmetic.
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// v * 2^e for any e, in two steps within the normal exponents.
__device__ __forceinline__ float scale_pow2(float v, int e) {
    const int a = max(-126, min(127, e)), b = max(-126, min(127, e - a));
    return v * __uint_as_float((uint32_t)(a + 127) << 23) * __uint_as_float((uint32_t)(b + 127) << 23);
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ void group_barrier(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(2 + group), "r"(threads) : "memory");
}
template <class T>
__device__ __forceinline__ void compute_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * T::kWarps) : "memory");
}

// What a block shares besides the rows of x, the ring and the partial sums.
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];      // weight stages
    uint64_t scales_full[2], scales_empty[2];
    int count[kMaxExperts];         // rows per expert
    int start[kMaxExperts + 1];     // first tile of each expert
    int tok_row[kTok];              // rows r of the staged tile
    int tok_exp[kTok];              // x = staged value * 2^tok_exp
    unsigned tok_max[kTok];
    int failed;                     // a wait gave up: all later waits return at once
};

__device__ __noinline__ void slow_wait(Shared &sh, uint32_t bar, uint32_t parity) {
    volatile int *failed = &sh.failed;
    if (!*failed && !ptx::mbar_wait(bar, parity)) *failed = 1;
}
__device__ __forceinline__ void wait_or_fail(Shared &sh, uint64_t &bar, uint32_t parity) {
    const uint32_t a = ptx::smem_u32(&bar);
    if (!ptx::mbar_test_wait(a, parity)) slow_wait(sh, a, parity);
}

// Rows per expert and the first tile of each.  Called by the whole block.
template <class T>
__device__ __forceinline__ void count_tiles(const Params &q, Shared &sh) {
    const int tid = threadIdx.x;
    for (int e = tid; e < q.E; e += T::kThreads) sh.count[e] = q.row_ids ? 0 : q.R;
    __syncthreads();
    if (q.row_ids) {
        for (int r = tid; r < q.R; r += T::kThreads) {
            const int e = __ldg(q.row_ids + r);
            if (e >= 0 && e < q.E)
                atomicAdd(&sh.count[e], 1);
            else if (blockIdx.x == 0)
                raise_device_error(MOE_DEVERR_BAD_EXPERT_ID);
        }
        __syncthreads();
    }
    if (tid < 32) {
        const int per = (q.E + 31) / 32, e0 = tid * per, e1 = min(e0 + per, q.E);
        int sum = 0;
        for (int e = e0; e < e1; ++e) sum += (sh.count[e] + q.L.nt - 1) / q.L.nt;
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (tid >= d) incl += v;
        }
        int run = incl - sum;
        for (int e = e0; e < e1; ++e) {
            sh.start[e] = run;
            run += (sh.count[e] + q.L.nt - 1) / q.L.nt;
        }
        if (tid == 31) sh.start[q.E] = incl;
    }
    __syncthreads();
}

// The rows of tile `slot` of expert e (ascending r), and their x as f16 in shared memory.
// Called by the computing warps.  Returns the number of rows.
template <class T, class X>
__device__ __forceinline__ int stage_x(const Params &q, Shared &sh, uint8_t *xs, int e, int slot) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int j0 = (slot - sh.start[e]) * q.L.nt;
    const int ntok = min(q.L.nt, sh.count[e] - j0);
    compute_barrier<T>();              // the previous tile's rows are no longer read
    if (tid < 32) {
        if (q.row_ids) {
            int seen = 0;
            for (int base = 0; base < q.R && seen < j0 + ntok; base += 32) {
                const int r = base + lane;
                const bool mine = r < q.R && __ldg(q.row_ids + r) == e;
                const unsigned m = __ballot_sync(0xFFFFFFFFu, mine);
                const int rank = seen + __popc(m & ((1u << lane) - 1u)) - j0;
                if (mine && rank >= 0 && rank < ntok) sh.tok_row[rank] = r;
                seen += __popc(m);
            }
        } else if (lane < ntok) {
            sh.tok_row[lane] = j0 + lane;
        }
        if (lane < kTok) sh.tok_max[lane] = 0u;
    }
    compute_barrier<T>();
    const int words = q.K / 8;
    const auto row_of = [&](int t) {
        return reinterpret_cast<const uint4 *>(static_cast<const X *>(q.x) + (sh.tok_row[t] / q.rows_per_x) * q.x_stride);
    };
    if constexpr (std::is_same<X, __nv_bfloat16>::value) {
        for (int t = 0; t < ntok; ++t) {
            const uint4 *src = row_of(t);
            unsigned m = 0;
            for (int c = tid; c < words; c += 32 * T::kWarps) {
                const uint4 v = __ldg(src + c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
                    if (lo < 0x7F80u) m = max(m, lo);
                    if (hi < 0x7F80u) m = max(m, hi);
                }
            }
            m = __reduce_max_sync(0xFFFFFFFFu, m);
            if (lane == 0 && m) atomicMax(&sh.tok_max[t], m);
        }
        compute_barrier<T>();
        for (int t = 0; t < ntok; ++t) {
            const uint4 *src = row_of(t);
            const unsigned m = sh.tok_max[t];
            // exponent of the largest value, less 14; at least -120, so that 2^-exp is a normal fp32
            const int ex = m ? max((int)(m >> 7) - 127 - 14, -120) : 0;
            const float f = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (tid == 0) sh.tok_exp[t] = ex;
            for (int c = tid; c < words; c += 32 * T::kWarps) {
                const uint4 v = __ldg(src + c);
                uint4 h;
                h.x = pack_f16x2(bf16lo_to_f32(v.x) * f, bf16hi_to_f32(v.x) * f);
                h.y = pack_f16x2(bf16lo_to_f32(v.y) * f, bf16hi_to_f32(v.y) * f);
                h.z = pack_f16x2(bf16lo_to_f32(v.z) * f, bf16hi_to_f32(v.z) * f);
                h.w = pack_f16x2(bf16lo_to_f32(v.w) * f, bf16hi_to_f32(v.w) * f);
                *reinterpret_cast<uint4 *>(xs + t * q.L.xs + c * 16) = h;
            }
        }
    } else {
        for (int t = 0; t < ntok; ++t) {
            const uint4 *src = row_of(t);
            if (tid == 0) sh.tok_exp[t] = 0;
            for (int c = tid; c < words; c += 32 * T::kWarps)
                *reinterpret_cast<uint4 *>(xs + t * q.L.xs + c * 16) = __ldg(src + c);
        }
    }
    compute_barrier<T>();
    return ntok;
}

// The scale bytes of weight rows n0 .. n0 + rows - 1 of expert e: a run of bytes that starts
// anywhere, copied as the 16-byte granules that hold it (the first byte lands at its
// address modulo 16).  Called by one warp; arrives once on `full`.
template <bool kNv>
__device__ __forceinline__ void issue_scales(const Params &q, uint8_t *dst, uint64_t &full, int e, int n0, int rows) {
    const int per_row = q.K / (kNv ? 16 : 32), lane = threadIdx.x & 31;
    const int64_t first = ((int64_t)e * q.N + n0) * per_row, last = first + (int64_t)rows * per_row;
    const int64_t total = (int64_t)q.E * q.N * per_row, lo = first & ~int64_t(15);
    int64_t hi = (last + 15) & ~int64_t(15);
    if (hi > total) {               // the bank's last bytes do not fill a granule: plain loads
        hi = total & ~int64_t(15);
        const int64_t i = max(hi, first) + lane;
        if (i < total) dst[i - lo] = __ldg(q.scales + i);
        __syncwarp();
    }
    if (lane == 0) {
        const uint32_t bar = ptx::smem_u32(&full), bytes = hi > lo ? (uint32_t)(hi - lo) : 0u;
        ptx::mbar_arrive_expect_tx(bar, bytes);
        if (bytes) ptx::bulk_load(ptx::smem_u32(dst), q.scales + lo, bytes, bar);
    }
}

// What a warp keeps of the rows of its group while it works on an item.  Lane l stands for
// row l when the scales become factors; lanes without a row of the matrix read its first.
struct RowScales {
    uint32_t bytes;      // shared address of the row's scale bytes
    uint32_t worst;      // MXFP4: the largest scale met; NVFP4: without the sign
    int ref;             // MXFP4: factors are relative to this scale
};

// The factors of this warp's blocks first .. first + n - 1 (of 32 elements) of every row:
// MXFP4 [block][g][row / 8] fp32, NVFP4 [block][half][g][row / 8] f16x2 (both halves the
// scale), g = row % 8.
template <class T, bool kNv>
__device__ __forceinline__ void make_factors(uint32_t factors, RowScales &rs, int first, int n,
                                             float (&acc)[T::kTiles][4]) {
    const int lane = threadIdx.x & 31, g = lane & 7, r = lane >> 3;
    const bool mine = lane < T::kGroupRows;
    const uint32_t dst = factors + (g * 2 * T::kTiles + r) * 4;
    constexpr int kStep = 8 * 2 * T::kTiles * 4;        // bytes of the factors of one block (half)
    if constexpr (kNv) {
#pragma unroll
        for (int i = 0; i < kWarpBlocks; ++i) {
            if (i >= n) break;
            const uint32_t a = rs.bytes + 2 * (first + i), c = lds8(a) | (lds8(a + 1) << 8);
            rs.worst = max(rs.worst, max(c & 0x7Fu, (c >> 8) & 0x7Fu));
            const uint32_t both = e4m3x2_to_f16x2(c);
            if (mine) {
                sts32(dst + 2 * i * kStep, __byte_perm(both, both, 0x1010));
                sts32(dst + (2 * i + 1) * kStep, __byte_perm(both, both, 0x3232));
            }
        }
    } else {
        int s[kWarpBlocks], top = 0;
#pragma unroll
        for (int i = 0; i < kWarpBlocks; ++i) {
            s[i] = (int)lds8(rs.bytes + first + min(i, n - 1));
            top = max(top, s[i]);
        }
        rs.worst = max(rs.worst, (uint32_t)top);
        if (rs.ref < 0) rs.ref = top;
        // Factors stay below 2^64: when a later stage brings larger scales, the sums are
        // brought to the new reference.
        const int up = top > rs.ref + 64 ? top - rs.ref : 0;
        if (__any_sync(0xFFFFFFFFu, up)) {
            rs.ref += up;
#pragma unroll
            for (int m = 0; m < T::kTiles; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int by = __shfl_sync(0xFFFFFFFFu, up, (lane >> 2) + 8 * h + 16 * m);
                    acc[m][2 * h] = scale_pow2(acc[m][2 * h], -by);
                    acc[m][2 * h + 1] = scale_pow2(acc[m][2 * h + 1], -by);
                }
        }
        if (mine) {
            const int low = rs.ref - 127;
#pragma unroll
            for (int i = 0; i < kWarpBlocks; ++i) sts32(dst + i * kStep, (uint32_t)(max(s[i], low) - low) << 23);
        }
    }
    __syncwarp();
}

// This warp's n (at most kWarpBlocks) blocks of one stage.  Lane (g, t): rows g, g + 8, ...
// of the group, row g of x, elements 8t .. 8t + 7 of a block (the order of k inside an mma
// is free as long as both operands use it).  Swizzled boxes: the 16-byte unit u of row r
// lies at unit u ^ (r % 8), and a block is a unit.  acc: rows g, g + 8 of tile m x columns
// 2t, 2t + 1.
template <class T, bool kNv, bool kWhole>
__device__ __forceinline__ void multiply_blocks(uint32_t weights, uint32_t x, uint32_t factors, int unit, int n,
                                                float (&acc)[T::kTiles][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < kWarpBlocks; ++i) {
        if (!kWhole && i >= n) break;
        const uint32_t w = weights + (((unit + i) ^ g) << 4);
        const uint4 xv = lds128(x + i * 64);
        uint32_t f[2 * T::kTiles];
        const uint32_t fa = factors + (kNv ? (2 * i + (t >> 1)) * 8 + g : i * 8 + g) * 8 * T::kTiles;
        if constexpr (T::kTiles == 2) {
            const uint4 v = lds128(fa);
            f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
        } else {
            const uint2 v = lds64(fa);
            f[0] = v.x, f[1] = v.y;
        }
#pragma unroll
        for (int m = 0; m < T::kTiles; ++m) {
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(lds32(w + m * 2048), h0);
            e2m1x8_to_f16(lds32(w + m * 2048 + 1024), h1);
            if constexpr (kNv) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h0[j] = mul_f16x2(h0[j], f[2 * m]);
                    h1[j] = mul_f16x2(h1[j], f[2 * m + 1]);
                }
                mma_f16<false>(acc[m], h0[0], h1[0], h0[1], h1[1], xv.x, xv.y);
                mma_f16<false>(acc[m], h0[2], h1[2], h0[3], h1[3], xv.z, xv.w);
            } else {
                float c[4];
                mma_f16<true>(c, h0[0], h1[0], h0[1], h1[1], xv.x, xv.y);
                mma_f16<false>(c, h0[2], h1[2], h0[3], h1[3], xv.z, xv.w);
                const float f0 = __uint_as_float(f[2 * m]), f1 = __uint_as_float(f[2 * m + 1]);
                acc[m][0] = fmaf(c[0], f0, acc[m][0]);
                acc[m][1] = fmaf(c[1], f0, acc[m][1]);
                acc[m][2] = fmaf(c[2], f1, acc[m][2]);
                acc[m][3] = fmaf(c[3], f1, acc[m][3]);
            }
        }
    }
}

template <class T, class X, class Out, bool kNv, bool kSwiGlu>
__global__ void __launch_bounds__(T::kThreads, T::kBlocksPerSm) matvec_kernel(const __grid_constant__ CUtensorMap weights,
                                                             const __grid_constant__ Params q) {
    extern __shared__ uint8_t dynamic_smem[];
    __shared__ Shared sh;
    uint8_t *sm = dynamic_smem + ((1024u - (ptx::smem_u32(dynamic_smem) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < q.L.stages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.empty[i]), T::kWarps);
        }
        for (int i = 0; i < q.L.scale_bufs; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh.scales_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.scales_empty[i]), T::kWarps);
        }
        ptx::fence_mbarrier_init();
        sh.failed = 0;
    }
    pdl_wait();
    pdl_trigger();
    count_tiles<T>(q, sh);
    const int n_tiles = (q.N + T::kRows - 1) / T::kRows, chunks = (q.K + T::kStageK - 1) / T::kStageK;
    const int64_t items = (int64_t)sh.start[q.E] * n_tiles;
    const int beg = (int)(items * blockIdx.x / gridDim.x), end = (int)(items * (blockIdx.x + 1) / gridDim.x);
    int slot = beg / n_tiles, tile = beg - slot * n_tiles, e = 0;
    int stage = 0, sbuf = 0;
    uint32_t phase = 0, sphase = 0;

    if (warp == T::kWarps) {
        for (int it = beg; it < end; ++it) {
            while (sh.start[e + 1] <= slot) ++e;
            const int n0 = tile * T::kRows;
            for (int c = 0; c < chunks; ++c) {
                wait_or_fail(sh, sh.empty[stage], phase ^ 1u);
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = ptx::smem_u32(&sh.full[stage]);
                    const int units = min(T::kStageK, q.K - c * T::kStageK);
                    const int boxes = (units + 255) / 256;
                    ptx::mbar_arrive_expect_tx(bar, boxes * T::kBoxBytes);
                    for (int b = 0; b < boxes; ++b)
                        ptx::tma_load_2d(ptx::smem_u32(sm + stage * T::kStageBytes + b * T::kBoxBytes), &weights,
                                         c * (T::kStageK / 2) + b * 128, e * q.N + n0, bar);
                }
                if (c == 0) {
                    wait_or_fail(sh, sh.scales_empty[sbuf], sphase ^ 1u);
                    __syncwarp();
                    issue_scales<kNv>(q, sm + q.L.scales + sbuf * q.L.scale_bytes, sh.scales_full[sbuf], e, n0,
                                      min(T::kRows, q.N - n0));
                    if (++sbuf == q.L.scale_bufs) {
                        sbuf = 0;
                        sphase ^= 1u;
                    }
                }
                if (++stage == q.L.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (++tile == n_tiles) {
                tile = 0;
                ++slot;
            }
        }
        return;
    }

    const int group = warp / T::kSplit, part = warp % T::kSplit, g = lane >> 2, t = lane & 3;
    const int per_row = q.K / (kNv ? 16 : 32);
    const int n_out = kSwiGlu ? q.N / 2 : q.N;
    const uint32_t ring = ptx::smem_u32(sm) + part / 2 * T::kBoxBytes + (group * T::kGroupRows + g) * 128 + t * 4;
    const uint32_t factors = ptx::smem_u32(sm + q.L.factors) + warp * (kNv ? 2 : 1) * (T::kFactorBytes / T::kWarps);
    float *red = reinterpret_cast<float *>(sm + q.L.red) + group * T::kSplit * T::kGroupRows * kTok;
    int staged = -1, ntok = 0;
    int tok_exp[2] = {0, 0};
    uint32_t x0 = 0;
    for (int it = beg; it < end; ++it) {
        const int n0 = tile * T::kRows + group * T::kGroupRows;      // this group's first row
        if (slot != staged) {
            while (sh.start[e + 1] <= slot) ++e;
            ntok = stage_x<T, X>(q, sh, sm + q.L.x, e, slot);
            staged = slot;
#pragma unroll
            for (int i = 0; i < 2; ++i) tok_exp[i] = 2 * t + i < ntok ? sh.tok_exp[2 * t + i] : 0;
            // columns past the staged rows repeat the last one (and are not stored)
            x0 = ptx::smem_u32(sm + q.L.x) + min(g, ntok - 1) * q.L.xs + part * (kWarpBlocks * 64) + t * 16;
        }
        const int my_row = lane < T::kGroupRows && n0 + lane < q.N ? group * T::kGroupRows + lane : 0;
        RowScales rs;
        rs.worst = 0;
        rs.ref = -1;
        rs.bytes = ptx::smem_u32(sm + q.L.scales) + sbuf * q.L.scale_bytes +
                   ((uint32_t)(e * q.N + tile * T::kRows) * (uint32_t)per_row & 15u) + my_row * per_row;
        // the bias and scale of the outputs this thread will store
        constexpr int kOut = T::kGroupRows * kTok / (32 * T::kSplit) > 0 ? T::kGroupRows * kTok / (32 * T::kSplit) : 1;
        float bias[kOut], scale2[kOut];
#pragma unroll
        for (int j = 0; j < kOut; ++j) {
            const int row = (part * 32 + lane + j * 32 * T::kSplit) / kTok, n = n0 + row;
            const bool live = row < T::kGroupRows && n < q.N;
            bias[j] = live && q.bias ? __ldg(q.bias + (int64_t)e * q.N + n) : 0.0f;
            scale2[j] = kNv && live && q.scale2 ? __ldg(q.scale2 + (kSwiGlu ? 2 * e + (row & 1) : e)) : 1.0f;
        }
        wait_or_fail(sh, sh.scales_full[sbuf], sphase);
        float acc[T::kTiles][4];
#pragma unroll
        for (int m = 0; m < T::kTiles; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
        for (int c = 0; c < chunks; ++c) {
            const int first = c * (T::kStageK / 32) + part * kWarpBlocks, n = min(kWarpBlocks, q.K / 32 - first);
            if (n > 0) make_factors<T, kNv>(factors, rs, first, n, acc);
            wait_or_fail(sh, sh.full[stage], phase);
            // whole stages without a test per block, so that all their loads go out first
            if (n == kWarpBlocks)
                multiply_blocks<T, kNv, true>(ring + stage * T::kStageBytes, x0 + c * (T::kStageK * 2), factors,
                                              (part & 1) * kWarpBlocks, n, acc);
            else if (n > 0)
                multiply_blocks<T, kNv, false>(ring + stage * T::kStageBytes, x0 + c * (T::kStageK * 2), factors,
                                               (part & 1) * kWarpBlocks, n, acc);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[stage]));
            if (++stage == q.L.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.scales_empty[sbuf]));
        if (++sbuf == q.L.scale_bufs) {
            sbuf = 0;
            sphase ^= 1u;
        }
        if (rs.worst == (kNv ? 127u : 255u)) raise_device_error(MOE_DEVERR_BAD_SCALE);
        if constexpr (!kNv) {
            // from the reference scales and the staged x to the true scale
            int ex[T::kTiles][2];
            bool plain = rs.worst != 255u;
#pragma unroll
            for (int m = 0; m < T::kTiles; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ex[m][h] = __shfl_sync(0xFFFFFFFFu, rs.ref - 127, g + 8 * h + 16 * m);
                    plain = plain && min(ex[m][h] + tok_exp[0], ex[m][h] + tok_exp[1]) >= -126 &&
                            max(ex[m][h] + tok_exp[0], ex[m][h] + tok_exp[1]) <= 127;
                }
            if (__all_sync(0xFFFFFFFFu, plain)) {
#pragma unroll
                for (int m = 0; m < T::kTiles; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[m][i] *= __uint_as_float((uint32_t)(ex[m][i >> 1] + tok_exp[i & 1] + 127) << 23);
            } else {              // exponents past fp32's own, or a row that an invalid scale makes NaN
#pragma unroll
                for (int m = 0; m < T::kTiles; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool bad = __shfl_sync(0xFFFFFFFFu, rs.worst, g + 8 * (i >> 1) + 16 * m) == 255u;
                        acc[m][i] = bad ? __uint_as_float(0x7FC00000u) : scale_pow2(acc[m][i], ex[m][i >> 1] + tok_exp[i & 1]);
                    }
            }
        }
        // join the warps' sums
        group_barrier(group, 32 * T::kSplit);          // the previous item's are read
#pragma unroll
        for (int m = 0; m < T::kTiles; ++m) {
            float *mine = red + (part * T::kGroupRows + 16 * m + g) * kTok + 2 * t;
            *reinterpret_cast<float2 *>(mine) = make_float2(acc[m][0], acc[m][1]);
            *reinterpret_cast<float2 *>(mine + 8 * kTok) = make_float2(acc[m][2], acc[m][3]);
        }
        group_barrier(group, 32 * T::kSplit);
#pragma unroll
        for (int j = 0; j < kOut; ++j) {
            const int o = part * 32 + lane + j * 32 * T::kSplit;
            if (o >= T::kGroupRows * kTok) break;                      // whole warps
            const int row = o / kTok, tok = o % kTok, n = n0 + row;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < T::kSplit; ++w) v += red[w * T::kGroupRows * kTok + o];
            const bool live = n < q.N && tok < ntok;
            if constexpr (kNv) v = live ? scale_pow2(v, sh.tok_exp[tok]) * scale2[j] : 0.0f;
            v += bias[j];
            if constexpr (kSwiGlu) {
                const float up = __shfl_xor_sync(0xFFFFFFFFu, v, kTok);      // row + 1
                if (live && !(row & 1))
                    static_cast<Out *>(q.out)[(int64_t)sh.tok_row[tok] * n_out + n / 2] =
                        f32_to_elem<Out>(clamped_swiglu_f32(v, up, q.alpha, q.limit));
            } else if (live) {
                static_cast<Out *>(q.out)[(int64_t)sh.tok_row[tok] * n_out + n] = f32_to_elem<Out>(v);
            }
        }
        if (++tile == n_tiles) {
            tile = 0;
            ++slot;
        }
    }
    if (sh.failed) {                 // a wait gave up: the copies still under way, once more with a limit
        for (int i = 0; i < q.L.stages; ++i) ptx::mbar_wait(ptx::smem_u32(&sh.full[i]), i < stage ? phase : phase ^ 1u);
        for (int i = 0; i < q.L.scale_bufs; ++i)
            ptx::mbar_wait(ptx::smem_u32(&sh.scales_full[i]), i < sbuf ? sphase : sphase ^ 1u);
    }
}

}  // namespace mv
}  // namespace moe
