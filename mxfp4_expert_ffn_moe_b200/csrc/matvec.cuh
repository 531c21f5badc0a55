// matvec.cuh -- products of a few rows with 4-bit weights (MXFP4 or NVFP4).
//
//   y[r, n] = s2 * sum_k W[e, n, k] x[r / rows_per_x, k] + bias[e, n],   e = row_ids[r]
// with W = E2M1(code) * scale(block); kSwiGlu: outputs 2i (gate) and 2i+1 (up) become the
// clamped SwiGLU of the expert layer.
//
// Bound by HBM: a weight is half a byte and serves the few rows of its expert.  At 6.5 TB/s
// an SM has to take 44 weights per clock, so the work per weight decides:
//  * Codes are decoded by cvt.rn.f16x2.e2m1x2 (measured: 1.2 issue slots a weight; shifts and
//    masks take 2.3) and multiplied on the tensor cores by mma.sync m16n8k16 (f16 in, fp32
//    sums): 16 weight rows x 16 k against up to 8 rows of x, so 1 to 8 rows cost the same
//    (measured with the decode alone: 77 weights per clock and SM).  tcgen05 would need the
//    decoded weights in shared memory first, which costs more than the product at these
//    sizes.
//  * f16 holds every E2M1 value, and every E2M1 * E4M3 product (at most 6 significant bits,
//    2^-10 .. 2688), exactly.  bf16 x is brought to f16 by a power of two per row of x
//    (its largest finite value to 2^14 .. 2^15): bf16's 8 bits stay exact down to 2^-31 of
//    the row's largest value and are rounded to 2^-39 of it below, far under the 2^-24 of
//    the fp32 sum.  Products are then exact, the sums are fp32, the result is rounded once.
//  * NVFP4 scales multiply the weights in f16 (exact).  E8M0 scales do not fit f16; they
//    multiply the fp32 sums of their 32-element block, relative to a scale of the warp's
//    slice of the row, so that no intermediate overflows before the result does (blocks
//    2^100 below that scale may lose bits to fp32's subnormals, from 2^127 they drop out).  Each warp turns the scale bytes of its blocks
//    into factors once per stage, a row to a lane, instead of in each lane that uses them.
//  * Weights arrive as TMA boxes of 128 bytes x the item's rows, 128-byte swizzled (the 8
//    rows x 4 words of a fragment load then fall into 32 different banks), into a ring of
//    stages filled by a warp of its own.  An item's scale bytes are one contiguous run that
//    starts anywhere: one bulk copy of the 16-byte granules that hold it.
// An item is kRows weight rows x K against one tile of at most 8 rows of x of one expert;
// CTAs take contiguous runs of items (expert by expert), so the rows of x are staged once
// per expert a CTA meets.  kSplit warps share a group of rows, each with kBlocks blocks of
// 32 elements of every stage; their sums are joined in warp order, so the same call gives
// the same bits.
//
// Measured (device time, gate_up of 64 tokens over 128 experts of 5760 x 2880, 0.98 GB): 202 to
// 220 us in a steady run (about 1.7 GHz under the power cap), 183 us in a short burst, 5.3 TB/s, 82%
// of the copy rate; in bursts also: 150 us with the products left out, and 185 us with all weights
// in L2, so the computing warps bound it.  No single part holds them back (of 193 us then: without
// the decode 180, the mma 195, the factors 182, the join 179): sixteen warps' dependent steps per
// stage do.  More warps with fewer registers, eight warps with twice the rows, epilogue warps of
// their own, deeper or shallower rings and factors made a stage ahead were all slower.  Long K with
// several rows (8 rows of 28672 x 8192 50 us for 19 at the copy rate: x leaves room for the low tile
// only) and more than 8 rows of one matrix (32 of 5760 x 2880 15 us for 1.4: decoded anew for every 8)
// are furthest from it.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "dequant.cuh"
#include "pair_rows.cuh"
#include "ring.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace mv {

constexpr int kTok = 8;                // rows of x of an item (mma N)
constexpr int kMaxStages = 8;
constexpr int kMaxExperts = 256;
constexpr int kMaxRows = 1024;

// kWarps computing warps (one more issues the copies), kSplit of them over the K of each
// group of 16 * kTiles weight rows, with kBlocks 32-element blocks of every stage each.
template <int kWarps_, int kSplit_, int kTiles_, int kBlocks_>
struct Tile {
    static constexpr int kWarps = kWarps_, kSplit = kSplit_, kTiles = kTiles_, kBlocks = kBlocks_;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kGroups = kWarps / kSplit;
    static constexpr int kGroupRows = 16 * kTiles;
    static constexpr int kRows = kGroups * kGroupRows;           // weight rows of an item
    static constexpr int kStageK = kSplit * kBlocks * 32;        // their elements in a stage
    static constexpr int kBoxBytes = kRows * 128;                // 256 elements of every row
    static constexpr int kStageBytes = kStageK / 256 * kBoxBytes;
    static constexpr int kRedBytes = kWarps * kGroupRows * kTok * 4;
    static constexpr int kFactorBytes = kWarps * kBlocks * kGroupRows * 4;   // twice that for NVFP4
    static_assert(kStageK % 256 == 0 && kTiles == 2, "whole boxes; a lane per row of the group");
};

// Shared-memory layout of a call (host-computed; offsets and strides in bytes from a
// 1024-byte boundary).
struct Layout {
    int nt;                // rows of x per tile, at most kTok
    int stages;            // of the weight ring, which starts at 0
    int scale_bufs;        // items whose scales are held
    int scale_stride;      // of a weight row's scales
    int scale_bytes;       // of one item's scales, and its bias (fp32) and scale2 behind them
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
    bool zero_skipped;          // rows whose id is outside [0, E) become zeros
    Layout L;
};

// A row of x is 64 bytes past a multiple of 128, so the two rows of a quarter-warp's
// 16-byte loads fall into different banks.
__host__ __device__ constexpr int x_row_stride(int K) { return 2 * K + ((64 - 2 * K) & 127); }

// Clamped SwiGLU; a NaN stays one (fminf would replace it by the limit).  A result kept in
// fp32 gets the library exponential and a full division; the fast forms' 1e-6 is far below
// the rounding of a 16-bit one.
template <class Out>
__device__ __forceinline__ float swiglu(float gate, float up, float alpha, float limit) {
    const float g = gate > limit ? limit : gate;
    const float u = up > limit ? limit : up < -limit ? -limit : up;
    const float sig = sizeof(Out) == 4 ? 1.0f / (1.0f + expf(-alpha * g)) : __fdividef(1.0f, 1.0f + __expf(-alpha * g));
    return (u + 1.0f) * (g * sig);
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

// Loads of shared memory are volatile: they keep their order with the barriers around them,
// but may move past arithmetic.

// Four 8-row x 16-byte matrices, a row address from each lane (lane l: row l % 8 of matrix
// l / 8): lane (g, t) receives word t of row g of each.
__device__ __forceinline__ uint4 ldmatrix4(uint32_t a) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
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
    uint64_t red_empty[8];          // a group's partial sums are read
    int count[kMaxExperts];         // rows per expert
    int start[kMaxExperts + 1];     // first tile of each expert
    int tok_row[kTok];              // rows r of the staged tile
    int tok_exp[kTok];              // x = staged value * 2^tok_exp
    unsigned tok_max[kTok];
    int failed;                     // a wait gave up
    int16_t ids[kMaxRows];          // the rows' experts, -1 outside [0, E)
};

// Rows per expert and the first tile of each.  Called by the whole block.
template <class T>
__device__ __forceinline__ void count_tiles(const Params &q, Shared &sh) {
    const int tid = threadIdx.x;
    for (int e = tid; e < q.E; e += T::kThreads) sh.count[e] = q.row_ids ? 0 : q.R;
    __syncthreads();
    if (q.row_ids) {
        for (int r = tid; r < q.R; r += T::kThreads) {
            const int e = __ldg(q.row_ids + r);
            const bool known = e >= 0 && e < q.E;
            sh.ids[r] = known ? (int16_t)e : (int16_t)-1;
            if (known)
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

// Rows of tile `slot` of expert e.
__device__ __forceinline__ int tile_rows(const Params &q, const Shared &sh, int e, int slot) {
    return min(q.L.nt, sh.count[e] - (slot - sh.start[e]) * q.L.nt);
}

// The rows of tile `slot` of expert e (ascending r), and their x as f16 in shared memory.
// Called by the computing warps.  Returns the number of rows.  This sits on the critical
// path of a small call and of each change of expert, so it crosses global memory once,
// with all warps on all rows at once (a unit of work is 128 16-byte words of a row, four
// loads in flight a lane); bf16 is converted in place once the rows' largest values are known.
template <class T, class X>
__device__ __forceinline__ int stage_x(const Params &q, Shared &sh, uint8_t *xs, int e, int slot) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j0 = (slot - sh.start[e]) * q.L.nt;
    const int ntok = tile_rows(q, sh, e, slot);
    int *tok_row = sh.tok_row, *tok_exp = sh.tok_exp;
    compute_barrier<T>();           // the previous tile's rows are no longer read
    if (warp == 0) {
        if (q.row_ids) {
            for (int base = 0, seen = 0; base < q.R && seen < j0 + ntok; base += 32) {
                const int r = base + lane;
                const bool mine = r < q.R && sh.ids[r] == e;
                const unsigned m = __ballot_sync(0xFFFFFFFFu, mine);
                const int rank = seen + __popc(m & ((1u << lane) - 1u)) - j0;
                if (mine && rank >= 0 && rank < ntok) tok_row[rank] = r;
                seen += __popc(m);
            }
        } else if (lane < ntok) {
            tok_row[lane] = j0 + lane;
        }
        if (lane < kTok) sh.tok_max[lane] = 0u;
    }
    compute_barrier<T>();
    constexpr bool kScaled = std::is_same<X, __nv_bfloat16>::value;
    const int words = q.K / 8, segs = (words + 127) / 128;
    for (int u = warp; u < ntok * segs; u += T::kWarps) {
        const int t = u / segs, c0 = (u - t * segs) * 128 + lane;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const X *>(q.x) +
                                                           (tok_row[t] / q.rows_per_x) * q.x_stride);
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c0 + 32 * i < words ? __ldg(src + c0 + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c0 + 32 * i < words) *reinterpret_cast<uint4 *>(xs + t * q.L.xs + (c0 + 32 * i) * 16) = v[i];
            if constexpr (kScaled) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
                    m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                }
            }
        }
        if constexpr (kScaled) {
            m = __reduce_max_sync(0xFFFFFFFFu, m);
            if (lane == 0 && m) atomicMax(&sh.tok_max[t], m);
        }
    }
    if constexpr (kScaled) {
        compute_barrier<T>();
        for (int u = warp; u < ntok * segs; u += T::kWarps) {
            const int t = u / segs, c0 = (u - t * segs) * 128 + lane;
            const unsigned m = sh.tok_max[t];
            // exponent of the largest value, less 14; at least -120, so that 2^-exp is a normal fp32
            const int ex = m ? max((int)(m >> 7) - 127 - 14, -120) : 0;
            const float f = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (c0 == 0) tok_exp[t] = ex;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c0 + 32 * i >= words) continue;
                uint4 *p = reinterpret_cast<uint4 *>(xs + t * q.L.xs + (c0 + 32 * i) * 16);
                const uint4 v = *p;
                *p = make_uint4(pack_f16x2(bf16lo_to_f32(v.x) * f, bf16hi_to_f32(v.x) * f),
                                pack_f16x2(bf16lo_to_f32(v.y) * f, bf16hi_to_f32(v.y) * f),
                                pack_f16x2(bf16lo_to_f32(v.z) * f, bf16hi_to_f32(v.z) * f),
                                pack_f16x2(bf16lo_to_f32(v.w) * f, bf16hi_to_f32(v.w) * f));
            }
        }
    } else if (tid < ntok) {
        tok_exp[tid] = 0;
    }
    compute_barrier<T>();
    return ntok;
}

// The scale bytes of weight rows n0 .. n0 + rows - 1 of expert e.  They are a run of bytes
// that starts anywhere, copied as the 16-byte granules that hold it (the first byte lands
// at its address modulo 16); where rows of a multiple of 32 bytes would put the same bytes
// of many rows into one bank, a copy per row spreads them.  Called by one warp; arrives
// once on `full`, behind all that the warp has written.
template <bool kNv>
__device__ __forceinline__ void issue_scales(const Params &q, uint8_t *dst, uint64_t &full, int e, int n0, int rows) {
    const int per_row = q.K / (kNv ? 16 : 32), lane = threadIdx.x & 31;
    const uint32_t bar = ptx::smem_u32(&full);
    const int64_t row0 = (int64_t)e * q.N + n0, first = row0 * per_row, last = first + (int64_t)rows * per_row;
    if (q.L.scale_stride != per_row) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(rows * per_row));
        __syncwarp();
        for (int r = lane; r < rows; r += 32)
            ptx::bulk_load(ptx::smem_u32(dst + r * q.L.scale_stride), q.scales + first + (int64_t)r * per_row, per_row, bar);
        return;
    }
    const int64_t total = (int64_t)q.E * q.N * per_row, lo = first & ~int64_t(15);
    int64_t hi = (last + 15) & ~int64_t(15);
    if (hi > total) {               // the bank's last bytes do not fill a granule: plain loads
        hi = total & ~int64_t(15);
        const int64_t i = max(hi, first) + lane;
        if (i < total) dst[i - lo] = __ldg(q.scales + i);
        ptx::fence_proxy_async_smem();      // a later item's copy writes there through the async proxy
    }
    __syncwarp();
    if (lane == 0) {
        const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) : 0u;
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

// The factors of this warp's n blocks of a stage (block i of the warp is the stage's block
// kSplit * i + part; `first` is block 0 counted from the row's start) for every row of the
// group: MXFP4 [block][g][row / 8] fp32, NVFP4 [block][half][g][row / 8] f16x2 (both halves
// the scale), g = row % 8.
template <class T, bool kNv>
__device__ __forceinline__ void make_factors(uint32_t factors, RowScales &rs, int first, int n,
                                             float (&acc)[T::kTiles][4]) {
    const int lane = threadIdx.x & 31;
    const uint32_t dst = factors + ((lane & 7) * 4 + (lane >> 3)) * 4;
    if constexpr (kNv) {
#pragma unroll
        for (int i = 0; i < T::kBlocks; ++i) {
            const uint32_t a = rs.bytes + 2 * (first + T::kSplit * min(i, n - 1)), c = lds8(a) | (lds8(a + 1) << 8);
            rs.worst = max(rs.worst, max(c & 0x7Fu, (c >> 8) & 0x7Fu));
            const uint32_t both = e4m3x2_to_f16x2(c);
            sts32(dst + 2 * i * 128, __byte_perm(both, both, 0x1010));
            sts32(dst + (2 * i + 1) * 128, __byte_perm(both, both, 0x3232));
        }
    } else {
        int s[T::kBlocks], top = 0;
#pragma unroll
        for (int i = 0; i < T::kBlocks; ++i) {
            s[i] = (int)lds8(rs.bytes + first + T::kSplit * min(i, n - 1));
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
        const int low = rs.ref - 127;
#pragma unroll
        for (int i = 0; i < T::kBlocks; ++i) sts32(dst + i * 128, (uint32_t)(max(s[i], low) - low) << 23);
    }
    __syncwarp();
}

// This warp's n blocks of one stage.  Lane (g, t): rows g, g + 8, g + 16, g + 24 of the
// group, row g of x, elements 8t .. 8t + 7 of a block (the order of k inside an mma is free
// as long as both operands use it).  Swizzled boxes: the 16-byte unit u of row r lies at
// unit u ^ (r % 8), and a block is a unit.  `weights`: this lane's row for ldmatrix, in the
// box of the warp's first block; `unit`: that block's place in the row.  acc: rows g, g + 8
// of tile m x columns 2t, 2t + 1.  kWhole: n = kBlocks, without a test per block.
template <class T, bool kNv, bool kWhole>
__device__ __forceinline__ void multiply_blocks(uint32_t weights, uint32_t unit, uint32_t x, uint32_t factors, int n,
                                                float (&acc)[T::kTiles][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < T::kBlocks; ++i) {
        if (!kWhole && i >= n) break;
        const uint4 w = ldmatrix4(weights + T::kSplit * i / 8 * T::kBoxBytes + (unit ^ ((T::kSplit * i & 7) << 4)));
        const uint4 xv = lds128(x + T::kSplit * i * 64);
        const uint4 f = lds128(factors + (kNv ? (2 * i + (t >> 1)) * 128 : i * 128) + g * 16);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w}, factor[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int m = 0; m < T::kTiles; ++m) {
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(words[2 * m], h0);
            e2m1x8_to_f16(words[2 * m + 1], h1);
            if constexpr (kNv) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h0[j] = mul_f16x2(h0[j], factor[2 * m]);
                    h1[j] = mul_f16x2(h1[j], factor[2 * m + 1]);
                }
                mma_f16<false>(acc[m], h0[0], h1[0], h0[1], h1[1], xv.x, xv.y);
                mma_f16<false>(acc[m], h0[2], h1[2], h0[3], h1[3], xv.z, xv.w);
            } else {
                float c[4];
                mma_f16<true>(c, h0[0], h1[0], h0[1], h1[1], xv.x, xv.y);
                mma_f16<false>(c, h0[2], h1[2], h0[3], h1[3], xv.z, xv.w);
                const float f0 = __uint_as_float(factor[2 * m]), f1 = __uint_as_float(factor[2 * m + 1]);
                acc[m][0] = fmaf(c[0], f0, acc[m][0]);
                acc[m][1] = fmaf(c[1], f0, acc[m][1]);
                acc[m][2] = fmaf(c[2], f1, acc[m][2]);
                acc[m][3] = fmaf(c[3], f1, acc[m][3]);
            }
        }
    }
}

template <class T, class X, class Out, bool kNv, bool kSwiGlu>
__global__ void __launch_bounds__(T::kThreads, 1) matvec_kernel(const __grid_constant__ CUtensorMap weights,
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
        for (int i = 0; i < T::kGroups; ++i) ptx::mbar_init(ptx::smem_u32(&sh.red_empty[i]), T::kSplit);
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
        // The bias and scale2 of an item are loaded while the item before it is issued: waiting
        // for plain loads here would hold the weights up.
        float bias[T::kRows / 32] = {}, scale2 = 1.0f;
        const auto load_tail = [&]() {
            const int64_t row = (int64_t)e * q.N + tile * T::kRows + lane;
#pragma unroll
            for (int i = 0; i < T::kRows / 32; ++i)
                if (q.bias && tile * T::kRows + lane + 32 * i < q.N) bias[i] = __ldg(q.bias + row + 32 * i);
            if (kNv && q.scale2 && lane < 2) scale2 = __ldg(q.scale2 + (kSwiGlu ? 2 * e + lane : e));
        };
        const auto find_expert = [&]() {
            while (sh.start[e + 1] <= slot) ++e;
        };
        if (beg < end) {
            find_expert();
            load_tail();
        }
        bool ok = true;
        for (int it = beg; it < end && ok; ++it) {
            const int e0 = e, n0 = tile * T::kRows;
            for (int c = 0; c < chunks; ++c) {
                ok = __all_sync(0xFFFFFFFFu, wait_or_fail(sh.failed, sh.empty[stage], phase ^ 1u));
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t bar = ptx::smem_u32(&sh.full[stage]);
                    const int boxes = (min(T::kStageK, q.K - c * T::kStageK) + 255) / 256;
                    ptx::mbar_arrive_expect_tx(bar, boxes * T::kBoxBytes);
                    for (int b = 0; b < boxes; ++b)
                        ptx::tma_load_2d(ptx::smem_u32(sm + stage * T::kStageBytes + b * T::kBoxBytes), &weights,
                                         c * (T::kStageK / 2) + b * 128, e0 * q.N + n0, bar);
                }
                if (++stage == q.L.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (c == 0) {
                    ok = __all_sync(0xFFFFFFFFu, wait_or_fail(sh.failed, sh.scales_empty[sbuf], sphase ^ 1u));
                    if (!ok) break;
                    uint8_t *dst = sm + q.L.scales + sbuf * q.L.scale_bytes;
                    float *tail = reinterpret_cast<float *>(dst + q.L.scale_bytes) - 2;
#pragma unroll
                    for (int i = 0; i < T::kRows / 32; ++i) tail[lane + 32 * i - T::kRows] = bias[i];
                    if (lane < 2) tail[lane] = scale2;
                    issue_scales<kNv>(q, dst, sh.scales_full[sbuf], e0, n0, min(T::kRows, q.N - n0));
                    if (++sbuf == q.L.scale_bufs) {
                        sbuf = 0;
                        sphase ^= 1u;
                    }
                    if (++tile == n_tiles) {
                        tile = 0;
                        ++slot;
                    }
                    if (it + 1 < end) {
                        find_expert();
                        load_tail();
                    }
                }
            }
        }
        wait_for_fills(sh.full, q.L.stages, stage, phase);
        wait_for_fills(sh.scales_full, q.L.scale_bufs, sbuf, sphase);
        return;
    }

    constexpr int kRed = T::kGroupRows * kTok;         // outputs of a group
    const int n_out = kSwiGlu ? q.N / 2 : q.N;
    if (q.zero_skipped && q.row_ids)
        for (int r = blockIdx.x; r < q.R; r += gridDim.x)
            if (sh.ids[r] < 0)
                for (int i = tid; i < n_out; i += 32 * T::kWarps)
                    static_cast<Out *>(q.out)[(int64_t)r * n_out + i] = f32_to_elem<Out>(0.0f);
    const int group = warp / T::kSplit, part = warp % T::kSplit, g = lane >> 2, t = lane & 3;
    const int per_row = q.K / (kNv ? 16 : 32);
    const uint32_t ring = ptx::smem_u32(sm) + part / 8 * T::kBoxBytes + (group * T::kGroupRows + lane) * 128;
    const uint32_t unit = ((part ^ lane) & 7) << 4;
    const uint32_t factors = ptx::smem_u32(sm + q.L.factors) + warp * (kNv ? 2 : 1) * (T::kFactorBytes / T::kWarps);
    int staged = -1, ntok = 0;
    bool ok = true;                                    // no wait of this thread for a copy gave up
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
            x0 = ptx::smem_u32(sm + q.L.x) + min(g, ntok - 1) * q.L.xs + part * 64 + t * 16;
        }
        const int my_row = n0 + lane < q.N ? group * T::kGroupRows + lane : 0;
        RowScales rs;
        rs.worst = 0;
        rs.ref = -1;
        rs.bytes = ptx::smem_u32(sm + q.L.scales) + sbuf * q.L.scale_bytes +
                   ((uint32_t)(e * q.N + tile * T::kRows) * (uint32_t)per_row & 15u) + my_row * q.L.scale_stride;
        ok &= wait_or_fail(sh.failed, sh.scales_full[sbuf], sphase);
        float acc[T::kTiles][4];
#pragma unroll
        for (int m = 0; m < T::kTiles; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
        for (int c = 0; c < chunks; ++c) {
            const int first = c * (T::kStageK / 32) + part;
            const int n = (q.K / 32 - first + T::kSplit - 1) / T::kSplit;        // at least kBlocks in a whole stage
            if (n > 0) make_factors<T, kNv>(factors, rs, first, n, acc);
            ok &= wait_or_fail(sh.failed, sh.full[stage], phase);
            const uint32_t w = ring + stage * T::kStageBytes, x = x0 + c * (T::kStageK * 2);
            if (n >= T::kBlocks)
                multiply_blocks<T, kNv, true>(w, unit, x, factors, n, acc);
            else if (n > 0)
                multiply_blocks<T, kNv, false>(w, unit, x, factors, n, acc);
            __syncwarp();
            if (lane == 0 && ok) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[stage]));
            if (++stage == q.L.stages) {
                stage = 0;
                phase ^= 1u;
            }
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
        // join the warps' sums, in warp order; then scale2, bias, activation, one rounding
        float *red = reinterpret_cast<float *>(sm + q.L.red) + group * T::kSplit * kRed;
        float *mine = red + part * kRed + g * kTok + 2 * t;
        wait_or_fail(sh.failed, sh.red_empty[group], ((it - beg) & 1) ^ 1u);      // the previous item's are read
#pragma unroll
        for (int m = 0; m < T::kTiles; ++m) {
            *reinterpret_cast<float2 *>(mine + 16 * m * kTok) = make_float2(acc[m][0], acc[m][1]);
            *reinterpret_cast<float2 *>(mine + (16 * m + 8) * kTok) = make_float2(acc[m][2], acc[m][3]);
        }
        group_barrier(group, 32 * T::kSplit);
        const float *tail = reinterpret_cast<const float *>(sm + q.L.scales + (sbuf + 1) * q.L.scale_bytes) - 2;
        const auto joined = [&](int row, int tok) {      // row of the group
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < T::kSplit; ++w) v += red[w * kRed + row * kTok + tok];
            if constexpr (kNv) v = scale_pow2(v, tok < ntok ? sh.tok_exp[tok] : 0) * tail[kSwiGlu ? row & 1 : 0];
            return v + tail[group * T::kGroupRows + row - T::kRows];
        };
        // a thread's output: a row and a column, or a gate and up row (2i, 2i + 1) and a column
        constexpr int kOutputs = kSwiGlu ? kRed / 2 : kRed;
#pragma unroll
        for (int j = 0; j < (kOutputs + 32 * T::kSplit - 1) / (32 * T::kSplit); ++j) {
            const int o = (j * T::kSplit + part) * 32 + lane, tok = o % kTok, row = (kSwiGlu ? 2 : 1) * (o / kTok);
            if (o >= kOutputs || n0 + row >= q.N || tok >= ntok) continue;
            float v = joined(row, tok);
            if constexpr (kSwiGlu) v = swiglu<Out>(v, joined(row + 1, tok), q.alpha, q.limit);
            static_cast<Out *>(q.out)[(int64_t)sh.tok_row[tok] * n_out + (n0 + row) / (kSwiGlu ? 2 : 1)] = f32_to_elem<Out>(v);
        }
        __syncwarp();
        if (lane == 0) {
            ptx::mbar_arrive(ptx::smem_u32(&sh.red_empty[group]));
            if (ok) ptx::mbar_arrive(ptx::smem_u32(&sh.scales_empty[sbuf]));
        }
        if (++sbuf == q.L.scale_bufs) {
            sbuf = 0;
            sphase ^= 1u;
        }
        if (++tile == n_tiles) {
            tile = 0;
            ++slot;
        }
    }
}

}  // namespace mv
}  // namespace moe
