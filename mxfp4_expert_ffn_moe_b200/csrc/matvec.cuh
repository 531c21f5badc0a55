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
//    multiply the fp32 sums of their 32-element block, relative to the largest scale of the
//    warp's slice of the row, so no intermediate overflows before the result does
//    (blocks 2^-190 below the largest scale of the slice drop out).
//  * Weights arrive by bulk asynchronous copies, one per row of a 16-row tile, into a ring
//    of stages filled by a ninth warp; the scale bytes of each row, which start anywhere,
//    come as the 16-byte granules that hold them.
// An item is 16 weight rows x K against one tile of at most 8 rows of one expert; CTAs take
// contiguous runs of items (expert by expert), so the rows of x are staged once per
// expert a CTA meets.  The eight warps split K by 32-element blocks and their sums are
// joined in warp order: the same call gives the same bits.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "dequant.cuh"
#include "pair_rows.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace mv {

constexpr int kRows = 16;              // weight rows of an item (mma M)
constexpr int kTok = 8;                // rows of x of an item (mma N)
constexpr int kWarps = 8;              // computing warps; one more issues the copies
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxStages = 4;
constexpr int kStageK = 4096;          // most elements of a weight row in one stage
constexpr int kMaxExperts = 256;

// Shared-memory layout of a call (host-computed; offsets and strides in bytes).
struct Layout {
    int nt;                // rows of x per tile, at most kTok
    int kc, chunks;        // elements of a weight row per stage, stages per item
    int stages;
    int ws, ss, xs;        // strides of a weight row, a row's scales, a row of x
    int ring, red, total;  // the rows of x start at 0
};

struct Params {
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
    Layout L;
};

// Strides: a weight row is an odd number of 16-byte units, so the 8 rows x 4 words of a
// fragment load fall into 32 different banks; a row of x is 64 bytes past a multiple of
// 128, so the two rows of a quarter-warp's 16-byte loads do.  A row's scales start at any
// byte of their first granule.
__host__ __device__ constexpr int weight_stride(int kc) { return ((kc / 32) | 1) * 16; }
__host__ __device__ constexpr int scale_stride(int kc, int block) { return (kc / block + 15 + 15) / 16 * 16; }
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

// c += A B, A 16 x 16 (weights), B 16 x 8 (x), f16 in, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

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

__device__ __forceinline__ void compute_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// What a block shares besides the rows of x, the ring and the partial sums.
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int count[kMaxExperts];         // rows per expert
    int start[kMaxExperts + 1];     // first tile of each expert
    int tok_row[kTok];              // rows r of the staged tile
    int tok_exp[kTok];              // x = staged value * 2^tok_exp
    unsigned tok_max[kTok];
    int failed;                     // a wait gave up: all later waits return at once
};

__device__ __forceinline__ void wait_or_fail(Shared &sh, uint64_t &bar, uint32_t parity) {
    if (*reinterpret_cast<volatile int *>(&sh.failed)) return;
    if (!ptx::mbar_wait(ptx::smem_u32(&bar), parity)) *reinterpret_cast<volatile int *>(&sh.failed) = 1;
}

// Rows per expert and the first tile of each.  Called by the whole block.
__device__ __forceinline__ void count_tiles(const Params &q, Shared &sh) {
    const int tid = threadIdx.x;
    for (int e = tid; e < q.E; e += kThreads) sh.count[e] = q.row_ids ? 0 : q.R;
    __syncthreads();
    if (q.row_ids) {
        for (int r = tid; r < q.R; r += kThreads) {
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
template <class X>
__device__ __forceinline__ int stage_x(const Params &q, Shared &sh, uint8_t *xs, int e, int slot) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int j0 = (slot - sh.start[e]) * q.L.nt;
    const int ntok = min(q.L.nt, sh.count[e] - j0);
    compute_barrier();              // the previous tile's rows are no longer read
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
    compute_barrier();
    const int words = q.K / 8;
    const auto row_of = [&](int t) {
        return reinterpret_cast<const uint4 *>(static_cast<const X *>(q.x) + (sh.tok_row[t] / q.rows_per_x) * q.x_stride);
    };
    if constexpr (std::is_same<X, __nv_bfloat16>::value) {
        for (int t = 0; t < ntok; ++t) {
            const uint4 *src = row_of(t);
            unsigned m = 0;
            for (int c = tid; c < words; c += 32 * kWarps) {
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
        compute_barrier();
        for (int t = 0; t < ntok; ++t) {
            const uint4 *src = row_of(t);
            const unsigned m = sh.tok_max[t];
            // exponent of the largest value, less 14; at least -120, so that 2^-exp is a normal fp32
            const int ex = m ? max((int)(m >> 7) - 127 - 14, -120) : 0;
            const float f = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (tid == 0) sh.tok_exp[t] = ex;
            for (int c = tid; c < words; c += 32 * kWarps) {
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
            for (int c = tid; c < words; c += 32 * kWarps)
                *reinterpret_cast<uint4 *>(xs + t * q.L.xs + c * 16) = __ldg(src + c);
        }
    }
    compute_barrier();
    return ntok;
}

// The copies of one stage: lane l < 16 brings weight row l, lane 16 + l the granules of its
// scales.  Every lane arrives once on `bar`.
template <bool kNv>
__device__ __forceinline__ void issue_stage(const Params &q, uint8_t *stage, uint64_t &full, int e, int n0, int k0, int kn) {
    constexpr int kBlock = kNv ? 16 : 32;
    const int lane = threadIdx.x & 31, row = lane & 15;
    const uint32_t bar = ptx::smem_u32(&full);
    if (n0 + row >= q.N) {
        ptx::mbar_arrive(bar);
        return;
    }
    const int64_t first = ((int64_t)e * q.N + n0 + row) * q.K + k0;
    if (lane < 16) {
        ptx::mbar_arrive_expect_tx(bar, kn / 2);
        ptx::bulk_load(ptx::smem_u32(stage + row * q.L.ws), q.blocks + first / 2, kn / 2, bar);
        return;
    }
    const int64_t a = first / kBlock, total = (int64_t)q.E * q.N * (q.K / kBlock);
    const int64_t lo = a & ~int64_t(15);
    int64_t hi = (a + kn / kBlock + 15) & ~int64_t(15);
    uint8_t *dst = stage + kRows * q.L.ws + row * q.L.ss;
    if (hi > total) {               // the bank's last bytes do not fill a granule: plain loads
        hi = total & ~int64_t(15);
        for (int64_t i = max(hi, a); i < total; ++i) dst[i - lo] = __ldg(q.scales + i);
    }
    const uint32_t bytes = (uint32_t)(hi - lo);
    if (!bytes) {
        ptx::mbar_arrive(bar);
        return;
    }
    ptx::mbar_arrive_expect_tx(bar, bytes);
    ptx::bulk_load(ptx::smem_u32(dst), q.scales + lo, bytes, bar);
}

// This warp's 32-element blocks (warp, warp + 8, ...) of one stage.  Lane (g, t): rows g and
// g + 8 of the weights, row g of x, elements 8t .. 8t + 7 of a block (the order of k inside
// an mma is free as long as both operands use it).  acc: rows g, g + 8 x columns 2t, 2t + 1,
// for MXFP4 in units of 2^(e0, e1), see below.
template <bool kNv>
__device__ __forceinline__ void multiply_stage(const Params &q, const uint8_t *xs, const uint8_t *stage, int e, int n0, int k0,
                                               int kn, int ntok, const int (&tok_exp)[2], float (&acc)[4]) {
    constexpr int kBlock = kNv ? 16 : 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int blocks = kn / 32;
    const uint32_t w0 = ptx::smem_u32(stage) + g * q.L.ws + t * 4, w1 = w0 + 8 * q.L.ws;
    const uint32_t x0 = ptx::smem_u32(xs) + g * q.L.xs + k0 * 2 + t * 16;
    const uint32_t sc = ptx::smem_u32(stage) + kRows * q.L.ws;
    // the byte a row's scales start at inside their first granule
    const auto scales_of = [&](int row) {
        return sc + row * q.L.ss + (uint32_t)((((int64_t)e * q.N + n0 + row) * (q.K / kBlock) + k0 / kBlock) & 15);
    };
    const uint32_t s0 = scales_of(g), s1 = scales_of(g + 8);
    const bool x_row = g < ntok;
    if constexpr (kNv) {
        uint32_t worst0 = 0, worst1 = 0;
        for (int b = warp; b < blocks; b += kWarps) {
            const uint32_t c0 = lds8(s0 + 2 * b + (t >> 1)), c1 = lds8(s1 + 2 * b + (t >> 1));
            const uint32_t q0 = lds32(w0 + b * 16), q1 = lds32(w1 + b * 16);
            uint4 xv = make_uint4(0u, 0u, 0u, 0u);
            if (x_row) xv = lds128(x0 + b * 64);
            worst0 = max(worst0, c0 & 0x7Fu);
            worst1 = max(worst1, c1 & 0x7Fu);
            const uint32_t both = e4m3x2_to_f16x2(c0 | (c1 << 8));
            const uint32_t f0 = __byte_perm(both, both, 0x1010), f1 = __byte_perm(both, both, 0x3232);
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(q0, h0);
            e2m1x8_to_f16(q1, h1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h0[i] = mul_f16x2(h0[i], f0);
                h1[i] = mul_f16x2(h1[i], f1);
            }
            mma_f16(acc, h0[0], h1[0], h0[1], h1[1], xv.x, xv.y);
            mma_f16(acc, h0[2], h1[2], h0[3], h1[3], xv.z, xv.w);
        }
        if ((worst0 == 0x7Fu && n0 + g < q.N) || (worst1 == 0x7Fu && n0 + g + 8 < q.N))
            raise_device_error(MOE_DEVERR_BAD_SCALE);
    } else {
        // the largest scale of each row in this warp's blocks: two lanes a row
        uint32_t top = 0;
        if (n0 + (lane >> 1) < q.N) {
            const uint32_t s = scales_of(lane >> 1);
            for (int b = warp + kWarps * (lane & 1); b < blocks; b += 2 * kWarps) top = max(top, lds8(s + b));
        }
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        if (top == 255u) raise_device_error(MOE_DEVERR_BAD_SCALE);
        const int top0 = (int)__shfl_sync(0xFFFFFFFFu, top, 2 * g), top1 = (int)__shfl_sync(0xFFFFFFFFu, top, 2 * (g + 8));
        // scale factors 2^(s - top + 64)
        const int d0 = 191 - top0, d1 = 191 - top1;
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int b = warp; b < blocks; b += kWarps) {
            const int c0 = (int)lds8(s0 + b), c1 = (int)lds8(s1 + b);
            const uint32_t q0 = lds32(w0 + b * 16), q1 = lds32(w1 + b * 16);
            uint4 xv = make_uint4(0u, 0u, 0u, 0u);
            if (x_row) xv = lds128(x0 + b * 64);
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(q0, h0);
            e2m1x8_to_f16(q1, h1);
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(c, h0[0], h1[0], h0[1], h1[1], xv.x, xv.y);
            mma_f16(c, h0[2], h1[2], h0[3], h1[3], xv.z, xv.w);
            const float f0 = __uint_as_float((uint32_t)max(c0 + d0, 0) << 23);
            const float f1 = __uint_as_float((uint32_t)max(c1 + d1, 0) << 23);
            part[0] = fmaf(c[0], f0, part[0]);
            part[1] = fmaf(c[1], f0, part[1]);
            part[2] = fmaf(c[2], f1, part[2]);
            part[3] = fmaf(c[3], f1, part[3]);
        }
        const float nan = __uint_as_float(0x7FC00000u);
        const int e0 = top0 - 127 - 64, e1 = top1 - 127 - 64;
        acc[0] += top0 == 255 ? nan : scale_pow2(part[0], e0 + tok_exp[0]);
        acc[1] += top0 == 255 ? nan : scale_pow2(part[1], e0 + tok_exp[1]);
        acc[2] += top1 == 255 ? nan : scale_pow2(part[2], e1 + tok_exp[0]);
        acc[3] += top1 == 255 ? nan : scale_pow2(part[3], e1 + tok_exp[1]);
    }
}

template <class X, class Out, bool kNv, bool kSwiGlu>
__global__ void __launch_bounds__(kThreads, 2) matvec_kernel(const __grid_constant__ Params q) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < q.L.stages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[i]), 32);
            ptx::mbar_init(ptx::smem_u32(&sh.empty[i]), kWarps);
        }
        ptx::fence_mbarrier_init();
        sh.failed = 0;
    }
    pdl_wait();
    pdl_trigger();
    count_tiles(q, sh);
    const int n_tiles = (q.N + kRows - 1) / kRows;
    const int64_t items = (int64_t)sh.start[q.E] * n_tiles;
    const int beg = (int)(items * blockIdx.x / gridDim.x), end = (int)(items * (blockIdx.x + 1) / gridDim.x);
    const int stage_bytes = kRows * (q.L.ws + q.L.ss);
    uint8_t *ring = sm + q.L.ring;
    int stage = 0, e = 0;
    uint32_t phase = 0;

    if (warp == kWarps) {
        for (int it = beg; it < end; ++it) {
            const int slot = it / n_tiles, n0 = (it - slot * n_tiles) * kRows;
            while (sh.start[e + 1] <= slot) ++e;
            for (int c = 0; c < q.L.chunks; ++c) {
                const int k0 = c * q.L.kc, kn = min(q.L.kc, q.K - k0);
                wait_or_fail(sh, sh.empty[stage], phase ^ 1u);
                __syncwarp();
                issue_stage<kNv>(q, ring + stage * stage_bytes, sh.full[stage], e, n0, k0, kn);
                if (++stage == q.L.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        return;
    }

    float *red = reinterpret_cast<float *>(sm + q.L.red);     // [2][kWarps][kRows][kTok]
    const int n_out = kSwiGlu ? q.N / 2 : q.N;
    int staged = -1, ntok = 0;
    int tok_exp[2] = {0, 0};
    for (int it = beg; it < end; ++it) {
        const int slot = it / n_tiles, n0 = (it - slot * n_tiles) * kRows;
        if (slot != staged) {
            while (sh.start[e + 1] <= slot) ++e;
            ntok = stage_x<X>(q, sh, sm, e, slot);
            staged = slot;
#pragma unroll
            for (int i = 0; i < 2; ++i) tok_exp[i] = 2 * (lane & 3) + i < ntok ? sh.tok_exp[2 * (lane & 3) + i] : 0;
        }
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int c = 0; c < q.L.chunks; ++c) {
            const int k0 = c * q.L.kc, kn = min(q.L.kc, q.K - k0);
            wait_or_fail(sh, sh.full[stage], phase);
            multiply_stage<kNv>(q, sm, ring + stage * stage_bytes, e, n0, k0, kn, ntok, tok_exp, acc);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[stage]));
            if (++stage == q.L.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // join the warps' sums; the other half of `red` was last read before this barrier
        float *part = red + (it & 1) * kWarps * kRows * kTok;
        float *mine = part + warp * kRows * kTok + (lane >> 2) * kTok + 2 * (lane & 3);
        *reinterpret_cast<float2 *>(mine) = make_float2(acc[0], acc[1]);
        *reinterpret_cast<float2 *>(mine + 8 * kTok) = make_float2(acc[2], acc[3]);
        compute_barrier();
        if (tid < kRows * kTok) {
            const int row = tid / kTok, tok = tid % kTok, n = n0 + row;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += part[w * kRows * kTok + tid];
            const bool live = n < q.N && tok < ntok;
            if (live) {
                if constexpr (kNv) {
                    v = scale_pow2(v, sh.tok_exp[tok]);
                    if (q.scale2) v *= __ldg(q.scale2 + (kSwiGlu ? 2 * e + (row & 1) : e));
                }
                if (q.bias) v += __ldg(q.bias + (int64_t)e * q.N + n);
            }
            if constexpr (kSwiGlu) {
                const float up = __shfl_xor_sync(0xFFFFFFFFu, v, kTok);      // row + 1
                if (live && !(row & 1))
                    static_cast<Out *>(q.out)[(int64_t)sh.tok_row[tok] * n_out + n / 2] =
                        f32_to_elem<Out>(clamped_swiglu_f32(v, up, q.alpha, q.limit));
            } else if (live) {
                static_cast<Out *>(q.out)[(int64_t)sh.tok_row[tok] * n_out + n] = f32_to_elem<Out>(v);
            }
        }
    }
    if (sh.failed) {                 // a wait gave up: the copies still under way, once more with a limit
        for (int i = 0; i < q.L.stages; ++i) ptx::mbar_wait(ptx::smem_u32(&sh.full[i]), i < stage ? phase : phase ^ 1u);
    }
}

}  // namespace mv
}  // namespace moe
