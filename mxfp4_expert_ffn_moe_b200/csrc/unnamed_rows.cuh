// unnamed_rows.cuh -- zeros in the rows of a spread's buffer (pair_rows.cuh) that no pair
// names, by a launch behind the spread, for calls of many pairs.
//
// A cluster of eight blocks has a share of the rows.  Each block reads an eighth of
// pair_rows and marks the rows named, a byte each, in the shared memory of the block that
// keeps them (row i of the share: block i % 8); then each zeroes its rows that are not
// marked.  So all pairs are read once per cluster, not once per block, and the rows are
// written by all SMs.  Where no row is left out it takes 8 us of a call for 131072 pairs,
// 30 us for 1048576 (bound by the reading and marking).
#pragma once
#include "pair_rows.cuh"
#include "router.cuh"

namespace moe {

constexpr int kZeroCluster = 8;
constexpr int kZeroThreads = 1024;
constexpr int kZeroMarks = 32 * 1024;      // bytes of a block: 262,144 rows of a share at once

// Unit: what a row is stored by, a 16-byte word or an element; `units` a row, `stride` apart.
template <class Unit>
__global__ void __launch_bounds__(kZeroThreads) zero_unnamed_kernel(const __grid_constant__ PairRows q, Unit *rows, int64_t stride,
                                                                    int64_t units) {
    __shared__ __align__(16) uint8_t marks[kZeroMarks];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = (int)q.T * q.k, R = (int)q.R;
    const int rank = (int)rtr::cluster_rank(), cluster = (int)blockIdx.x / kZeroCluster, clusters = (int)gridDim.x / kZeroCluster;
    const int lo = (int)((int64_t)R * cluster / clusters), hi = (int)((int64_t)R * (cluster + 1) / clusters);
    const uint32_t own = ptx::smem_u32(marks);
    pdl_wait();
    pdl_trigger();
    for (int base = lo; base < hi; base += min(kZeroCluster * kZeroMarks, hi - base)) {
        const int n = min(kZeroCluster * kZeroMarks, hi - base), mine = (n - rank + kZeroCluster - 1) / kZeroCluster;
        const auto mark = [&](int r) {
            const uint32_t at = (uint32_t)r - (uint32_t)base;           // past n for negative entries too
            if (at < (uint32_t)n)
                asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(rtr::peer_addr(own + at / kZeroCluster, at % kZeroCluster)),
                             "r"(1) : "memory");
        };
        for (int i = tid; i < kZeroMarks / 16; i += kZeroThreads) reinterpret_cast<uint4 *>(marks)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
        rtr::cluster_sync();            // cleared before anyone marks
        if (!q.pair_rows) {             // pair p has row p
            for (int i = rank * kZeroThreads + tid; i < min(n, P - base); i += kZeroCluster * kZeroThreads) mark(base + i);
        } else {
            constexpr int kWords = 4, kStep = kZeroCluster * kZeroThreads;      // 16-byte words in flight a thread
            const int words = (reinterpret_cast<uintptr_t>(q.pair_rows) & 15u) == 0 ? P / 4 : 0, first = rank * kZeroThreads + tid;
            for (int i = first; i < words; i += kWords * kStep) {
                int4 v[kWords];
#pragma unroll
                for (int u = 0; u < kWords; ++u)
                    v[u] = i + u * kStep < words ? __ldg(reinterpret_cast<const int4 *>(q.pair_rows) + i + u * kStep)
                                                 : make_int4(-1, -1, -1, -1);
#pragma unroll
                for (int u = 0; u < kWords; ++u) {
                    mark(v[u].x);
                    mark(v[u].y);
                    mark(v[u].z);
                    mark(v[u].w);
                }
            }
            for (int64_t i = 4 * (int64_t)words + first; i < P; i += kStep) mark(__ldg(q.pair_rows + i));
        }
        __syncwarp();
        rtr::cluster_sync();            // all marked; from here on each block reads its own
        for (int i = 32 * warp; i < mine; i += kZeroThreads) {
            unsigned left = __ballot_sync(0xFFFFFFFFu, i + lane < mine && !marks[i + lane]);
            for (; left; left &= left - 1) {
                Unit *row = rows + (base + (int64_t)kZeroCluster * (i + __ffs(left) - 1) + rank) * stride;
                for (int64_t c = lane; c < units; c += 32) row[c] = Unit{};
            }
        }
        __syncthreads();                // read before they are cleared again
    }
}

}  // namespace moe
