// lora.cuh -- what the low-rank adapter kernels share: asynchronous row copies, the 16 x 8 x 16 bf16 MMA on
// register fragments, the scan that finds a block's rows, and launches in clusters.
#pragma once

#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

namespace rdot {

// 16 bytes global -> shared, or 16 zero bytes where `live` is false (src is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// An arrival on `bar`, one of those it was initialised for, once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8 x 8 matrices of 16-bit elements; lanes 8i .. 8i+7 give the row addresses of matrix i.
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// d [16 x 8] += a [16 x 16] b [16 x 8], fp32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}

__device__ __forceinline__ float4 ld_shared_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_cluster_u4(uint32_t addr, const uint4& v) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// tmem_ld_32x32b_x32 for 8 columns.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// 16 columns; and back.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Whether the phase has completed, without waiting; the same in every lane.
__device__ __forceinline__ bool mbar_test_uniform(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, ok);
}

// Sum over a block of THREADS threads of `v`, and of the threads before this one. `part`: shared, an entry a warp;
// the caller synchronises between uses.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += u;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        before += w < warp ? part[w] : 0;
        all += part[w];
    }
    *total = all;
    return before + incl - v;
}

constexpr int LORA_THREADS = 128;
constexpr int LORA_SIZES = 8;   // sizes a thread holds: 1024 groups over 128 threads

// A block's tile: the rows of group g (G: rows of no group), sorted positions p0 .. p0 + rows - 1.
struct LoraTile {
    int g;
    int p0;
    int rows;
};

// Tile `w` of the rows cut into tiles of at most R rows that do not cross a group's end: the groups in
// order, then the rows past the last one. rows = 0 past the last tile. A negative size counts as 0, ends are
// clamped to M. Every thread gets the tile; all sizes are loaded at once, one pass.
template <int R, int THREADS>
__device__ __forceinline__ LoraTile lora_find_tile(const int32_t* __restrict__ sizes, int G, int M, int w) {
    static_assert(THREADS * LORA_SIZES >= RDOT_MAX_GROUPS, "every size has a thread");
    __shared__ long long part[2][THREADS / 32];
    __shared__ LoraTile found;
    const int per = (G + THREADS - 1) / THREADS;   // consecutive groups per thread, <= LORA_SIZES
    const int g0 = threadIdx.x * per;
    int s[LORA_SIZES];
    long long sum = 0;
#pragma unroll
    for (int i = 0; i < LORA_SIZES; ++i) s[i] = (i < per && g0 + i < G) ? max(__ldg(sizes + g0 + i), 0) : 0;
#pragma unroll
    for (int i = 0; i < LORA_SIZES; ++i) sum += s[i];
    if (threadIdx.x == 0) found = LoraTile{G, 0, 0};
    long long total, tiles_total;
    const long long first = block_scan<THREADS>(sum, part[0], &total);
    long long at = first, tiles = 0;
#pragma unroll
    for (int i = 0; i < LORA_SIZES; ++i) {
        const long long b = min(at, static_cast<long long>(M)), e = min(at + s[i], static_cast<long long>(M));
        tiles += (e - b + R - 1) / R;
        at += s[i];
    }
    long long t = block_scan<THREADS>(tiles, part[1], &tiles_total);
    if (w >= t && w < t + tiles) {
        at = first;
#pragma unroll
        for (int i = 0; i < LORA_SIZES; ++i) {
            const int b = static_cast<int>(min(at, static_cast<long long>(M)));
            const int e = static_cast<int>(min(at + s[i], static_cast<long long>(M)));
            const int n = static_cast<int>((static_cast<long long>(e) - b + R - 1) / R);
            if (w >= t && w < t + n) {
                const int p0 = b + static_cast<int>(w - t) * R;
                found = LoraTile{g0 + i, p0, min(R, e - p0)};
            }
            t += n;
            at += s[i];
        }
    }
    if (threadIdx.x == 0 && w >= tiles_total) {
        const long long p0 = min(total, static_cast<long long>(M)) + (w - tiles_total) * R;
        if (p0 < M) found = LoraTile{G, static_cast<int>(p0), static_cast<int>(min(static_cast<long long>(R), M - p0))};
    }
    __syncthreads();
    return found;
}

// Row numbers of a tile's sorted positions into shared memory, -1 for none (past the tile, or an entry of
// `order` outside [0, M)). The caller synchronises.
template <int R, int THREADS>
__device__ __forceinline__ void lora_tile_rows(int* row_of, const LoraTile& tile, const int32_t* __restrict__ order, int M) {
    for (int i = threadIdx.x; i < R; i += THREADS) {
        int row = -1;
        if (i < tile.rows) {
            row = order ? __ldg(order + tile.p0 + i) : tile.p0 + i;
            if (row < 0 || row >= M) row = -1;
        }
        row_of[i] = row;
    }
}

// bf16 of a value and of what the rounding left, so that hi + lo has a relative error of 2^-16. Of an infinity or
// NaN, hi alone. (lo may be 0 or of the other sign, so an infinite weight may give NaN for an infinity. Cutting hi
// would leave lo of hi's sign and the product right, for twice the error; looking for such results in each stage took 3
// to 9 % of a decode batch's time.)
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(a, b);
    const float fa = __uint_as_float(hi << 16), fb = __uint_as_float(hi & 0xffff0000u);
    lo = pack_bf16x2(isfinite(fa) ? a - fa : 0.f, isfinite(fb) ? b - fb : 0.f);
}

// launch_pdl (pdl.cuh) with clusters of `cluster` blocks along x, chosen at the launch.
//
// The library's other kernels with tensor memory take it before the wait on the kernel before and signal at once: their
// shared memory leaves no room on the SM for another such kernel. Of lora_tall.cu two blocks share an SM, so it and
// lora_grad.cu take theirs only after the wait, and signal after that: no block holds tensor memory while it waits for a
// grid one of whose blocks is still to get its own.
template <typename... Params, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(Params...), dim3 grid, dim3 block, int cluster, size_t shm,
                               cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = shm;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

}  // namespace rdot
