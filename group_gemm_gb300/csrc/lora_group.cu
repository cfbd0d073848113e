// lora_group.cu -- the rows of a batch sorted by adapter, once for every projection that carries adapters.
//
// order is the stable sort of the rows by id, rows whose id lies outside [0, G) last; group_sizes counts each
// id's rows. A counting sort in one launch: a cluster of blocks, each warp of which owns a run of consecutive
// rows. Each warp counts its ids in a table of its own in shared memory; per id, the counts of the warps and
// blocks before it (the blocks' totals read through distributed shared memory) and of all lower ids give the
// warp's first place; then the warp places its rows 32 at a time, equal ids by their lane. No atomics
// between warps, so the order is the stable sort's. A few microseconds of latency are its bound.
#include "kernels.h"
#include "lora.cuh"
#include "pdl.cuh"

namespace rdot {

namespace {

constexpr int GROUP_THREADS = 1024;
constexpr int GROUP_WARPS = GROUP_THREADS / 32;

// shared memory: counts [32 warps][G + 1], then the block's totals [G + 1]
__global__ void __launch_bounds__(GROUP_THREADS) lora_group_kernel(const int32_t* __restrict__ ids, int M, int G,
                                                                   int32_t* __restrict__ group_sizes,
                                                                   int32_t* __restrict__ order) {
    extern __shared__ int32_t counts[];
    __shared__ int32_t warp_sum[GROUP_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster_ctas()), rank = static_cast<int>(cluster_ctarank());
    const int B = G + 1;   // the last bin: rows without an adapter
    int32_t* totals = counts + GROUP_WARPS * B;
    int32_t* mine = counts + warp * B;

    grid_dependency_enter();
    // units of 32 rows, `per` to a warp: the first `tables` warps of a block have some (64 rows of 256 adapters with all 32
    // warps' tables cleared and added up: 5.5 us, with two 4.7)
    const long long units = (static_cast<long long>(M) + 31) / 32;
    const int shift = 5 + 31 - __clz(C);   // log2 of the warps; C is a power of two
    const long long per = (units + (1LL << shift) - 1) >> shift;
    const long long w = static_cast<long long>(rank) * GROUP_WARPS + warp;
    const long long u0 = min(units, w * per), u1 = min(units, u0 + per);
    const int tables = static_cast<int>(min(units, static_cast<long long>(GROUP_WARPS)));
    const auto bin = [&](long long u) -> int {   // -1 past the end
        const long long r = 32 * u + lane;
        if (r >= M) return -1;
        const int id = __ldg(ids + r);
        return id >= 0 && id < G ? id : G;
    };
    if (warp < tables)
        for (int b = lane; b < B; b += 32) mine[b] = 0;
    __syncwarp();
    constexpr int U = 8;   // loads in flight
    for (long long u = u0; u < u1; u += U) {
        int id[U];
#pragma unroll
        for (int j = 0; j < U; ++j) id[j] = u + j < u1 ? bin(u + j) : -1;
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (id[j] >= 0) atomicAdd(mine + id[j], 1);   // this warp's table
    }
    __syncthreads();
    // per bin, the warps' counts become the counts before each warp of this block
    for (int b = tid; b < B; b += GROUP_THREADS) {
        int32_t run = 0;
#pragma unroll 8
        for (int v = 0; v < tables; ++v) {
            const int32_t c = counts[v * B + b];
            counts[v * B + b] = run;
            run += c;
        }
        totals[b] = run;
    }
    cluster_sync();
    // a thread holds a bin, thread 0 bin 1024 as well where there are that many
    int32_t before = 0, all = 0;
    if (tid < B)
        for (int q = 0; q < C; ++q) {
            int32_t v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(totals + tid), q)) : "memory");
            before += q < rank ? v : 0;
            all += v;
        }
    int32_t extra = 0;   // bin 1024's rows in the blocks before this one
    if (B > GROUP_THREADS && tid == 0)
        for (int q = 0; q < rank; ++q) {
            int32_t v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(totals + GROUP_THREADS), q)) : "memory");
            extra += v;
        }
    if (rank == 0 && tid < G) group_sizes[tid] = all;
    int32_t incl = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    cluster_sync();   // also: the totals have been read, they may be replaced
    int32_t base = 0, sum = 0;
    for (int v = 0; v < GROUP_WARPS; ++v) {
        base += v < warp ? warp_sum[v] : 0;
        sum += warp_sum[v];
    }
    if (tid < B) totals[tid] = base + incl - all + before;   // the block's first place of each bin
    if (B > GROUP_THREADS && tid == 0) totals[GROUP_THREADS] = sum + extra;
    __syncthreads();
    if (warp < tables)
        for (int b = lane; b < B; b += 32) mine[b] += totals[b];
    __syncwarp();
    for (long long u = u0; u < u1; u += U) {
        int id[U];
#pragma unroll
        for (int j = 0; j < U; ++j) id[j] = u + j < u1 ? bin(u + j) : -1;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (u + j >= u1) break;
            const unsigned same = __match_any_sync(0xffffffffu, id[j]);
            const int place = id[j] >= 0 ? mine[id[j]] + __popc(same & ((1u << lane) - 1)) : 0;
            __syncwarp();
            if (id[j] >= 0) {
                order[place] = static_cast<int32_t>(32 * (u + j) + lane);
                if (lane == __ffs(same) - 1) mine[id[j]] += __popc(same);
            }
            __syncwarp();
        }
    }
}

}  // namespace

cudaError_t launch_lora_group(const int32_t* ids, int M, int G, int32_t* group_sizes, int32_t* order,
                              cudaStream_t stream) {
    const auto bytes = [](int groups) { return (GROUP_WARPS + 1) * (groups + 1) * static_cast<int>(sizeof(int32_t)); };
    const size_t shm = bytes(G);
    // one limit for every call: another thread may launch with other groups in between
    const cudaError_t e = cudaFuncSetAttribute(lora_group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(RDOT_MAX_GROUPS));
    if (e != cudaSuccess) return e;
    // (16384 rows of 64 adapters: 17.0, 10.6, 7.9 and 7.0 us with 1, 2, 4 and 8 blocks; 64 rows of 256: 4.7 with one)
    const int C = M <= 1024 ? 1 : M <= 4096 ? 4 : 8;
    return launch_pdl_cluster(lora_group_kernel, dim3(C), dim3(GROUP_THREADS), C, shm, stream, ids, M, G, group_sizes, order);
}

}  // namespace rdot
