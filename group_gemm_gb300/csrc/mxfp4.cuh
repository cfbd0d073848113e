// mxfp4.cuh -- what the MXFP4 kernels share: the block-scaled 4-bit MMA and the scale blocks.
//
// Number format (OCP Microscaling Formats v1.0, MXFP4): E2M1 elements, two per byte with the lower
// index in the low nibble, one E8M0 scale (value 2^(s-127), 255 = NaN) per 32 consecutive elements
// along the contraction. Both operands are K-major: a row's codes are K/2 contiguous bytes.
//
// A K stage is 128 code bytes (256 elements) of a row, one 128-byte swizzle row: four MMAs of K = 64
// (tcgen05.mma kind::mxf4, scale_vec::2X: two scales per row and MMA). The scales of 128 rows x 4
// consecutive scale blocks (128 elements) form a 512-byte atom, byte 16 (r % 32) + 4 (r / 32) + kblock;
// it occupies 4 tensor-memory columns, replicated over the four lane quarters (lane l of each holds
// bytes 16 l .. 16 l + 15), and the MMA reads the scales of rows 32q .. 32q+31 from column q. One atom serves two
// MMAs: scale-factor id 0 picks the word's bytes 0-1, id 2 its bytes 2-3.
#pragma once

#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace rdot {

// Instruction descriptor for kind::mxf4 (32 bits): [4,6) B scale-factor id, [7,10) A format (1 = E2M1),
// [10,12) B format (1 = E2M1), [17,23) N >> 3, [23] scale type (1 = UE8M0), [27,29) M >> 7, [29,31) A
// scale-factor id, [31] 0: K = 64. Both operands are K-major; D is fp32.
__device__ __forceinline__ constexpr uint32_t idesc_mxf4(int m, int n, uint32_t sf_id) {
    return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(m >> 7) << 27) | (sf_id << 29);
}

template <int CTAS>
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
            : "memory");
}

// group_scan_warp (sched.cuh) with each size loaded once, for up to 32 groups a lane's: its three passes
// over the sizes are three L2 round trips at the start of every CTA (one token top-2 of 8, 4096 -> 14336:
// 15.0 against 15.6 us; 300 rows x 1024 -> 1408, 8 experts: 5.5 against 6.5 us).
__device__ __forceinline__ int mx4_group_scan(const int32_t* __restrict__ group_sizes, int G, int M, int BM, int NT,
                                              int32_t* off, int32_t* tile_prefix) {
    if (G > 32) return group_scan_warp(group_sizes, G, M, BM, NT, off, tile_prefix);
    const int lane = threadIdx.x & 31;
    const int s = lane < G ? __ldg(group_sizes + lane) : 0;
    const int bad = __any_sync(0xffffffffu, s < 0);
    long long end = max(s, 0);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, end, d);
        if (lane >= d) end += v;
    }
    const long long start = min(end - max(s, 0), static_cast<long long>(M));
    const bool over = __any_sync(0xffffffffu, end > M);
    end = min(end, static_cast<long long>(M));
    const int tiles = static_cast<int>((end - start + BM - 1) / BM) * NT;
    int tend = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, tend, d);
        if (lane >= d) tend += v;
    }
    if (lane < G) {
        off[lane] = static_cast<int32_t>(start);
        tile_prefix[lane] = tend - tiles;
    }
    if (lane == G - 1) {
        off[G] = static_cast<int32_t>(end);
        tile_prefix[G] = tend;
    }
    return bad || over ? RDOT_STATUS_BIT_GROUP_SIZES : 0;
}

// mbar_wait (ptx.cuh) that looks at the clock only after MX4_TRIES waits, where mbar_wait reads the global
// timer before its second look (16384 rows x 4096 -> 14336: 304 against 320 us; one token 15.0 against 15.7).
// A caller's wait limit counts from there: a nanosecond still stops every call (8 of 8 at K = 256 to 8192).
constexpr int MX4_TRIES = 32;

__device__ __forceinline__ bool mx4_wait(uint64_t* bar, uint32_t parity, const WaitGuard& g) {
    for (int i = 0; i < MX4_TRIES; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, g);
}

__device__ __forceinline__ bool mx4_wait_warp(uint64_t* bar, uint32_t parity, const WaitGuard& g) {
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = mx4_wait(bar, parity, g) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// A wait by every lane of a warp whose control flow stays uniform: the MMA warps run their loops with all
// lanes and elect one only for the tcgen05 instructions, so that descriptors and addresses stay in uniform
// registers. (In a lane-0 branch each MMA took about 100 clocks to issue, more than it takes to run with
// N = 64; see mxfp4_tc2.cu.)
__device__ __forceinline__ bool mx4_wait_uniform(uint64_t* bar, uint32_t parity, const WaitGuard& g) {
    for (int i = 0; i < MX4_TRIES; ++i)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, g)) != 0;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Eight 32-bit registers of each lane to eight tensor-memory columns of the warp's lane quarter.
__device__ __forceinline__ void tmem_st_32x8(uint32_t taddr, uint4 a, uint4 b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Scale gather of a token or row tile. The rows' scales are plain [M, K/32]: a tile starts at its
// group's first row, so no fixed layout could hold them as atoms. A warp loads a row per lane at a time,
// the scales of MX4_GROUP consecutive K stages (64 bytes), one group ahead of the one in use, and puts
// them into shared memory as atoms, from which the warps that fill tensor memory read 16 bytes a lane.
// Blocks past K read as 0 (their codes are zeros).
constexpr int MX4_GROUP = 8;
constexpr int MX4_GROUP_BYTES = MX4_GROUP * 2 * MX4_ATOM_BYTES;   // atoms of a group: 8 KB

// R rows a lane: first, first + 32, ... of a tile of `rows` rows at row0 (rows past it read as 0). The paths
// by width are kept apart, each with all its loads ahead of their uses: merged into one, every load was
// waited for (65536 rows x 256 -> 1024: 67 against 36 us). Reading single bytes is the slow one: a load a byte,
// one stage in flight (65536 rows x 96 -> 1024: 55 us for 20 us of bytes; see also mxfp4_tc2.cu).
template <int R>
__device__ __forceinline__ void load_scale_group(const Mx4Args& a, int row0, int rows, int first, int ks0,
                                                 uint2 (&v)[R][MX4_GROUP]) {
    const uint8_t* base[R];
    bool live[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        base[r] = a.lhs_scale + (static_cast<long long>(row0) + first + 32 * r) * a.KB + 8 * ks0;
        live[r] = first + 32 * r < rows;
    }
    const int stages = a.KS - ks0;      // left, this group's among them
    const int blocks = a.KB - 8 * ks0;
    if (a.scale_vec == 16) {   // whole pairs of stages, 16 bytes each
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < MX4_GROUP; j += 2) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (live[r] && j < stages) u = __ldg(reinterpret_cast<const uint4*>(base[r]) + (j >> 1));
                v[r][j] = make_uint2(u.x, u.y);
                v[r][j + 1] = make_uint2(u.z, u.w);
            }
    } else if (a.scale_vec == 8) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < MX4_GROUP; ++j) {
                v[r][j] = make_uint2(0u, 0u);
                if (live[r] && j < stages) v[r][j] = __ldg(reinterpret_cast<const uint2*>(base[r]) + j);
            }
    } else if (a.scale_vec == 4) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < MX4_GROUP; ++j) {
                v[r][j] = make_uint2(0u, 0u);
                if (live[r] && 8 * j < blocks) v[r][j].x = __ldg(reinterpret_cast<const uint32_t*>(base[r]) + 2 * j);
                if (live[r] && 8 * j + 4 < blocks) v[r][j].y = __ldg(reinterpret_cast<const uint32_t*>(base[r]) + 2 * j + 1);
            }
    } else {
#pragma unroll
        for (int j = 0; j < MX4_GROUP; ++j) {
            uint32_t b[R][8];   // one stage's bytes of all rows in flight
            if (j < stages) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        b[r][i] = 0u;
                        if (live[r] && 8 * j + i < blocks) b[r][i] = __ldg(base[r] + 8 * j + i);
                    }
#pragma unroll
                for (int r = 0; r < R; ++r)
                    v[r][j] = make_uint2(b[r][0] | b[r][1] << 8 | b[r][2] << 16 | b[r][3] << 24,
                                         b[r][4] | b[r][5] << 8 | b[r][6] << 16 | b[r][7] << 24);
            }
        }
    }
}

// Row r of the tile (0 .. 127) into the group's atoms, `stages` of them.
__device__ __forceinline__ void put_scale_group(uint8_t* atoms, int r, const uint2 (&v)[MX4_GROUP], int stages) {
    uint8_t* p = atoms + 16 * (r & 31) + 4 * (r >> 5);
#pragma unroll
    for (int j = 0; j < MX4_GROUP; ++j) {
        if (j >= stages) break;
        *reinterpret_cast<uint32_t*>(p + 2 * j * MX4_ATOM_BYTES) = v[j].x;
        *reinterpret_cast<uint32_t*>(p + (2 * j + 1) * MX4_ATOM_BYTES) = v[j].y;
    }
}

}  // namespace rdot
