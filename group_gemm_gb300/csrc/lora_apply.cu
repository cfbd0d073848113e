// lora_apply.cu -- low-rank adapters beside a projection: out = base + scale[g] (x first[g]^T) second[g]. The form for
// few rows (lora_tall.cu: many).
//
// For a tile of 16 rows of one group the kernel forms t = scale[g] x first[g]^T (contraction over the K columns of
// x) and then base + t second[g], in one launch and without t's round trip through memory. Both weights lie
// [G, r, width], their long axis contiguous, so the forward (first = down, second = up) and the gradient of the
// input (first = up, second = down) are the same kernel. With a row or two to an adapter it streams weights:
// HBM's latency and rate bound it, not the MMAs (mma.sync, 16 x 8 x 16, half of a tile's rows empty or more).
//
// A cluster of C blocks takes a tile: each contracts its share of the columns of x, the fp32 partial sums are
// added through distributed shared memory in a fixed order, and each then writes its share of the output's
// columns. So a few rows still spread over many SMs, and results do not depend on timing. 64 rows over 256
// adapters, 4096 -> 14336, rank 16: 18.3 us with C = 8, 72 us with C = 1. With very few tiles D clusters take one:
// each forms all of t, and writes a D-th of the columns (1 row, 4096 -> 14336, rank 64: D = 1 23.6, D = 8 14.3 us).
// The ring is as deep as it can be with the blocks that have to share an SM: a second round of blocks costs more than
// the loads a longer ring has in flight (the 64 rows above: six stages, three blocks on an SM 24.8, five 18.3, four
// 20.2; 128 rows of 128 adapters: 25.4, 25.5 and 20.8; rank 128, 64 rows of 16: one block with five stages 38, two with
// three 27). Stages of 128 columns: of 64 a fifth slower.
//
// t keeps fp32 accuracy into the second product: it enters as two bf16 terms, t = hi + lo with lo the rounded
// rest (relative error 2^-16, below the output's own rounding of 2^-8), two MMAs in place of one. hi is also
// what is returned as t, the operand of the weight gradient.
#include <cuda_bf16.h>

#include "kernels.h"
#include "lora.cuh"
#include "pdl.cuh"

namespace rdot {

namespace {

template <int RP_, int STAGES_, int THREADS_ = LORA_THREADS>
struct ApplyCfg {
    static constexpr int R = LORA_FEW_ROWS;            // rows of a tile: an MMA's
    static constexpr int RP = RP_;                     // rank, rounded up
    static constexpr int THREADS = THREADS_;           // rank 64: 256, 128 rows of 128 adapters, 4096 -> 14336, 57 us against 66 for 128
    static constexpr int WARPS = THREADS / 32;         // along the columns in the second product
    static constexpr int WK = 4;                       // along the columns in the first, WARPS / WK along the ranks
    static constexpr int BK = RP <= 64 ? 128 : 64;     // columns per stage
    static constexpr int PITCH = 2 * BK + 16;          // bytes: 16 off a multiple of 128, so ldmatrix has no conflicts
    static constexpr int SLOT = (R + RP) * PITCH;      // x or base rows, then weight rows
    static constexpr int STAGES = STAGES_;
    // The MMAs cut their sums at each step of 16 columns, always towards 0: a warp takes 512 of its columns at most before it
    // adds its sums, rounded, to those in shared memory. (3000 rows of 32 groups, 14336 -> 512, rank 32: 47.4 us, 45.7 without.)
    static constexpr int STRETCH = 512 / (BK / WK);    // stages
    static constexpr int PP = RP + 4;                  // pitch of the partial sums (fp32)
    static constexpr int TP = RP + 8;                  // pitch of hi and lo (bf16)
    static constexpr int PART = WK * R * PP * 4;
    static constexpr int SMEM = STAGES * SLOT + PART + 2 * R * TP * 2;
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS) lora_apply_kernel(LoraArgs a, int D) {
    constexpr int R = Cfg::R, RP = Cfg::RP, WK = Cfg::WK, BK = Cfg::BK, PITCH = Cfg::PITCH;
    constexpr int THREADS = Cfg::THREADS, WARPS = Cfg::WARPS, RW = RP / (WARPS / WK);   // RW: ranks of a warp
    constexpr int S = Cfg::STAGES, PP = Cfg::PP, TP = Cfg::TP;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int row_of[R];   // each tile row's row of x, base and out; -1 for none
    float* part = reinterpret_cast<float*>(smem + S * Cfg::SLOT);
    uint16_t* thi = reinterpret_cast<uint16_t*>(smem + S * Cfg::SLOT + Cfg::PART);
    uint16_t* tlo = thi + R * TP;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wk = warp % WK, r0 = warp / WK * RW;
    const int C = static_cast<int>(cluster_ctas()), rank = static_cast<int>(cluster_ctarank());

    grid_dependency_enter();
    const LoraTile tile = lora_find_tile<R, THREADS>(a.group_sizes, a.G, a.M, static_cast<int>(blockIdx.x) / (C * D));
    if (tile.rows == 0) return;   // the whole cluster
    const int part_n = static_cast<int>(blockIdx.x) / C % D;
    const bool live = tile.g < a.G;
    lora_tile_rows<R, THREADS>(row_of, tile, a.order, a.M);
    __syncthreads();

    const int nk = live ? (a.K + BK - 1) / BK : 0, nn = (a.N + BK - 1) / BK;
    // this block's stages: chunks rank, rank + C, ... of x's width, so that the cluster reads neighbouring columns at a
    // time; of the output's the same over the tile's D clusters
    const int rank_n = part_n * C + rank, step_n = C * D;
    const int first_stages = nk > rank ? (nk - rank + C - 1) / C : 0;
    int second_stages = nn > rank_n ? (nn - rank_n + step_n - 1) / step_n : 0;
    if (!live && a.base == a.out) second_stages = 0;   // rows without an adapter, in place: they stay as they are
    const int stages = first_stages + second_stages;
    const uint32_t ring = smem_u32(smem);

    // stage i of this block into its slot: 16-byte pieces, zeros outside the tensors
    const auto load = [&](int i) {
        if (i < stages) {
            constexpr int V = BK / 8;   // pieces of a row
            const bool one = i < first_stages;
            const int width = one ? a.K : a.N;
            const int c0 = (one ? i * C + rank : (i - first_stages) * step_n + rank_n) * BK + (tid % V) * 8;
            const uint16_t* rows = static_cast<const uint16_t*>(one ? a.x : a.base);
            const uint16_t* weight = static_cast<const uint16_t*>(one ? a.first : a.second);
            const bool in = c0 < width;
            const uint32_t dst = ring + (i % S) * Cfg::SLOT + (tid % V) * 16;
            if (rows) {
#pragma unroll
                for (int r = tid / V; r < R; r += THREADS / V) {
                    const int row = row_of[r];
                    const bool ok = in && row >= 0;
                    cp_async16(dst + r * PITCH, rows + (ok ? static_cast<long long>(row) * width + c0 : 0), ok);
                }
            }
            if (live) {
#pragma unroll
                for (int r = tid / V; r < RP; r += THREADS / V) {
                    const bool ok = in && r < a.rank;
                    cp_async16(dst + (R + r) * PITCH,
                               weight + (ok ? (static_cast<long long>(tile.g) * a.rank + r) * width + c0 : 0), ok);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load(i);

    int i = 0;
    if (live) {
        float acc[RW / 8][4] = {};
        float* const mine = part + wk * R * PP + (lane >> 2) * PP + r0 + 2 * (lane & 3);
        // this lane's sums into its place of `part`, or onto what that holds
        const auto put = [&](bool first) {
#pragma unroll
            for (int j = 0; j < RW / 8; ++j) {
                float2 *p = reinterpret_cast<float2*>(mine + 8 * j), *q = reinterpret_cast<float2*>(mine + 8 * PP + 8 * j);
                if (!first) {
                    const float2 u = *p, v = *q;
                    acc[j][0] += u.x;
                    acc[j][1] += u.y;
                    acc[j][2] += v.x;
                    acc[j][3] += v.y;
                }
                *p = make_float2(acc[j][0], acc[j][1]);
                *q = make_float2(acc[j][2], acc[j][3]);
            }
        };
        for (int stop = min(first_stages, Cfg::STRETCH);; ++i) {   // the end of the stretch
            if (i == stop) {
                put(i <= Cfg::STRETCH);
                if (i == first_stages) break;
                stop = min(first_stages, i + Cfg::STRETCH);
#pragma unroll
                for (int j = 0; j < RW / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
            }
            cp_async_wait<S - 2>();
            __syncthreads();
            load(i + S - 1);
            const uint32_t slot = ring + (i % S) * Cfg::SLOT;
            const uint32_t ax = slot + (lane & 15) * PITCH + (lane >> 4) * 16;
            const uint32_t bx = slot + (R + r0 + (lane & 7) + ((lane >> 4) << 3)) * PITCH + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int kk = wk; kk < BK / 16; kk += WK) {
                uint32_t fa[4];
                ldmatrix_x4(fa, ax + kk * 32);
#pragma unroll
                for (int j = 0; j < RW / 16; ++j) {
                    uint32_t fb[4];
                    ldmatrix_x4(fb, bx + j * 16 * PITCH + kk * 32);
                    mma_16816(acc[2 * j], fa, fb[0], fb[1]);
                    mma_16816(acc[2 * j + 1], fa, fb[2], fb[3]);
                }
            }
        }
        // partial sums of the warps, then of the cluster's blocks
        __syncthreads();
        if (C > 1) {
            for (int e = tid; e < R * RP / 4; e += THREADS) {
                float4* p = reinterpret_cast<float4*>(part + (e / (RP / 4)) * PP + 4 * (e % (RP / 4)));
                float4 s = *p;
#pragma unroll
                for (int w = 1; w < WK; ++w) {
                    const float4 v = p[w * R * PP / 4];
                    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
                }
                *p = s;
            }
            cluster_sync();
        }
        const float scale = a.scale ? __ldg(a.scale + tile.g) : 1.f;
        for (int e = tid; e < R * RP / 4; e += THREADS) {
            const int r = e / (RP / 4), c = 4 * (e % (RP / 4));
            float* p = part + r * PP + c;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (C > 1) {
                const uint32_t addr = smem_u32(p);
#pragma unroll 4
                for (int q = 0; q < C; ++q) {
                    const float4 v = ld_shared_cluster_f4(mapa_shared(addr, q));
                    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
                }
            } else {
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(p + w * R * PP);
                    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
                }
            }
            // ranks past the adapter's are 0 whatever x holds (there x times the zero weights may be NaN)
            const bool in = c < a.rank;
            const float v[4] = {in ? s.x * scale : 0.f, in ? s.y * scale : 0.f, in ? s.z * scale : 0.f, in ? s.w * scale : 0.f};
            uint2 hi, lo;
            split_bf16x2(v[0], v[1], hi.x, lo.x);
            split_bf16x2(v[2], v[3], hi.y, lo.y);
            *reinterpret_cast<uint2*>(thi + r * TP + c) = hi;
            *reinterpret_cast<uint2*>(tlo + r * TP + c) = lo;
            if (rank_n == 0 && a.t && r < tile.rows && in)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.t) + static_cast<long long>(tile.p0 + r) * a.rank + c) = hi;
        }
        if (C > 1) {
            __syncwarp();
            cluster_arrive();   // this block has read the others' sums
        }
        __syncthreads();
    } else if (rank_n == 0 && a.t) {
        for (long long e = tid; e < static_cast<long long>(tile.rows) * a.rank / 4; e += THREADS)
            reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.t) + static_cast<long long>(tile.p0) * a.rank)[e] = make_uint2(0u, 0u);
    }

    // t as MMA fragments: held in registers while they are few
    constexpr bool KEEP = RP <= 32;
    const uint32_t ahi = smem_u32(thi) + (lane & 15) * TP * 2 + (lane >> 4) * 16, alo = ahi + R * TP * 2;
    uint32_t th[KEEP ? RP / 16 : 1][4], tl[KEEP ? RP / 16 : 1][4];
    if (KEEP && live) {
#pragma unroll
        for (int kk = 0; kk < RP / 16; ++kk) {
            ldmatrix_x4(th[kk], ahi + kk * 32);
            ldmatrix_x4(tl[kk], alo + kk * 32);
        }
    }
    for (; i < stages; ++i) {
        cp_async_wait<S - 2>();
        __syncthreads();
        load(i + S - 1);
        uint8_t* slot = smem + (i % S) * Cfg::SLOT;
        const uint32_t bx = smem_u32(slot) + (R + (lane & 15)) * PITCH + (lane >> 4) * 16;
        constexpr int COLS = BK / WARPS;   // this warp's columns of the stage
#pragma unroll
        for (int n = 0; n < COLS; n += 16) {
            if (!live && a.base) continue;   // a copy
            // the sums start from base and go back to its place in the stage; a 32-bit word holds two columns of a lane
            uint32_t* const p = reinterpret_cast<uint32_t*>(slot + (lane >> 2) * PITCH + (warp * COLS + n + 2 * (lane & 3)) * 2);
            float acc[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t b = a.base ? p[half * 2 * PITCH + 4 * h] : 0u;
                    acc[h][2 * half] = __uint_as_float(b << 16);
                    acc[h][2 * half + 1] = __uint_as_float(b & 0xffff0000u);
                }
            if (live) {
#pragma unroll
                for (int kk = 0; kk < RP / 16; ++kk) {
                    uint32_t fb[4];
                    ldmatrix_x4_trans(fb, bx + kk * 16 * PITCH + (warp * COLS + n) * 2);
                    uint32_t fh[4], fl[4];
                    if (KEEP) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            fh[j] = th[KEEP ? kk : 0][j];
                            fl[j] = tl[KEEP ? kk : 0][j];
                        }
                    } else {
                        ldmatrix_x4(fh, ahi + kk * 32);
                        ldmatrix_x4(fl, alo + kk * 32);
                    }
                    mma_16816(acc[0], fh, fb[0], fb[1]);
                    mma_16816(acc[1], fh, fb[2], fb[3]);
                    mma_16816(acc[0], fl, fb[0], fb[1]);
                    mma_16816(acc[1], fl, fb[2], fb[3]);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    p[half * 2 * PITCH + 4 * h] = pack_bf16x2(acc[h][2 * half], acc[h][2 * half + 1]);
        }
        __syncwarp();
        // the warp's rows and columns of the stage, 16 bytes a lane
        constexpr int V = COLS / 8;
        const int c0 = ((i - first_stages) * step_n + rank_n) * BK + warp * COLS + (lane % V) * 8;
#pragma unroll
        for (int r = lane / V; r < 16; r += 32 / V) {
            const int row = row_of[r];
            if (row >= 0 && c0 < a.N)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + static_cast<long long>(row) * a.N + c0) =
                    *reinterpret_cast<const uint4*>(slot + r * PITCH + (warp * COLS + (lane % V) * 8) * 2);
        }
    }
    if (live && C > 1) cluster_wait();   // the others have read this block's sums
}

template <class Cfg>
cudaError_t launch_cfg(const LoraArgs& a, long long tiles, int C, int D, cudaStream_t stream) {
    auto kern = lora_apply_kernel<Cfg>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(tiles * C * D)), dim3(Cfg::THREADS), C, Cfg::SMEM, stream, a, D);
}

}  // namespace

cudaError_t launch_lora_apply(const LoraArgs& a, int C, int D, int blocks, cudaStream_t stream) {
    constexpr int R = LORA_FEW_ROWS;
    // a tile more for each group that ends inside one, one more for the rows of no group
    const long long tiles = (static_cast<long long>(a.M) + R - 1) / R + (a.G < a.M ? a.G : a.M) + 1;
    // the deepest ring with which that many blocks fit an SM's shared memory
    if (a.rank <= 16)
        return blocks <= 3 ? launch_cfg<ApplyCfg<16, 6>>(a, tiles, C, D, stream)
             : blocks <= 4 ? launch_cfg<ApplyCfg<16, 5>>(a, tiles, C, D, stream)
                           : launch_cfg<ApplyCfg<16, 4>>(a, tiles, C, D, stream);
    if (a.rank <= 32)
        return blocks <= 2 ? launch_cfg<ApplyCfg<32, 5>>(a, tiles, C, D, stream)
                           : launch_cfg<ApplyCfg<32, 3>>(a, tiles, C, D, stream);
    if (a.rank <= 64) return launch_cfg<ApplyCfg<64, 4, 256>>(a, tiles, C, D, stream);
    return launch_cfg<ApplyCfg<128, 3>>(a, tiles, C, D, stream);
}

}  // namespace rdot
