// mxfp4_skinny.cu -- MXFP4 ragged-dot forward for a few rows per group (decode), operands swapped.
//
// out[i, :] = A[i, :] B[g(i)] with A, B in MXFP4 (mxfp4.cuh), fp32 accumulation, bf16 out, computed as
// out_g^T = B_g A_g^T: 128 weight columns on the MMA's M, up to 64 token rows on its N. What bounds it
// is streaming the routed experts' codes and scales (17/32 byte per weight) from HBM; with few experts,
// how evenly the SMs share them and what a CTA's start and end cost. A work item is a 128-column atom
// of a group for one token tile. Every CTA takes the same number of whole items; the items that are
// left over are cut into halves or quarters (64 or 32 columns) where that many parts still fit the
// CTAs, so the last round costs half or a quarter of an item. A part loads only its columns' rows, at
// their natural place in the stage, and the MMA's other rows are not read out.
//
// Warp 0 streams the codes (one TMA box a stage: with 32-row boxes alone issuing took longer than the
// bytes), warp 7 the token codes and weight scales, warp 6 gathers the token rows' scale bytes into
// atoms a group of stages ahead. Warps 8..11 wait for all of a stage's data, write its scales to their
// tensor-memory lane quarter and tell warp 1, which issues the MMAs and waits for nothing else: copies
// by tcgen05.cp would run in order with the MMAs, as long as them. Warps 2..5 read out one 32-column
// quarter each.
//
// Measured: one token top-2 of 8, 4096 -> 14336: 15.1 us, of which a launch with one stage takes 4.9 (62 MB at
// 6.1 TB/s in the rest; the pair kernel 19.9 us); 64 tokens top-8 of 256 (143 experts routed), 7168 -> 4096:
// 314-321 us by GPU, 7.0-7.1 TB/s of codes and scales. The ring's depth does not matter above five stages for one token;
// 64 tokens take 2 % longer with five than with eight.
#include <cuda_bf16.h>

#include "drain.cuh"
#include "kernels.h"
#include "mxfp4.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "sched.cuh"

namespace rdot {

namespace {

constexpr int THREADS = 384;
constexpr int SCALE_WARP = 8;   // the first of four
constexpr int Q_BYTES = 32 * MX4_STAGE_BYTES;   // one quarter's codes of a stage: 4 KB
constexpr int W_BYTES = 4 * Q_BYTES;
constexpr int X_BOX = 16 * MX4_STAGE_BYTES;     // 16 token rows: 2 KB
constexpr int SF_BYTES = 2 * MX4_ATOM_BYTES;    // a stage's two scale atoms
constexpr int SFX_BYTES = 2 * MX4_GROUP_BYTES;  // the token rows' scale atoms, two groups of stages
constexpr int MISC_BYTES = 16;
constexpr int SF_COLS = 16;                     // per stage: two weight atoms, two token atoms
constexpr int TMEM_COLS = 256;

constexpr int TT = MX4_SKINNY_ROWS;             // token rows per tile (64)
constexpr int STAGES = 8;
constexpr int X_BYTES = TT * MX4_STAGE_BYTES;
constexpr int STAGE_BYTES = W_BYTES + X_BYTES + SF_BYTES;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
// full, xfull, sfull, empty; afull[2], aempty[2], tfull[2], tempty[2], drain
constexpr int BAR_BYTES = (4 * STAGES + 10) / 2 * 16;
constexpr int TMEM_SF_BASE = 2 * TT;            // after the two accumulators
static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms stay 1 KB aligned");
static_assert(TMEM_SF_BASE + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");

size_t smem_bytes(int G) {
    return 1024 + RING_BYTES + SFX_BYTES + BAR_BYTES + MISC_BYTES + sizeof(int32_t) * 2 * (G + 1);
}

__device__ __forceinline__ void tmem_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// A tile: quarters [q0, q1) of 128-column atom nb, for one token tile of a group.
struct SkinnyTile {
    int g, row0, rows, nb, q0, q1;
};

// The CTA's share of `items`: `whole` whole items (blockIdx.x + i gridDim.x), then, if `part` >= 0, quarters
// [q0, q0 + width) of item `part`.
struct SkinnyShare {
    int whole, part, q0, width;
};

__device__ __forceinline__ SkinnyShare skinny_share(int items) {
    const int grid = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
    SkinnyShare s;
    s.whole = items / grid;
    const int left = items - s.whole * grid;          // < grid
    s.width = 4 * left <= grid ? 1 : 2 * left <= grid ? 2 : 4;
    const int parts = 4 / s.width;
    s.part = b < left * parts ? s.whole * grid + b / parts : -1;
    s.q0 = s.width * (b % parts);
    return s;
}

// Tile i of the share, 0 .. whole (the last one only if part >= 0; it may lie past N: then q1 <= q0).
__device__ __forceinline__ SkinnyTile skinny_tile(int i, const SkinnyShare& sh, const Mx4Args& a, const int32_t* tprefix,
                                                  const int32_t* off) {
    const bool whole = i < sh.whole;
    const int item = whole ? static_cast<int>(blockIdx.x) + i * static_cast<int>(gridDim.x) : sh.part;
    const Tile t = decode_tile(item, tprefix, off, a.G, TT, a.NB, true);
    SkinnyTile s;
    s.g = t.g;
    s.row0 = t.row0;
    s.rows = t.rows;
    s.nb = t.nt;
    s.q0 = whole ? 0 : sh.q0;
    s.q1 = min(s.q0 + (whole ? 4 : sh.width), (a.N - 128 * t.nt + 31) / 32);
    return s;
}

__global__ void __launch_bounds__(THREADS, 1)
    mxfp4_skinny_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w128,
                        const __grid_constant__ CUtensorMap tmap_w64, const __grid_constant__ CUtensorMap tmap_w32,
                        Mx4Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sfx_buf = smem + RING_BYTES;
    uint8_t* bars = sfx_buf + SFX_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(bars);   // a stage's weight codes have landed
    uint64_t* xfull = full + STAGES;                      // its token codes and weight scales
    uint64_t* sfull = xfull + STAGES;                     // all of these, and its scales are in tensor memory
    uint64_t* empty = sfull + STAGES;
    uint64_t* afull = empty + STAGES;                     // the token rows' scales of a group of stages
    uint64_t* aempty = afull + 2;
    uint64_t* tfull = aempty + 2;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
    int32_t* off = reinterpret_cast<int32_t*>(bars + BAR_BYTES + MISC_BYTES);
    int32_t* tprefix = off + a.G + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&xfull[s], 1);
            mbar_init(&sfull[s], 4);   // the scale warps
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], 4);
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 128);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmap_x);
        tma_prefetch_desc(&tmap_w128);
        tma_prefetch_desc(&tmap_w64);
        tma_prefetch_desc(&tmap_w32);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, TMEM_COLS);
        tmem_relinquish();
    }
    grid_dependency_enter();   // group sizes and the token codes come from earlier kernels
    if (warp == 2) {
        const int bad = mx4_group_scan(a.group_sizes, a.G, a.M, TT, a.NB, off, tprefix);
        if (bad && lane == 0 && blockIdx.x == 0 && a.status) atomicOr(a.status, bad);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = *tmem_holder;
    const SkinnyShare sh = skinny_share(tprefix[a.G]);
    const int tiles = sh.whole + (sh.part >= 0 ? 1 : 0);
    const WaitGuard guard{abort_flag, a.status, a.timeout_ns};

    if (warp == 0) {
        // ------------------------------------------------------------------ weight codes
        const bool elected = elect_one();
        uint32_t stage = 0, phase = 0, issued_mask = 0, issued_phase = 0;
        bool ok = true;
        for (int i = 0; i < tiles && ok; ++i) {
            const SkinnyTile t = skinny_tile(i, sh, a, tprefix, off);
            const CUtensorMap* map = i < sh.whole || sh.width == 4 ? &tmap_w128 : sh.width == 2 ? &tmap_w64 : &tmap_w32;
            const int rows = i < sh.whole ? 128 : 32 * sh.width;
            for (int ks = 0; ks < a.KS && t.q0 < t.q1; ++ks) {
                ok = mx4_wait_uniform(&empty[stage], phase ^ 1, guard);
                if (!ok) break;
                if (elected) {
                    mbar_arrive_expect_tx(&full[stage], rows * MX4_STAGE_BYTES);
                    // rows past N and bytes past K arrive as zeros
                    tma_load_3d(smem + stage * STAGE_BYTES + t.q0 * Q_BYTES, map, &full[stage], ks * MX4_STAGE_BYTES,
                                t.nb * 128 + 32 * t.q0, t.g);
                }
                __syncwarp();
                issued_mask |= 1u << stage;
                issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (elected) drain_loads<STAGES>(full, issued_mask, issued_phase, guard);
        __syncwarp();
    } else if (warp == 7) {
        // ------------------------------------------------------------------ token codes, weight scales
        const bool elected = elect_one();
        const uint64_t x_policy = l2_policy_evict_last();   // a token tile is read by every column tile
        uint32_t stage = 0, phase = 0, issued_mask = 0, issued_phase = 0;
        bool ok = true;
        for (int i = 0; i < tiles && ok; ++i) {
            const SkinnyTile t = skinny_tile(i, sh, a, tprefix, off);
            const int nx = (t.rows + 15) / 16;
            const uint8_t* sfw = a.rhs_scale + (static_cast<long long>(t.g) * a.NB + t.nb) * a.KA * MX4_ATOM_BYTES;
            for (int ks = 0; ks < a.KS && t.q0 < t.q1; ++ks) {
                ok = mx4_wait_uniform(&empty[stage], phase ^ 1, guard);
                if (!ok) break;
                uint8_t* st = smem + stage * STAGE_BYTES;
                const int atoms = min(2, a.KA - 2 * ks);
                if (elected) {
                    mbar_arrive_expect_tx(&xfull[stage], nx * X_BOX + atoms * MX4_ATOM_BYTES);
                    for (int j = 0; j < nx; ++j)
                        tma_load_2d_hint(st + W_BYTES + j * X_BOX, &tmap_x, &xfull[stage], ks * MX4_STAGE_BYTES,
                                         t.row0 + 16 * j, x_policy);
                    bulk_load(st + W_BYTES + X_BYTES, sfw + static_cast<long long>(ks) * SF_BYTES,
                              atoms * MX4_ATOM_BYTES, &xfull[stage]);
                }
                __syncwarp();
                issued_mask |= 1u << stage;
                issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (elected) drain_loads<STAGES>(xfull, issued_mask, issued_phase, guard);
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------------------ token scale gather
        // lane l loads rows l and l + 32 of the token tile. (in, kn) is the group of stages being loaded, one
        // ahead of the one being stored, across tiles too
        uint32_t buf = 0, phase = 0;
        uint2 nxt[2][MX4_GROUP];
        int in = 0, kn = 0;
        SkinnyTile tn{};
        const auto load = [&] { load_scale_group(a, tn.row0, tn.rows, lane, kn, nxt); };
        if (tiles > 0) {
            tn = skinny_tile(0, sh, a, tprefix, off);
            load();
        }
        while (in < tiles && tn.q0 < tn.q1) {
            if (!mx4_wait_uniform(&aempty[buf], phase ^ 1, guard)) break;
#pragma unroll
            for (int r = 0; r < 2; ++r)
                put_scale_group(sfx_buf + buf * MX4_GROUP_BYTES, lane + 32 * r, nxt[r], a.KS - kn);
            __syncwarp();
            if (lane == 0) mbar_arrive(&afull[buf]);
            buf ^= 1;
            phase ^= buf == 0 ? 1 : 0;
            kn += MX4_GROUP;
            if (kn >= a.KS) {
                kn = 0;
                if (++in < tiles) tn = skinny_tile(in, sh, a, tprefix, off);
            }
            if (in < tiles) load();
        }
    } else if (warp >= SCALE_WARP) {
        // ------------------------------------------------------------------ scales
        const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;   // this warp's tensor-memory lanes
        uint32_t stage = 0, phase = 0, buf = 0, aphase = 0;
        bool ok = true;
        for (int i = 0; i < tiles && ok; ++i) {
            const SkinnyTile t = skinny_tile(i, sh, a, tprefix, off);
            for (int ks = 0; ks < a.KS && t.q0 < t.q1; ++ks) {
                const int j = ks % MX4_GROUP;
                if (j == 0) ok = mx4_wait_uniform(&afull[buf], aphase, guard);
                // this stage's loads were issued after the MMAs that read its scale columns had completed
                ok = ok && mx4_wait_uniform(&xfull[stage], phase, guard);
                if (!ok) break;
                tc_fence_after();
                const uint4* sx = reinterpret_cast<const uint4*>(sfx_buf + buf * MX4_GROUP_BYTES) + 64 * j + lane;
                const uint4* sw = reinterpret_cast<const uint4*>(smem + stage * STAGE_BYTES + W_BYTES + X_BYTES) + lane;
                const uint4 x0 = sx[0], x1 = sx[32], w0 = sw[0], w1 = sw[32];
                const uint32_t t0 = tmem_base + TMEM_SF_BASE + SF_COLS * stage + quarter;
                tmem_st_32x8(t0, w0, x0);
                tmem_st_32x8(t0 + 8, w1, x1);
                const bool last = j == MX4_GROUP - 1 || ks + 1 == a.KS;   // of this buffer of token scales
                __syncwarp();
                if (lane == 0 && last) mbar_arrive(&aempty[buf]);   // every lane's values are in registers
                ok = mx4_wait_uniform(&full[stage], phase, guard);
                tmem_st_wait();   // also on a stop: tensor memory is freed with no store of this warp in flight
                if (!ok) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfull[stage]);
                if (last) {
                    buf ^= 1;
                    aphase ^= buf == 0 ? 1 : 0;
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        const bool elected = elect_one();
        uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
        bool ok = true;
        for (int i = 0; i < tiles; ++i) {
            const SkinnyTile t = skinny_tile(i, sh, a, tprefix, off);
            if (t.q0 >= t.q1) break;   // only ever the last tile
            const int n = 16 * ((t.rows + 15) / 16);
            ok = mx4_wait_uniform(&tempty[acc], acc_phase ^ 1, guard);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * TT;
            const uint32_t idesc0 = idesc_mxf4(128, n, 0), idesc1 = idesc_mxf4(128, n, 2);
            for (int ks = 0; ks < a.KS; ++ks) {
                ok = mx4_wait_uniform(&sfull[stage], phase, guard);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sw = smem_u32(smem + stage * STAGE_BYTES);
                const uint64_t wdesc = smem_desc_sw128(sw, 16, 1024), xdesc = smem_desc_sw128(sw + W_BYTES, 16, 1024);
                const uint32_t sf_t = tmem_base + TMEM_SF_BASE + SF_COLS * stage;
                const int steps = min(4, (a.K - ks * MX4_STAGE_K + 63) / 64);   // MMAs of K = 64 with data
                if (elected) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        // +32 bytes (descriptor units of 16) per 64 elements inside the swizzled row
                        const uint32_t w_t = sf_t + 8 * (kk >> 1);
                        mma_mxf4<1>(d_tmem, wdesc + 2 * kk, xdesc + 2 * kk, (kk & 1) ? idesc1 : idesc0, w_t, w_t + 4,
                                    (ks | kk) != 0 ? 1u : 0u);
                    }
                    mma_commit(&empty[stage]);
                    if (ks + 1 == a.KS) mma_commit(&tfull[acc]);
                }
                __syncwarp();
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
        // all MMAs issued by this thread complete before teardown frees TMEM
        if (elected) {
            mma_commit(drain);
            int dummy;
            const WaitGuard dguard = drain_guard(guard, &dummy);
            (void)mbar_wait(drain, 0, dguard);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------------------ epilogue
        const int q = warp & 3;   // TMEM lane quarter: columns 32 q + lane of the tile's atom
        uint32_t acc = 0, acc_phase = 0;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
        for (int i = 0; i < tiles; ++i) {
            const SkinnyTile t = skinny_tile(i, sh, a, tprefix, off);
            if (t.q0 >= t.q1) break;
            if (!mx4_wait_warp(&tfull[acc], acc_phase, guard)) break;
            tc_fence_after();
            const int col = t.nb * 128 + q * 32 + lane;
            if (q >= t.q0 && q < t.q1) {
                for (int j0 = 0; j0 < t.rows; j0 += 16) {
                    uint32_t v[16];   // v[j]: token row row0 + j0 + j
                    tmem_ld_32x16(tmem_base + acc * TT + j0 + (static_cast<uint32_t>(q * 32) << 16), v);
                    tmem_ld_wait();
                    if (col < a.N) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (j0 + j >= t.rows) break;
                            out[(static_cast<long long>(t.row0) + j0 + j) * a.N + col] =
                                __float2bfloat16_rn(__uint_as_float(v[j]));
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            mbar_arrive(&tempty[acc]);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
        // zero rows [off[G], M): one contiguous range, split over CTAs and the 128 epilogue threads
        const long long b0 = static_cast<long long>(off[a.G]) * a.N * 2;
        const long long b1 = static_cast<long long>(a.M) * a.N * 2;   // both multiples of 16
        const long long nv = (b1 - b0) / 16;
        if (nv > 0) {
            uint4* base = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + b0);
            const long long per = (nv + gridDim.x - 1) / gridDim.x;
            const long long s = per * blockIdx.x;
            const long long e = min(nv, s + per);
            for (long long i = s + (threadIdx.x - 64); i < e; i += 128) base[i] = make_uint4(0, 0, 0, 0);
        }
    }

    // ---------------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

}  // namespace

cudaError_t launch_mxfp4_skinny(const CUtensorMap& tmap_x, const CUtensorMap (&tmap_w)[3], const Mx4Args& a, int grid,
                                cudaStream_t stream) {
    const size_t shm = smem_bytes(a.G);
    cudaError_t e = cudaFuncSetAttribute(mxfp4_skinny_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(shm));
    if (e != cudaSuccess) return e;
    return launch_pdl(mxfp4_skinny_kernel, dim3(grid), dim3(THREADS), shm, stream, tmap_x, tmap_w[0], tmap_w[1],
                      tmap_w[2], a);
}

}  // namespace rdot
