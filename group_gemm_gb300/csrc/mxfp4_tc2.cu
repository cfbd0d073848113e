// mxfp4_tc2.cu -- MXFP4 ragged-dot forward on CTA pairs (tcgen05 cta_group::2), 256 x 256 tiles.
//
// out[i, :] = A[i, :] B[g(i)] with A, B in MXFP4 (mxfp4.cuh), fp32 accumulation, bf16 out; rows past
// the last group end are zero. The pair mapping of fwd_tc2.cu and mxfp8_tc2.cu: per K stage (128 code
// bytes, 256 elements) CTA r stages rows [row0 + 128 r, +128) of the lhs codes, columns
// [n0 + 128 r, +128) of the rhs codes (16 KB each), the scale atoms of its rows (1 KB) and those of all
// 256 columns (2 KB). A pair tile asks half the operand bytes per SM of a 128 x 256 tile: at four bits
// the tensor cores consume a stage in 512 clocks, so a lone 128 x 256 tile would ask 100 bytes per
// clock and SM of L2, a pair tile 68.
//
// Scales reach tensor memory through registers, not through tcgen05.cp: the six copies a stage would need
// run in order with the MMAs on the tensor pipe (386 us without them against 531 with, in a timing copy
// of an earlier form without its row-scale gather, at the shapes below). Four scale warps per CTA, one for each lane quarter, write the stage's 24 columns with
// tcgen05.st: the rows' scales, gathered by another warp from global memory a group of stages ahead and
// put down as atoms; the weights' atoms (laid out once, by the quantiser), brought by TMA in a ring of
// their own. The even CTA issues M = 256, N = 256, K = 64 MMAs.
//
// Two accumulators share their middle: tensor memory holds 512 columns, the scales of five stages take
// 120, and a tile 256, so even tiles accumulate in columns [0, 256) and odd ones in [128, 384). The eight
// epilogue warps of a CTA read a tile's shared half out first, 64 columns each, and hand it back; the
// next tile then starts while they read the other half and store. (With one accumulator the MMAs waited
// about 2000 clocks a tile for the read-out, so about 1250.)
//
// Measured at 16384 rows x 4096 -> 14336, 8 experts: 300-310 us (6.2-6.4 PFLOP/s, by GPU) in a burst; 330-340 us
// sustained, where the power cap holds the clock at 1.7 GHz. At 4096 rows the tensor pipe is active 62 % of
// the clocks and L2 45 % busy (ncu); per stage the MMA warp spends about 500 clocks issuing (512 is the MMAs'
// own time) and 220 in its two waits. Short contractions are bound by the epilogue (65536 rows x 512 -> 4096:
// 120 us, 4.5 TB/s of output). Where K/32 is not a multiple of 4 the gather of the row scales, byte by byte with
// one stage in flight, sets the pace: 16384 rows x 2880 -> 5760, 32 experts 385 us, x 2816 107 us.
#include <cuda_bf16.h>

#include "drain.cuh"
#include "kernels.h"
#include "mxfp4.cuh"
#include "pairdrain.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "sched.cuh"

namespace rdot {

namespace {

constexpr int EPI_WARPS = 8;
constexpr int EPI_WARP = 4;                          // the first of eight; warps 0..3: codes, MMAs, weight scales, row scales
constexpr int SCALE_WARP = EPI_WARP + EPI_WARPS;     // the first of four
constexpr int THREADS = 32 * (SCALE_WARP + 4);
constexpr int BM = 256;                // rows per cluster tile
constexpr int BN = 256;
constexpr int STAGES = 5;
constexpr int A_BYTES = 128 * MX4_STAGE_BYTES;       // this CTA's 128 rows
constexpr int B_BYTES = 128 * MX4_STAGE_BYTES;       // this CTA's 128 columns
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int SFB_STAGES = 10;                       // the weight scales' own ring runs further ahead
constexpr int SFB_STAGE_BYTES = 4 * MX4_ATOM_BYTES;  // the scales of all 256 columns, 256 elements
constexpr int SFB_BYTES = SFB_STAGES * SFB_STAGE_BYTES;
constexpr int EPI_BYTES = EPI_WARPS * 32 * 64;      // a 32 x 32 bf16 block per epilogue warp
constexpr int BAR_BYTES = (3 * STAGES + 2 * SFB_STAGES + 8) / 2 * 16;   // full, sfull, empty; bfull, bempty; afull[2],
                                                                       // aempty[2], tfull, tempty, drain
constexpr int MISC_BYTES = 16;
constexpr int SFA_BYTES = 2 * MX4_GROUP_BYTES;       // the rows' scale atoms, two groups of stages
constexpr int XCH_BYTES = (sizeof(PairExchange<STAGES>) + 15) / 16 * 16;
constexpr int TMEM_COLS = 512;
constexpr int TMEM_SF_BASE = BN + BN / 2;            // after the two overlapping accumulators
constexpr int SF_COLS = 2 * (4 + 8);                 // per stage: two atoms of A and two of B (256 columns)
static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms stay 1 KB aligned");
static_assert(TMEM_SF_BASE + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");
constexpr uint32_t EMPTY_ARRIVALS = 2 * EPI_WARPS;

size_t smem_bytes(int G) {
    return 1024 + RING_BYTES + SFB_BYTES + SFA_BYTES + EPI_BYTES + BAR_BYTES + MISC_BYTES + XCH_BYTES +
           sizeof(int32_t) * 2 * (G + 1);
}

// Arrive on a barrier of the even CTA for work whose only data is tensor memory (scales written, an
// accumulator read): tcgen05.wait and tcgen05.fence order that data, so the arrive itself need not
// release this thread's other writes to the cluster. A release at cluster scope took about as long as a
// stage's MMAs, and one per stage set the kernel's pace (678 against 460 us at the shapes above).
__device__ __forceinline__ void mbar_arrive_tmem(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 32 rows x 64 accumulator columns of this warp's lane quarter as packed bf16: pk[c][j] holds columns
// 32c + 2j, 32c + 2j + 1 of row `lane`. Both loads are in flight together.
__device__ __forceinline__ void tmem_read_bf16_32x64(uint32_t taddr, uint32_t (&pk)[2][16]) {
    uint32_t v0[32], v1[32];
    tmem_ld_32x32b_x32(taddr, v0);
    tmem_ld_32x32b_x32(taddr + 32, v1);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        pk[0][j] = pack_bf16x2(__uint_as_float(v0[2 * j]), __uint_as_float(v0[2 * j + 1]));
        pk[1][j] = pack_bf16x2(__uint_as_float(v1[2 * j]), __uint_as_float(v1[2 * j + 1]));
    }
}

// Stores a 32 x 32 block already packed as bf16 (p[j]: columns 2j, 2j + 1 of row `lane`): turned through
// 2 KB of shared memory in 16-byte units (unit u of row r at u ^ (r / 2) % 4, conflict-free both ways), so that
// four lanes store 64 consecutive bytes of a row. Word-wise, as store_packed_bf16_32x32 turns its block, the
// epilogue took 4700 clocks a tile, more than the MMAs of a contraction below 2048.
__device__ __forceinline__ void store_block_bf16_v16(const uint32_t (&p)[16], uint4* stage, __nv_bfloat16* out,
                                                     long long ld, int rows_valid, int cols_valid) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        stage[4 * lane + (u ^ ((lane >> 1) & 3))] = make_uint4(p[4 * u], p[4 * u + 1], p[4 * u + 2], p[4 * u + 3]);
    __syncwarp();
    const int rr = lane >> 2, u = lane & 3;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = it * 8 + rr;
        const uint4 v = stage[4 * row + (u ^ ((row >> 1) & 3))];
        if (row < rows_valid && 8 * u < cols_valid) *reinterpret_cast<uint4*>(out + row * ld + 8 * u) = v;
    }
    __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    mxfp4_tc2_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ CUtensorMap tmap_sfb, Mx4Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sfb_ring = smem + RING_BYTES;
    uint8_t* sfa_buf = sfb_ring + SFB_BYTES;
    uint4* epi_stage = reinterpret_cast<uint4*>(sfa_buf + SFA_BYTES);
    uint8_t* bars = sfa_buf + SFA_BYTES + EPI_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(bars);
    uint64_t* sfull = full + STAGES;    // even CTA: both CTAs' scales of the stage are in tensor memory
    uint64_t* empty = sfull + STAGES;
    uint64_t* bfull = empty + STAGES;         // this CTA's weight scales of a stage are in shared memory
    uint64_t* bempty = bfull + SFB_STAGES;    // its scale warps have read them
    uint64_t* afull = bempty + SFB_STAGES;    // this CTA's row scales of a group of stages, two buffers
    uint64_t* aempty = afull + 2;
    uint64_t* tfull = aempty + 2;
    uint64_t* tempty = tfull + 1;
    uint64_t* drain = tempty + 1;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
    auto* xch = reinterpret_cast<PairExchange<STAGES>*>(bars + BAR_BYTES + MISC_BYTES);
    int32_t* off = reinterpret_cast<int32_t*>(bars + BAR_BYTES + MISC_BYTES + XCH_BYTES);
    int32_t* tprefix = off + a.G + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = static_cast<int>(cluster_id_x());
    const int nclusters = static_cast<int>(cluster_count_x());

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&sfull[s], 8);   // the four scale warps of each CTA
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < SFB_STAGES; ++s) {
            mbar_init(&bfull[s], 1);
            mbar_init(&bempty[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&afull[s], 1);
            mbar_init(&aempty[s], 4);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, EMPTY_ARRIVALS);
        mbar_init(drain, 1);
        mbar_init(&xch->bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmap_a);
        tma_prefetch_desc(&tmap_b);
        tma_prefetch_desc(&tmap_sfb);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, TMEM_COLS);
        tmem_relinquish_pair();
    }
    grid_dependency_enter();   // group sizes and operands may come from the previous kernel
    if (warp == 2) {
        const int bad = mx4_group_scan(a.group_sizes, a.G, a.M, BM, a.NT, off, tprefix);
        if (bad && lane == 0 && blockIdx.x == 0 && a.status) atomicOr(a.status, bad);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();

    const uint32_t tmem_base = *tmem_holder;
    const int W = tprefix[a.G];
    const bool m_inner = a.m_inner != 0;
    const WaitGuard guard{abort_flag, a.status, a.timeout_ns};

    if (warp == 0) {
        // ------------------------------------------------------------------ TMA producer (both CTAs)
        const bool elected = elect_one();
        uint32_t stage = 0, phase = 0;
        int pos = 0;   // load iterations issued (see pairdrain.cuh)
        bool ok = true;
        const int r = static_cast<int>(rank);
        for (int w = cluster; w < W && ok; w += nclusters) {
            const Tile t = decode_tile(w, tprefix, off, a.G, BM, a.NT, m_inner);
            const int n0 = t.nt * BN;
            // the odd CTA's A half unless wholly past the group, its B half unless wholly past N: what is
            // not loaded only feeds rows or columns that are not stored
            const int a1 = t.rows > 128 ? A_BYTES : 0;
            const int b1 = (n0 + 128 < a.N) ? B_BYTES : 0;
            const int my_a = r ? a1 : A_BYTES, my_b = r ? b1 : B_BYTES;
            for (int ks = 0; ks < a.KS; ++ks) {
                ok = mx4_wait_uniform(&empty[stage], phase ^ 1, guard);
                if (!ok) break;
                uint8_t* st = smem + stage * STAGE_BYTES;
                const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
                if (elected) {
                    if (leader) mbar_arrive_expect_tx(&full[stage], A_BYTES + a1 + B_BYTES + b1);
                    if (my_a) tma_load_2d_pair(st, &tmap_a, fb, ks * MX4_STAGE_BYTES, t.row0 + 128 * r);
                    if (my_b) tma_load_3d_pair(st + A_BYTES, &tmap_b, fb, ks * MX4_STAGE_BYTES, n0 + 128 * r, t.g);
                    xch->share[stage] = a1 + b1;   // the odd CTA's bytes of this iteration
                }
                __syncwarp();
                ++pos;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // every load either CTA issued lands before either CTA can leave (pairdrain.cuh)
        if (elected) pair_drain(xch, full, pos, leader, guard);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------------ weight scale producer (both CTAs)
        const bool elected = elect_one();
        uint32_t stage = 0, phase = 0, issued_mask = 0, issued_phase = 0;
        bool ok = true;
        for (int w = cluster; w < W && ok; w += nclusters) {
            const Tile t = decode_tile(w, tprefix, off, a.G, BM, a.NT, m_inner);
            const int row = t.g * a.NB + 2 * t.nt;   // two rows of the atoms' map: 128 columns each
            for (int ks = 0; ks < a.KS; ++ks) {
                ok = mx4_wait_uniform(&bempty[stage], phase ^ 1, guard);
                if (!ok) break;
                if (elected) {
                    // 2 x 256 words: the two column atoms' scales of this stage (zeros past the tensor)
                    mbar_arrive_expect_tx(&bfull[stage], SFB_STAGE_BYTES);
                    tma_load_2d(sfb_ring + stage * SFB_STAGE_BYTES, &tmap_sfb, &bfull[stage],
                                ks * (2 * MX4_ATOM_BYTES / 4), row);
                }
                __syncwarp();
                issued_mask |= 1u << stage;
                issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == SFB_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (elected) drain_loads<SFB_STAGES>(bfull, issued_mask, issued_phase, guard);
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------------ row scale gather (both CTAs)
        // lane l loads rows l, l + 32, l + 64, l + 96 of this CTA's half. (tn, kn) is the group of stages
        // being loaded, one ahead of the one being stored, across tiles too
        const int first = 128 * static_cast<int>(rank) + lane;
        uint32_t buf = 0, phase = 0;
        bool ok = true;
        uint2 nxt[4][MX4_GROUP];
        int wn = cluster, kn = 0;
        Tile tn{};
        const auto load = [&] { load_scale_group(a, tn.row0, tn.rows, first, kn, nxt); };
        if (wn < W) {
            tn = decode_tile(wn, tprefix, off, a.G, BM, a.NT, m_inner);
            load();
        }
        while (wn < W) {
            ok = mx4_wait_uniform(&aempty[buf], phase ^ 1, guard);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) put_scale_group(sfa_buf + buf * MX4_GROUP_BYTES, lane + 32 * i, nxt[i], a.KS - kn);
            __syncwarp();
            if (lane == 0) mbar_arrive(&afull[buf]);
            buf ^= 1;
            phase ^= buf == 0 ? 1 : 0;
            kn += MX4_GROUP;
            if (kn >= a.KS) {
                kn = 0;
                wn += nclusters;
                if (wn < W) tn = decode_tile(wn, tprefix, off, a.G, BM, a.NT, m_inner);
            }
            if (wn < W) load();
        }
    } else if (warp >= SCALE_WARP) {
        // ------------------------------------------------------------------ scales (both CTAs)
        const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;   // this warp's tensor-memory lanes
        uint32_t stage = 0, phase = 0, bstage = 0, bphase = 0, buf = 0, aphase = 0;
        bool ok = true;
        for (int w = cluster; w < W && ok; w += nclusters) {
            for (int ks = 0; ks < a.KS; ++ks) {
                const int j = ks % MX4_GROUP;
                if (j == 0) ok = mx4_wait_uniform(&afull[buf], aphase, guard);
                ok = ok && mx4_wait_uniform(&bfull[bstage], bphase, guard);
                if (!ok) break;
                // rows: [K atom]; weights: [column atom][K atom] of 32 x 16 bytes
                const uint4* sa = reinterpret_cast<const uint4*>(sfa_buf + buf * MX4_GROUP_BYTES) + 64 * j + lane;
                const uint4* sb = reinterpret_cast<const uint4*>(sfb_ring + bstage * SFB_STAGE_BYTES) + lane;
                const uint4 a0 = sa[0], a1 = sa[32], b00 = sb[0], b01 = sb[32], b10 = sb[64], b11 = sb[96];
                ok = mx4_wait_uniform(&empty[stage], phase ^ 1, guard);   // the MMAs that read these columns are done
                if (!ok) break;
                tc_fence_after();
                const uint32_t t = tmem_base + TMEM_SF_BASE + SF_COLS * stage + quarter;
                tmem_st_32x8(t, a0, b00);
                tmem_st_32x8(t + 8, b10, a1);
                tmem_st_32x8(t + 16, b01, b11);
                const bool last = j == MX4_GROUP - 1 || ks + 1 == a.KS;   // of this buffer of row scales
                __syncwarp();
                if (lane == 0) {   // every lane's values are in registers, taken by the stores above
                    mbar_arrive(&bempty[bstage]);
                    if (last) mbar_arrive(&aempty[buf]);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_tmem(mapa_shared(smem_u32(&sfull[stage]), 0));
                if (last) {
                    buf ^= 1;
                    aphase ^= buf == 0 ? 1 : 0;
                }
                if (++bstage == SFB_STAGES) {
                    bstage = 0;
                    bphase ^= 1;
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer (even CTA)
        if (leader) {
            const bool elected = elect_one();
            uint32_t stage = 0, phase = 0, acc_phase = 0;
            bool ok = true;
            for (int w = cluster; w < W && ok; w += nclusters) {
                ok = mx4_wait_uniform(tempty, acc_phase ^ 1, guard);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (acc_phase ? BN / 2 : 0);   // tiles alternate
                for (int ks = 0; ks < a.KS; ++ks) {
                    ok = mx4_wait_uniform(&full[stage], phase, guard) && mx4_wait_uniform(&sfull[stage], phase, guard);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                    const uint64_t adesc = smem_desc_sw128(sa, 16, 1024), bdesc = smem_desc_sw128(sa + A_BYTES, 16, 1024);
                    const uint32_t sf_t = tmem_base + TMEM_SF_BASE + SF_COLS * stage;
                    const int steps = min(4, (a.K - ks * MX4_STAGE_K + 63) / 64);   // MMAs of K = 64 with data
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            // +32 bytes (descriptor units of 16) per 64 elements inside the swizzled row
                            const uint32_t a_t = sf_t + 12 * (kk >> 1);
                            if (kk < steps)
                                mma_mxf4<2>(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc_mxf4(BM, BN, 2 * (kk & 1)),
                                            a_t, a_t + 4, (ks | kk) != 0 ? 1u : 0u);
                        }
                        mma_commit_pair_multicast(&empty[stage], 0x3);
                        if (ks + 1 == a.KS) mma_commit_pair_multicast(tfull, 0x3);
                    }
                    __syncwarp();
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                acc_phase ^= 1;
            }
            // the commit tracks what its own thread issued: one lane is elected once, for all of it
            if (elected) {
                mma_commit_pair(drain);
                int dummy;
                (void)mbar_wait(drain, 0, drain_guard(guard, &dummy));
            }
        }
        __syncwarp();
    } else if (warp >= EPI_WARP) {
        // ------------------------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3;
        const int half = (warp - EPI_WARP) / 4;
        uint4* stage_buf = epi_stage + (warp - EPI_WARP) * (32 * 64 / 16);
        uint32_t acc_phase = 0;
        for (int w = cluster; w < W; w += nclusters) {
            const Tile t = decode_tile(w, tprefix, off, a.G, BM, a.NT, m_inner);
            const bool ready = mx4_wait_warp(tfull, acc_phase, guard);
            if (!ready) break;
            tc_fence_after();
            const int first = 128 * static_cast<int>(rank) + q * 32;
            const int rows_valid = t.rows - first;
            __nv_bfloat16* out_rows =
                static_cast<__nv_bfloat16*>(a.out) + (static_cast<long long>(t.row0) + first) * a.N;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                // part 0: the half the accumulators share (columns 128.. of an even tile, 0.. of an odd one),
                // tensor-memory columns [128, 256); part 1: the tile's own, [0, 128) or [256, 384)
                const int tcol = (part == 0 ? BN / 2 : acc_phase ? BN : 0) + 64 * half;
                const int col0 = t.nt * BN + ((part == 0) != (acc_phase != 0) ? BN / 2 : 0) + 64 * half;
                uint32_t pk[2][16];
                tmem_read_bf16_32x64(tmem_base + tcol + (static_cast<uint32_t>(q * 32) << 16), pk);
                tc_fence_before();
                if (part == 0) {
                    // this warp has also read all of the tile before: the next tile may start
                    __syncwarp();
                    if (lane == 0) mbar_arrive_tmem(mapa_shared(smem_u32(tempty), 0));
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = col0 + c * 32;
                    if (rows_valid > 0 && col < a.N)
                        store_block_bf16_v16(pk[c], stage_buf, out_rows + col, a.N, rows_valid, a.N - col);
                }
            }
            acc_phase ^= 1;
        }
        {
            const long long b0 = static_cast<long long>(off[a.G]) * a.N * 2;
            const long long b1 = static_cast<long long>(a.M) * a.N * 2;
            const long long nv = (b1 - b0) / 16;
            if (nv > 0) {
                uint4* base = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + b0);
                const long long per = (nv + gridDim.x - 1) / gridDim.x;
                const long long s = per * blockIdx.x;
                const long long e = min(nv, s + per);
                for (long long i = s + (threadIdx.x - 32 * EPI_WARP); i < e; i += 32 * EPI_WARPS) base[i] = make_uint4(0, 0, 0, 0);
            }
        }
    }

    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

}  // namespace

cudaError_t launch_mxfp4_pair(const CUtensorMap& tmap_a, const CUtensorMap& tmap_b, const CUtensorMap& tmap_sfb,
                              const Mx4Args& a, int grid, cudaStream_t stream) {
    if (grid % 2) return cudaErrorInvalidValue;
    const size_t shm = smem_bytes(a.G);
    cudaError_t e = cudaFuncSetAttribute(mxfp4_tc2_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(shm));
    if (e != cudaSuccess) return e;
    return launch_pdl(mxfp4_tc2_kernel, dim3(grid), dim3(THREADS), shm, stream, tmap_a, tmap_b, tmap_sfb, a);
}

int mxfp4_pair_max_clusters(int G) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes(G);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    cudaError_t e = cudaFuncSetAttribute(mxfp4_tc2_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(cfg.dynamicSmemBytes));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, mxfp4_tc2_kernel, &cfg);
    return e == cudaSuccess ? n : 0;
}

}  // namespace rdot
