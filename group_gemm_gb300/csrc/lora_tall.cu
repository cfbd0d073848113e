// lora_tall.cu -- low-rank adapters beside a projection, for groups of many rows: the tcgen05 form of
// lora_apply.cu (same formulas, same split of t into hi + lo, same clusters along the columns).
//
// A tile is 128 rows of one group. Warp-specialised:
//   warp 0        producer: per stage 64 columns of the tile's rows (of x, then of base) and of the adapter's r
//                 weight rows, by TMA into an S-slot ring, in boxes of 32 rows: a short tile loads no row past
//                 its last box.
//   warp 1        tcgen05.mma: t's sums [128 x r] over the columns of x, in stretches of 512, then, per 64 output columns, hi and lo
//                 times the weights (K = 2r) into one of two accumulators.
//   warps 2..9    t: tensor memory -> (sum of the stretches) -> (sum over the cluster) -> scale -> hi, lo as the second product's A operand
//                 in shared memory; then the accumulators onto base, in base's own slot, and out as whole
//                 128-byte lines. Warps 2..5 take the even stages, 6..9 the odd ones.
//   warps 10..13  only with `order`: the rows by asynchronous 16-byte copies. (Four rows a TMA gather took
//                 58 ns to issue, 1.9 us a stage.)
// HBM bounds it: base and out pass once. 16384 rows of 8 groups, 4096 -> 14336, rank 16: 185 us, 5.8 TB/s (86 % of a
// copy's rate; tiles of 112 rows, one on each SM, the same), 14336 -> 4096 125 us. TMA takes the loads off the
// load/store pipe, which bounds the mma.sync form (242 and 182 us: 58 % of its wavefronts at 65 % of HBM's rate).
//
// Rows of the tile past its last (or with no valid row number) hold whatever the boxes or an earlier use left:
// a row of an accumulator depends on its own row alone, and they are not stored.
#include <cuda_bf16.h>

#include "drain.cuh"
#include "kernels.h"
#include "lora.cuh"
#include "mxfp4.cuh"
#include "pdl.cuh"
#include "ptx.cuh"

namespace rdot {

namespace {

constexpr int ROWS = 128;
constexpr int COLS = 64;            // columns per stage: one 128-byte swizzle row
constexpr int BOX_ROWS = 32;
constexpr uint32_t TMEM_COLS = 256; // t's sums at 0 and 128, then the accumulators at 128 and 192
constexpr uint32_t ACC0 = 128;
// Stages of a stretch of t's sums, 512 columns. The MMAs cut their sums to 24 bits at each step of 16 columns, always towards
// 0 (1e-5 of t over 14336 columns), so they add up a stretch at most; the epilogue warps add the stretches, rounded.
constexpr int STRETCH = 8;
constexpr uint32_t U1 = 128;        // a stretch's sums lie at 0, the next one's here

// Status bits of the waits that ran out in any call on this device, until they are cleared: the adapter calls have
// no workspace to report into.
__device__ int32_t g_status;

template <int RP_, int S_, int BLOCKS_, bool ORDER_>
struct TallCfg {
    static constexpr int RP = RP_;   // rank, rounded up
    static constexpr int S = S_;
    static constexpr bool ORDER = ORDER_;
    static constexpr int LOADERS = 4;                // warps
    static constexpr int THREADS = 32 * (10 + (ORDER ? LOADERS : 0));
    static constexpr int BLOCKS = BLOCKS_;           // per SM
    static constexpr int A_BYTES = ROWS * 128;
    static constexpr int SLOT = A_BYTES + RP * 128;
    static constexpr int T_BYTES = RP * 512 < A_BYTES ? A_BYTES : RP * 512;   // hi | lo; the cluster's partial sums before
    static constexpr int SMEM = 1024 + S * SLOT + T_BYTES;
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::BLOCKS)
    lora_tall_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_base,
                     const __grid_constant__ CUtensorMap map_first, const __grid_constant__ CUtensorMap map_second,
                     LoraArgs a, uint64_t timeout_ns) {
    constexpr int RP = Cfg::RP, S = Cfg::S, LOADERS = Cfg::LOADERS, THREADS = Cfg::THREADS;
    constexpr bool ORDER = Cfg::ORDER;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* tmat = smem + S * Cfg::SLOT;
    __shared__ __align__(8) uint64_t full[S], empty1[S], empty2[S], u_full[2], u_empty[2], t_ready, acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag;
    __shared__ __align__(16) int row_of[ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster_ctas()), rank = static_cast<int>(cluster_ctarank());

    grid_dependency_wait();
    const LoraTile tile = lora_find_tile<ROWS, THREADS>(a.group_sizes, a.G, a.M, static_cast<int>(blockIdx.x) / C);
    if (tile.rows == 0) return;   // the whole cluster
    lora_tile_rows<ROWS, THREADS>(row_of, tile, a.order, a.M);
    if (tile.g == a.G) {
        // rows without an adapter: out is base (nothing to do in place), t is 0
        __syncthreads();
        if (rank == 0 && a.t)
            for (long long e = tid; e < static_cast<long long>(tile.rows) * a.rank / 8; e += THREADS)
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.t) + static_cast<long long>(tile.p0) * a.rank)[e] = make_uint4(0u, 0u, 0u, 0u);
        if (a.base == a.out) return;
        const int vecs = a.N / 8;
        for (int r = rank * (THREADS / 32) + warp; r < tile.rows; r += C * (THREADS / 32)) {
            if (row_of[r] < 0) continue;
            const uint4* src = static_cast<const uint4*>(a.base) + static_cast<long long>(row_of[r]) * vecs;
            uint4* dst = static_cast<uint4*>(a.out) + static_cast<long long>(row_of[r]) * vecs;
            for (int i = lane; i < vecs; i += 32) dst[i] = a.base ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], ORDER ? 1 + 32 * LOADERS : 1);
            mbar_init(&empty1[s], 1);   // first product: the MMAs have read the slot
            mbar_init(&empty2[s], 4);   // second: the epilogue warps have stored from it
        }
        mbar_init(&t_ready, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&u_full[i], 1);
            mbar_init(&u_empty[i], 8);
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(&drain, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_holder, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Only now may the next kernel's blocks come: one of them beside this block could else take the tensor memory that this
    // one is about to ask for, and hold it while it waits for this grid to end.
    grid_launch_dependents();
    const uint32_t tmem = tmem_holder;
    const WaitGuard guard{&abort_flag, &g_status, timeout_ns};

    // this block's stages: chunks rank, rank + C, ... of both widths
    const int nk = (a.K + COLS - 1) / COLS, nn = (a.N + COLS - 1) / COLS;
    const int n1 = nk > rank ? (nk - rank + C - 1) / C : 0, n2 = nn > rank ? (nn - rank + C - 1) / C : 0;
    const int stages = n1 + n2;
    const int ranks = (a.rank + 15) & ~15;   // the MMAs' N and K: weight rows past the rank arrive as zeros

    // waits until stage i's slot has been read by the stage before it in the slot; by whole warps
    const auto slot_free = [&](int i) -> bool {
        if (i < S) return true;
        const int slot = i % S, j = i - S;
        const int uses1 = (n1 - slot + S - 1) / S;   // the slot's uses by the first product
        return j < n1 ? mx4_wait_uniform(&empty1[slot], (j / S) & 1, guard)
                      : mx4_wait_uniform(&empty2[slot], (j / S - uses1) & 1, guard);
    };

    // the cluster's three meetings over t, for the warps that have no part in it
    const auto meet_cluster = [] {
        for (int i = 0; i < 3; ++i) cluster_sync();
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- producer (uniform, one lane elected)
        const bool elected = elect_one();
        const int boxes = ORDER ? 0 : (tile.rows + BOX_ROWS - 1) / BOX_ROWS;
        uint32_t issued_mask = 0, issued_phase = 0;
        bool synced = C == 1;
        for (int i = 0; i < stages; ++i) {
            if (!synced && i == n1 + S) {   // from here a slot waits for the second product, which waits for the cluster
                meet_cluster();
                synced = true;
            }
            const int slot = i % S;
            if (!slot_free(i)) break;
            uint8_t* dst = smem + slot * Cfg::SLOT;
            const bool one = i < n1;
            const int c0 = ((one ? i : i - n1) * C + rank) * COLS;
            const int nb = one || a.base ? boxes : 0;
            if (elected) {
                mbar_arrive_expect_tx(&full[slot], nb * (BOX_ROWS * 128) + RP * 128);
                tma_load_3d(dst + Cfg::A_BYTES, one ? &map_first : &map_second, &full[slot], c0, 0, tile.g);
                for (int b = 0; b < nb; ++b)
                    tma_load_2d(dst + b * BOX_ROWS * 128, one ? &map_x : &map_base, &full[slot], c0, tile.p0 + b * BOX_ROWS);
            }
            __syncwarp();
            issued_mask |= 1u << slot;
            issued_phase = (issued_phase & ~(1u << slot)) | (static_cast<uint32_t>((i / S) & 1) << slot);
        }
        __syncwarp();
        if (!synced) meet_cluster();
        if (lane == 0) drain_loads<S>(full, issued_mask, issued_phase, guard);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer (uniform, one lane elected)
        const uint32_t idesc1 = idesc_f16(ROWS, ranks, true, true, false, false);
        const uint32_t idesc2 = idesc_f16(ROWS, COLS, true, true, false, true);
        const uint32_t ring = smem_u32(smem), ts = smem_u32(tmat);
        const bool elected = elect_one();
        bool ok = true;
        for (int i = 0; i < n1; ++i) {
            const int slot = i % S, c = i / STRETCH, u = c & 1;
            if (i % STRETCH == 0) ok = mx4_wait_uniform(&u_empty[u], ((c >> 1) & 1) ^ 1, guard);
            ok = ok && mx4_wait_uniform(&full[slot], (i / S) & 1, guard);
            if (!ok) break;
            if (ORDER) fence_proxy_async_smem();   // the copies were made in the generic proxy
            tc_fence_after();
            const uint32_t sa = ring + slot * Cfg::SLOT, sb = sa + Cfg::A_BYTES;
            if (elected) {
#pragma unroll
                for (int kk = 0; kk < COLS / 16; ++kk)
                    mma_f16(tmem + u * U1, smem_desc_sw128(sa + kk * 32, 16, 1024), smem_desc_sw128(sb + kk * 32, 16, 1024), idesc1,
                            (i % STRETCH | kk) != 0 ? 1u : 0u);
                mma_commit(&empty1[slot]);
                if (i % STRETCH == STRETCH - 1 || i == n1 - 1) mma_commit(&u_full[u]);
            }
            __syncwarp();
        }
        if (C > 1) meet_cluster();
        if (ok) ok = mx4_wait_uniform(&t_ready, 0, guard);
        for (int j = 0; ok && j < n2; ++j) {
            const int i = n1 + j, slot = i % S, b = j & 1;
            ok = mx4_wait_uniform(&acc_empty[b], ((j >> 1) & 1) ^ 1, guard) && mx4_wait_uniform(&full[slot], (i / S) & 1, guard);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sb = ring + slot * Cfg::SLOT + Cfg::A_BYTES, d = tmem + ACC0 + b * COLS;
            if (elected) {
                // column k of t (hi, then lo from `RP` on) lies in 64-column atoms of 16 KB, 128-byte rows
#pragma unroll
                for (int kk = 0; kk < RP / 16; ++kk) {
                    if (16 * kk >= ranks) break;
                    const uint64_t w = smem_desc_sw128(sb + kk * 2048, COLS * 128, 1024);
                    const int h = 16 * kk, l = RP + 16 * kk;
                    mma_f16(d, smem_desc_sw128(ts + (h >> 6) * Cfg::A_BYTES + (h & 63) * 2, 16, 1024), w, idesc2, kk != 0 ? 1u : 0u);
                    mma_f16(d, smem_desc_sw128(ts + (l >> 6) * Cfg::A_BYTES + (l & 63) * 2, 16, 1024), w, idesc2, 1u);
                }
                mma_commit(&acc_full[b]);
            }
            __syncwarp();
        }
        // all MMAs issued by this thread complete before teardown frees tensor memory
        if (elected) {
            mma_commit(&drain);
            int dummy;
            (void)mbar_wait(&drain, 0, drain_guard(guard, &dummy));
        }
        __syncwarp();
    } else if (warp < 10) {
        // ---------------------------------------------------------------- t, then the output
        const int half = warp >= 6 ? 1 : 0;  // of t's columns, of the stages
        const int q = warp & 3;              // the lane quarter of tensor memory that this warp may read
        const int r = 32 * q + lane;         // this lane's row
        const uint32_t trow = tmem + (static_cast<uint32_t>(32 * q) << 16);
        float4* part = reinterpret_cast<float4*>(tmat);   // partial sums, [rank / 4][row]
        const float scale = a.scale ? __ldg(a.scale + tile.g) : 1.f;
        constexpr int QUADS = RP / 8;        // this warp's columns of t, four at a time
        const int c0 = half * (RP / 2);
        float4 v[QUADS];
#pragma unroll
        for (int c = 0; c < QUADS; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        bool ok = true;
        for (int i = 0; i * STRETCH < n1; ++i) {
            ok = mx4_wait_warp(&u_full[i & 1], (i >> 1) & 1, guard);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < QUADS; c += 2) {
                uint32_t u[8];
                tmem_ld_32x32b_x8(trow + (i & 1) * U1 + c0 + 4 * c, u);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    v[c + j].x += __uint_as_float(u[4 * j]);
                    v[c + j].y += __uint_as_float(u[4 * j + 1]);
                    v[c + j].z += __uint_as_float(u[4 * j + 2]);
                    v[c + j].w += __uint_as_float(u[4 * j + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[i & 1]);
        }
        // eight columns of a row of t: a 16-byte piece of hi and of lo
        const auto split = [&](int h, const float4& x, const float4& y, uint4& hi, uint4& lo) {
            hi = lo = make_uint4(0u, 0u, 0u, 0u);
            if (h >= a.rank) return;   // past the rank 0, whatever x holds (there x times the zero weights may be NaN)
            split_bf16x2(x.x * scale, x.y * scale, hi.x, lo.x);
            split_bf16x2(x.z * scale, x.w * scale, hi.y, lo.y);
            split_bf16x2(y.x * scale, y.y * scale, hi.z, lo.z);
            split_bf16x2(y.z * scale, y.w * scale, hi.w, lo.w);
        };
        const auto place = [&](int row, int h) -> uint32_t {   // of the piece of columns h .. h + 7 in the operand
            return (h >> 6) * Cfg::A_BYTES + row * 128 + ((((h & 63) >> 3) ^ (row & 7)) << 4);
        };
        const auto keep = [&](int row, int h, const uint4& hi) {
            if (a.t && row < tile.rows && h < a.rank)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.t) + static_cast<long long>(tile.p0 + row) * a.rank + h) = hi;
        };
        if (C == 1) {
#pragma unroll
            for (int c = 0; c < QUADS; c += 2) {
                const int h = c0 + 4 * c;
                uint4 hi, lo;
                split(h, v[c], v[c + 1], hi, lo);
                keep(r, h, hi);
                *reinterpret_cast<uint4*>(tmat + place(r, h)) = hi;
                *reinterpret_cast<uint4*>(tmat + place(r, RP + h)) = lo;
            }
        } else {
            // Each block adds the partial sums of a C-th of the rows and gives every block hi and lo of them. (Each adding all
            // rows reads C times as much from the others: 8192 rows, rank 64, clusters of 8: 88 us against 74.)
            float4* mine = part + c0 / 4 * ROWS + r;
#pragma unroll
            for (int c = 0; c < QUADS; ++c) mine[c * ROWS] = v[c];
            cluster_sync();
            constexpr int PIECES = RP / 8, MAX = (ROWS / 2 * PIECES + 255) / 256;   // a lane's pieces: MAX with two blocks
            const int share = (ROWS + C - 1) / C;   // the last block's may be shorter
            uint4 hi[MAX], lo[MAX];
#pragma unroll
            for (int k = 0; k < MAX; ++k) {
                const int e = tid - 64 + 256 * k, row = rank * share + e % share, h = e / share * 8;
                if (e >= share * PIECES) break;
                if (row >= ROWS) continue;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                const uint32_t addr = smem_u32(part + h / 4 * ROWS + row);
#pragma unroll 4
                for (int p = 0; p < C; ++p) {
                    const uint32_t peer = mapa_shared(addr, p);
                    const float4 u = ld_shared_cluster_f4(peer), w = ld_shared_cluster_f4(peer + ROWS * 16);
                    x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
                    y = make_float4(y.x + w.x, y.y + w.y, y.z + w.z, y.w + w.w);
                }
                split(h, x, y, hi[k], lo[k]);
                keep(row, h, hi[k]);
            }
            cluster_sync();   // every block has read the sums: hi and lo take their place
#pragma unroll
            for (int k = 0; k < MAX; ++k) {
                const int e = tid - 64 + 256 * k, row = rank * share + e % share, h = e / share * 8;
                if (e >= share * PIECES) break;
                if (row >= ROWS) continue;
                for (int p = 0; p < C; ++p) {
                    const uint32_t peer = mapa_shared(smem_u32(tmat), p);
                    st_shared_cluster_u4(peer + place(row, h), hi[k]);
                    st_shared_cluster_u4(peer + place(row, RP + h), lo[k]);
                }
            }
            cluster_sync();
        }
        fence_proxy_async_smem();
        mbar_arrive(&t_ready);

        for (int j = half; ok && j < n2; j += 2) {
            const int i = n1 + j, slot = i % S;
            ok = mx4_wait_warp(&full[slot], (i / S) & 1, guard) && mx4_wait_warp(&acc_full[half], (j >> 1) & 1, guard);
            if (!ok) break;
            tc_fence_after();
            uint8_t* rows = smem + slot * Cfg::SLOT;
            uint8_t* mine = rows + r * 128;
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // 32 columns at a time
                uint32_t acc[32];
                tmem_ld_32x32b_x32(trow + ACC0 + half * COLS + 32 * p, acc);
                tmem_ld_wait();
                if (p == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[half]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4* at = reinterpret_cast<uint4*>(mine + (((4 * p + c) ^ (r & 7)) << 4));
                    const uint4 u = a.base ? *at : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = pack_bf16x2(__uint_as_float(w[e] << 16) + __uint_as_float(acc[8 * c + 2 * e]),
                                           __uint_as_float(w[e] & 0xffff0000u) + __uint_as_float(acc[8 * c + 2 * e + 1]));
                    *at = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            __syncwarp();
            const int col = (j * C + rank) * COLS + 8 * (lane & 7);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int rr = 32 * q + 4 * k + (lane >> 3);
                const int row = row_of[rr];
                if (row >= 0 && col < a.N)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + static_cast<long long>(row) * a.N + col) =
                        *reinterpret_cast<const uint4*>(rows + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            }
            fence_proxy_async_smem();   // the slot's next load comes after these writes
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty2[slot]);
        }
    } else if constexpr (ORDER) {
        // ---------------------------------------------------------------- rows through `order`
        constexpr int STEP = LOADERS * 4;   // a multiple of 8: the swizzle is the same for all of a lane's rows
        const int piece = lane & 7, first = (warp - 10) * 4 + (lane >> 3);
        // this lane's rows of the tile, in registers: a look-up in front of each copy would make it wait
        int own[ROWS / STEP];
#pragma unroll
        for (int k = 0; k < ROWS / STEP; ++k) own[k] = row_of[first + k * STEP];
        bool synced = C == 1;
        for (int i = 0; i < stages; ++i) {
            if (!synced && i == n1 + S) {
                meet_cluster();
                synced = true;
            }
            if (!slot_free(i)) break;
            const bool one = i < n1;
            if (one || a.base) {
                const int width = one ? a.K : a.N;
                const int c = ((one ? i : i - n1) * C + rank) * COLS + 8 * piece;
                const uint16_t* src = static_cast<const uint16_t*>(one ? a.x : a.base) + c;
                const uint32_t dst = smem_u32(smem + (i % S) * Cfg::SLOT) + first * 128 + ((piece ^ (first & 7)) << 4);
#pragma unroll
                for (int k = 0; k < ROWS / STEP; ++k)
                    if (k * STEP < tile.rows) {
                        const bool live = own[k] >= 0 && c < width;
                        cp_async16(dst + k * STEP * 128, live ? src + static_cast<long long>(own[k]) * width : a.x, live);
                    }
            }
            cp_async_arrive(&full[i % S]);
        }
        cp_async_commit();
        cp_async_wait<0>();   // nothing lands after the block has left
        __syncwarp();
        if (!synced) meet_cluster();
    }

    // ---------------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <class Cfg>
cudaError_t launch_cfg(const CUtensorMap (&maps)[4], const LoraArgs& a, int C, uint64_t timeout_ns, cudaStream_t stream) {
    auto kern = lora_tall_kernel<Cfg>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    // a tile more for each group that ends inside one, one more for the rows of no group
    const long long tiles = (static_cast<long long>(a.M) + ROWS - 1) / ROWS + (a.G < a.M ? a.G : a.M) + 1;
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(tiles * C)), dim3(Cfg::THREADS), C, Cfg::SMEM, stream, maps[0],
                              maps[1], maps[2], maps[3], a, timeout_ns);
}

template <bool ORDER>
cudaError_t launch_rank(const CUtensorMap (&maps)[4], const LoraArgs& a, int C, bool deep, uint64_t timeout_ns,
                        cudaStream_t stream) {
    if (deep) {
        if (a.rank <= 16) return launch_cfg<TallCfg<16, 8, 1, ORDER>>(maps, a, C, timeout_ns, stream);
        if (a.rank <= 32) return launch_cfg<TallCfg<32, 8, 1, ORDER>>(maps, a, C, timeout_ns, stream);
        if (a.rank <= 64) return launch_cfg<TallCfg<64, 7, 1, ORDER>>(maps, a, C, timeout_ns, stream);
        return launch_cfg<TallCfg<128, 4, 1, ORDER>>(maps, a, C, timeout_ns, stream);
    }
    if (a.rank <= 16) return launch_cfg<TallCfg<16, 5, 2, ORDER>>(maps, a, C, timeout_ns, stream);
    if (a.rank <= 32) return launch_cfg<TallCfg<32, 4, 2, ORDER>>(maps, a, C, timeout_ns, stream);
    if (a.rank <= 64) return launch_cfg<TallCfg<64, 3, 2, ORDER>>(maps, a, C, timeout_ns, stream);
    return launch_cfg<TallCfg<128, 4, 1, ORDER>>(maps, a, C, timeout_ns, stream);
}

}  // namespace

cudaError_t launch_lora_tall(const CUtensorMap (&maps)[4], const LoraArgs& a, int C, bool deep, uint64_t timeout_ns,
                             cudaStream_t stream) {
    return a.order ? launch_rank<true>(maps, a, C, deep, timeout_ns, stream)
                   : launch_rank<false>(maps, a, C, deep, timeout_ns, stream);
}

cudaError_t lora_tall_status(int32_t** word) {
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_status);
    *word = static_cast<int32_t*>(p);
    return e;
}

int lora_tall_box_rank(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

}  // namespace rdot
