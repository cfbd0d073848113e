// lora_grad.cu -- the gradients of low-rank adapters: dw[g] = t_g^T z_g, a contraction over a group's rows.
//
// With t = scale x down^T the gradient of up is t^T dy, and with dt = scale dy up^T that of down is dt^T x: one
// kernel, [rank x C] sums for each group. z is bf16 or an 8-bit checkpoint (E4M3 codes with a scale per row
// and 32 columns), widened to bf16 on the way to shared memory, so the activation is never written in 16 bits.
// The scales do not run along the contraction, so the block-scaled MMAs cannot take them.
//
// A work item is 128 columns of a group: D [128 columns x rank] in tensor memory, z as the MMA's A operand and t
// as its B, both as they lie in memory (MN-major), 64 rows a stage. z is read once; t, C/128 times from L2.
// Persistent blocks, one per SM, 19 warps (above rank 64, where the ring has six slots, 17: six teams):
//   warps 0..13   loaders, seven teams of two warps that take the stages in turn: z and t by asynchronous 16-byte
//                 copies into swizzled slots, zeros past the group's last row; codes instead through registers, a
//                 team's next stage while it widens the last. They run ahead over the items' ends, so short
//                 groups follow one another without a pause. (All loaders on every stage: 51 us against
//                 33 for 16384 x 4096 codes, rank 16; each stage's waits then lie in a row.)
//   warp 14       tcgen05.mma into one of four accumulators (three above rank 64), a stretch of 512 or 1024 rows at most into each
//   warps 15..18  epilogue: a lane a column, so that each rank's row of dw is stored in whole lines
// Few items: a cluster divides the group's rows, a block a share, and adds the fp32 partial sums through distributed
// shared memory in rank order. No atomics: the same result every time.
//
// What bounds it (times of the kernel replayed): bf16, the loads (5 TB/s of z in the steady state, and 16384 x 4096 of 8
// groups is 256 items for 152 SMs, two rounds: 29 us, floor 20); codes, 0.36 us a 64-row stage, of which widening, loads
// and MMAs each hide most of the others (29 us, floor 10.6); short groups, the epilogue's stores (4099 rows of 24 groups
// x 7168, rank 64: 23.5 us, floor 11.1); where one group has most rows, its items. Tried for those: each block a run of
// items of equal cost (stages and epilogues) in place of every 152nd, no faster with groups of one length or of skewed
// ones (31 us against 31, 38 against 35 for the last case).
#include <cuda_bf16.h>

#include "kernels.h"
#include "lora.cuh"
#include "mxfp4.cuh"
#include "pdl.cuh"

namespace rdot {

namespace {

constexpr int GC = 128;           // columns of an item
constexpr int GR = 64;            // rows of a stage
constexpr int LT = 64;            // threads of a team of loaders
constexpr int CHUNK = GR * 128;   // 64 columns x 64 rows of bf16: 8 KB
constexpr int ROW_RING = 4;       // a team's stages whose row numbers are held
constexpr int MASKS = 16;         // items whose NaN columns are held

__device__ int32_t g_status;      // bits of the waits that ran out, until they are cleared

template <int RP_, bool CODES_, bool ORDER_>
struct GradCfg {
    static constexpr int RP = RP_;
    static constexpr bool CODES = CODES_;
    static constexpr bool ORDER = ORDER_;
    static constexpr int TCHUNKS = (RP + 63) / 64;
    static constexpr int SLOT = (2 + TCHUNKS) * CHUNK;
    static constexpr int S = RP <= 64 ? 8 : 6;
    // 14 loader warps: with the other five, five to a quarter of the SM leave 96 registers a thread
    static constexpr int TEAMS = RP <= 64 ? 7 : 6;
    static constexpr int LOADERS = TEAMS * LT / 32;
    static constexpr int THREADS = 32 * (LOADERS + 5);
    // A team that reaches stage u has passed the wait of stage u - TEAMS, so stage u - TEAMS - S has been read. That must
    // cover stage u - 2S, else its wait could take the slot's phase before last for the last.
    static_assert(TEAMS <= S, "a wait tells two phases of a slot apart");
    static constexpr int RING = S * SLOT;                        // also the cluster's partial sums: RP x 512 bytes
    static constexpr int ROWS_BYTES = ORDER ? TEAMS * ROW_RING * GR * 4 : 0;
    static constexpr int SMEM = 1024 + RING + ROWS_BYTES;        // and the G + 1 offsets
    // Rows of a stretch. The MMAs cut their sums to 24 bits at each step of 16 rows, always towards 0, so an accumulator that
    // ran over a group of 131072 rows was off by 8e-5 (codes 3e-5: their products have fewer bits). It takes so many at
    // most that it stays within 6e-7, and the epilogue adds the stretches up in fp32, rounded, in tensor memory. (16384 x
    // 4096 of 8 groups, rank 16: codes 29.0 us, in stretches of 512 29.8, of any length 28.6; bf16 28.6, 28.2 of 1024,
    // 27.8 of any length.)
    static constexpr int STRETCH = CODES ? 1024 : 512;
    static constexpr int ACCS = RP <= 64 ? 4 : 3;                // accumulators; behind them the sums of an item's stretches
    static constexpr uint32_t TMEM_COLS = RP <= 16 ? 128 : RP <= 32 ? 256 : 512;
    static_assert(ACCS * RP + (RP + 31) / 32 * 32 <= TMEM_COLS, "they are read 32 columns at a time");
    static_assert(RP * 512 <= RING, "the partial sums fit the ring");
    static_assert(SMEM + (RDOT_MAX_GROUPS + 1) * 4 <= 227 * 1024 - 2048, "with the static shared memory it fits a block");
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two E4M3 codes, bytes J and J + 1 of w, as a bf16 pair times 2^-120. A code, sign-extended to 16 bits and moved up
// by four, has its sign, exponent and mantissa where bf16 has its sign, low exponent bits and high mantissa bits,
// subnormals included.
template <int J>
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t w) {
    uint32_t v;   // selector bit 3: the byte's sign, eight times
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(v) : "r"(w), "n"(J | (J | 8) << 4 | (J + 1) << 8 | ((J + 1) | 8) << 12));
    return (v * 16u) & 0x87f087f0u;
}

// Bit 7 of each byte: whether the code there is NaN (magnitude 127).
__device__ __forceinline__ uint32_t nan_code(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }

// What a block's items are cut from: item i is column block i % blocks of group i / blocks.
struct Items {
    const int32_t* off;     // [G + 1] shared: the groups' first positions
    int G, blocks;
    int dg, dcb;            // from one of the block's items to its next: groups, column blocks (no division on the way)
    int rank, C;            // the block's share of a group's stages: part `rank` of C

    // The block's rows of group g: n from sorted position p0 on.
    __device__ __forceinline__ void share(int g, int& p0, int& n) const {
        p0 = off[g];
        n = off[g + 1] - p0;
        if (C == 1) return;
        const unsigned all = (static_cast<unsigned>(n) + GR - 1) / GR;   // < 2^25
        const unsigned s0 = all * rank / C, s1 = all * (rank + 1) / C;
        p0 += static_cast<int>(s0 * GR);
        n = static_cast<int>(min(s1 * GR, static_cast<unsigned>(n)) - s0 * GR);
    }
    __device__ __forceinline__ void step(int& g, int& cb) const {
        g += dg;
        cb += dcb;
        if (cb >= blocks) {
            cb -= blocks;
            ++g;
        }
    }
};

// A place among the stages of a block's items.
struct Stage {
    int g, cb;      // the item after the current one
    int p0 = 0;     // the stage's first sorted position
    int n = 0;      // rows from there to the end of the block's share of the item; 0: no stage
    int c0 = 0;     // the item's first column
    int count = -1; // items with a row up to this one, less one

    // k >= 1 stages on: the stage's rows are p0 .. p0 + min(n, GR) - 1. False past the last (n is then 0).
    __device__ __forceinline__ bool advance(const Items& it, int k) {
        while (true) {
            const int left = n > GR ? (n - 1) / GR : 0;   // stages of this item after the current one
            if (k <= left) {
                p0 += k * GR;
                n -= k * GR;
                return true;
            }
            k -= left + 1;
            n = 0;
            while (n == 0) {
                if (g >= it.G) return false;
                c0 = cb * GC;
                it.share(g, p0, n);
                it.step(g, cb);
            }
            ++count;
            if (k == 0) return true;
        }
    }
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1) lora_grad_kernel(LoraGradArgs a, int blocks, bool out_bf16, uint64_t timeout_ns) {
    constexpr int RP = Cfg::RP, S = Cfg::S, TEAMS = Cfg::TEAMS, LOADERS = Cfg::LOADERS, THREADS = Cfg::THREADS, ACCS = Cfg::ACCS;
    constexpr int STRETCH = Cfg::STRETCH;
    constexpr bool CODES = Cfg::CODES, ORDER = Cfg::ORDER;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* rows = reinterpret_cast<int*>(smem + Cfg::RING);
    int32_t* off = reinterpret_cast<int32_t*>(smem + Cfg::RING + Cfg::ROWS_BYTES);
    __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[ACCS], acc_empty[ACCS], drain;
    __shared__ long long scan_part[THREADS / 32];
    __shared__ uint32_t tmem_holder;
    __shared__ uint32_t nan_cols[MASKS][GC / 32];
    __shared__ int abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster_ctas()), rank = static_cast<int>(cluster_ctarank());

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], LT / 32);   // a team's warps
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < ACCS; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(&drain, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < MASKS * (GC / 32)) nan_cols[tid / (GC / 32)][tid % (GC / 32)] = 0;
    // As in lora_tall.cu: tensor memory only once the kernel before has ended, the next one's blocks only once this block has
    // its own. Else a block could hold what a block of the kernel that it waits for is about to ask for.
    grid_dependency_wait();
    if (warp == LOADERS) {
        tmem_alloc(&tmem_holder, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    {
        // the groups' first positions, ends clamped to M, a negative size as 0
        constexpr int PER = (RDOT_MAX_GROUPS + THREADS - 1) / THREADS;
        long long v[PER], sum = 0, total;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = tid * PER + j;
            v[j] = i < a.G ? max(__ldg(a.group_sizes + i), 0) : 0;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) sum += v[j];
        long long at = block_scan<THREADS>(sum, scan_part, &total);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = tid * PER + j;
            if (i < a.G) off[i] = static_cast<int32_t>(min(at, static_cast<long long>(a.M)));
            at += v[j];
        }
        if (tid == 0) off[a.G] = static_cast<int32_t>(min(total, static_cast<long long>(a.M)));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_launch_dependents();
    const uint32_t tmem = tmem_holder;
    const WaitGuard guard{&abort_flag, &g_status, timeout_ns};
    const int first = static_cast<int>(blockIdx.x) / C, step = static_cast<int>(gridDim.x) / C;
    const int first_g = first / blocks, first_cb = first - first_g * blocks;
    const Items it{off, a.G, blocks, step / blocks, step % blocks, rank, C};
    const int ranks = (a.rank + 15) & ~15;   // the MMAs' N; t's columns past the rank are zeros

    if (warp < LOADERS) {
        // ---------------------------------------------------------------- loaders
        const int team = tid / LT, lt = tid % LT;
        Stage st{first_g, first_cb};   // the team's stage, and its next ones
        bool run = st.advance(it, 1 + team);
        Stage nx = st;
        if (!run || !nx.advance(it, TEAMS)) nx.n = 0;
        Stage far = nx;      // with `order`, of the row numbers: two of the team's stages on
        bool stopped = false;      // a wait ran out: with `order` the warp still meets the team at its barrier
        int* own_rows = rows + team * ROW_RING * GR;
        static_assert(LT == GR, "a thread a row number");
        const auto row_at = [&](const Stage& s, int i, int r) -> int {   // row of z for row r of the team's stage i, -1 for none
            if (r >= s.n) return -1;
            if (!ORDER) return s.p0 + r;
            const int row = own_rows[(i % ROW_RING) * GR + r];
            return row < a.M ? max(row, -1) : -1;
        };
        const auto row_number = [&](const Stage& s) -> int { return lt < s.n ? __ldg(a.order + s.p0 + lt) : -1; };
        const auto team_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(LT) : "memory"); };
        int number = -1;           // this thread's row number of the stage after the next
        if (ORDER) {
            own_rows[lt] = row_number(st);
            own_rows[GR + lt] = row_number(nx);
            if (far.n == 0 || !far.advance(it, TEAMS)) far.n = 0;
            number = row_number(far);
            team_sync();
        }
        // t's rows of the team's stage i into its slot
        constexpr int W = RP / 8;
        const auto load_t = [&](int i, uint32_t slot) {
#pragma unroll
            for (int e = lt; e < GR * W; e += LT) {
                const int r = e / W, j = e % W;
                const bool ok = 8 * j < a.rank && row_at(st, i, r) >= 0;
                cp_async16(slot + (2 + (j >> 3)) * CHUNK + r * 128 + (((j & 7) ^ (r & 7)) << 4),
                           static_cast<const uint16_t*>(a.t) + (ok ? static_cast<long long>(st.p0 + r) * a.rank + 8 * j : 0), ok);
            }
        };
        // codes: eight pieces of 16 a row, rows lt / 8, lt / 8 + 8, ...; a piece and its scale byte in registers
        constexpr int Q = CODES ? GR / 8 : 1;
        const int piece = CODES ? lt & 7 : lt & 15, r0 = CODES ? lt >> 3 : lt >> 4;
        const int sb = a.C / 32;   // scales of a row
        uint4 code[Q];
        uint32_t scale[Q];
        const auto fetch = [&](const Stage& s, int i) {
            const int c = s.c0 + 16 * piece;
            if (!ORDER && s.n >= GR && c < a.C) {   // whole stages: a step along the rows
                const uint8_t* p = static_cast<const uint8_t*>(a.z) + static_cast<long long>(s.p0 + r0) * a.C + c;
                const uint8_t* ps = a.z_scale + static_cast<long long>(s.p0 + r0) * sb + (c >> 5);
#pragma unroll
                for (int k = 0; k < Q; ++k, p += 8 * static_cast<long long>(a.C), ps += 8 * sb) {
                    code[k] = __ldg(reinterpret_cast<const uint4*>(p));
                    scale[k] = __ldg(ps);
                }
                return;
            }
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                const int row = c < a.C ? row_at(s, i, r0 + 8 * k) : -1;
                code[k] = make_uint4(0u, 0u, 0u, 0u);
                scale[k] = 127u;
                if (row >= 0) {
                    code[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.z) + static_cast<long long>(row) * a.C + c));
                    scale[k] = __ldg(a.z_scale + static_cast<long long>(row) * sb + (c >> 5));
                }
            }
        };
        uint32_t seen[4] = {};   // bit 7 of a byte: a NaN code in that column of the item
        if (CODES) fetch(st, 0);
        for (int i = 0; run; ++i) {   // the team's stage i, the block's stage u
            const int u = team + TEAMS * i, slot = u % S;
            const bool next = nx.n > 0;
            stopped = stopped || !mx4_wait_uniform(&empty[slot], ((u / S) & 1) ^ 1, guard);
            if (stopped && !ORDER) break;
            uint8_t* dst = smem + slot * Cfg::SLOT;
            if (!stopped) {
                load_t(i, smem_u32(dst));
                if constexpr (!CODES) {
                    const int c = st.c0 + 8 * piece;
#pragma unroll
                    for (int k = 0; k < GR / 4; ++k) {
                        const int r = r0 + 4 * k, row = row_at(st, i, r);
                        const bool ok = row >= 0 && c < a.C;
                        cp_async16(smem_u32(dst) + (piece >> 3) * CHUNK + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
                                   static_cast<const uint16_t*>(a.z) + (ok ? static_cast<long long>(row) * a.C + c : 0), ok);
                    }
                }
                cp_async_commit();
            }
            if constexpr (CODES) {
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const uint4 q = code[k];
                    const uint32_t s = scale[k], s1 = min(s, 134u);
                    seen[0] |= nan_code(q.x);
                    seen[1] |= nan_code(q.y);
                    seen[2] |= nan_code(q.z);
                    seen[3] |= nan_code(q.w);
                    // 2^120 x 2^(s - 127), in two steps where bf16 does not hold it
                    const uint32_t f = (s1 + 120u) * 0x00800080u;
                    uint32_t v[8] = {widen_e4m3x2<0>(q.x), widen_e4m3x2<2>(q.x), widen_e4m3x2<0>(q.y), widen_e4m3x2<2>(q.y),
                                     widen_e4m3x2<0>(q.z), widen_e4m3x2<2>(q.z), widen_e4m3x2<0>(q.w), widen_e4m3x2<2>(q.w)};
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = mul_bf16x2(v[j], f);
                    if (s > 134u) {
                        const uint32_t f2 = s == 255u ? 0x7fff7fffu : (s - s1 + 127u) * 0x00800080u;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = mul_bf16x2(v[j], f2);
                    }
                    const int r = r0 + 8 * k, unit = 2 * (piece & 3);
                    uint8_t* row = dst + (piece >> 2) * CHUNK + r * 128;
                    if (!stopped) {
                        *reinterpret_cast<uint4*>(row + ((unit ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4*>(row + (((unit + 1) ^ (r & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                }
                if (!next || nx.count != st.count) {
                    // the team's last stage of the item. A NaN code went in as 480 x scale: its column's sums are NaN
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t m = seen[j] & 0x80808080u;
                        if (m) {
                            const uint32_t bits = (m >> 7 & 1u) | (m >> 14 & 2u) | (m >> 21 & 4u) | (m >> 28 & 8u);
                            atomicOr(&nan_cols[st.count % MASKS][piece >> 1], bits << (16 * (piece & 1) + 4 * j));
                        }
                        seen[j] = 0;
                    }
                }
                fetch(nx, i + 1);
            }
            // the stage has landed; written in the generic proxy, read by the MMAs in the async one. (The fence once for all
            // by the MMA warp: 33 against 30 us for 16384 x 4096 codes.)
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && !stopped) mbar_arrive(&full[slot]);
            run = next;
            st = nx;
            if (ORDER) {
                own_rows[((i + 2) % ROW_RING) * GR + lt] = number;
                nx = far;
                if (far.n == 0 || !far.advance(it, TEAMS)) far.n = 0;
                number = row_number(far);
                team_sync();
            } else if (nx.n == 0 || !nx.advance(it, TEAMS)) {
                nx.n = 0;
            }
        }
        __syncwarp();
    } else if (warp == LOADERS) {
        // ---------------------------------------------------------------- MMA issuer (uniform, one lane elected)
        // Its own instructions cost more than the MMAs (four MMAs fewer change nothing), so they are few: counters for divisions,
        // descriptors made outside the elected branch (in uniform registers), the next stage's barrier looked at ahead of
        // this one's MMAs (16384 x 4096 codes: 1.7 us less).
        const bool elected = elect_one();
        const uint32_t idesc = idesc_f16(GC, ranks, true, true, true, true);
        const uint64_t da0 = smem_desc_sw128(smem_u32(smem), CHUNK, 1024), db0 = smem_desc_sw128(smem_u32(smem) + 2 * CHUNK, CHUNK, 1024);
        int slot = 0, count = 0;
        uint32_t phase = 0;
        bool ok = true, ready = false;
        for (int g = first_g, cb = first_cb; ok && g < a.G; it.step(g, cb)) {
            int p0, n;
            it.share(g, p0, n);
            for (int left = n; ok && left > 0;) {
                const int b = count % ACCS, from = left, to = max(left - STRETCH, 0);
                ok = mx4_wait_uniform(&acc_empty[b], ((count / ACCS) & 1) ^ 1, guard);
                for (; ok && left > to; left -= GR) {
                    ok = ready || mx4_wait_uniform(&full[slot], phase, guard);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = da0 + static_cast<uint32_t>(slot) * (Cfg::SLOT >> 4), db = db0 + static_cast<uint32_t>(slot) * (Cfg::SLOT >> 4);
                    const uint32_t fresh = left == from ? 0u : 1u;
                    uint64_t* const done = &empty[slot];
                    if (++slot == S) {
                        slot = 0;
                        phase ^= 1;
                    }
                    ready = mbar_test_uniform(&full[slot], phase);
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < GR / 16; ++kk)   // 16 rows: two groups of 8, 2 KB
                            if (16 * kk < left) mma_f16(tmem + b * RP, da + kk * 128, db + kk * 128, idesc, kk == 0 ? fresh : 1u);
                        mma_commit(done);
                        if (left - GR <= to) mma_commit(&acc_full[b]);
                    }
                    __syncwarp();
                }
                ++count;
            }
        }
        // all MMAs issued by this thread complete before teardown frees tensor memory
        if (elected) {
            mma_commit(&drain);
            int dummy;
            (void)mbar_wait(&drain, 0, drain_guard(guard, &dummy));
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3;                        // the lane quarter of tensor memory that this warp may read
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
        float* part = reinterpret_cast<float*>(smem);  // [rank][128 columns], once the ring is done with
        int count = 0, items = 0;                      // stretches, items with a row
        for (int g = first_g, cb = first_cb; g < a.G; it.step(g, cb)) {
            const int col = cb * GC + 32 * q + lane;
            int p0, n;
            it.share(g, p0, n);
            int b = count % ACCS;
            bool nan = false;
            if (n > 0) {
                if (!mx4_wait_warp(&acc_full[b], (count / ACCS) & 1, guard)) break;
                tc_fence_after();
                if (n > STRETCH) {
                    // every stretch, the last one too, into the sums
                    bool ok = true;
                    for (int left = n;;) {
#pragma unroll 1
                        for (int j0 = 0; j0 < a.rank; j0 += 16) {
                            uint32_t v[16], u[16];
                            tmem_ld_32x32b_x16(lanes + b * RP + j0, v);
                            if (left < n) {
                                tmem_ld_32x32b_x16(lanes + ACCS * RP + j0, u);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(u[j]) + __uint_as_float(v[j]));
                            } else {
                                tmem_ld_wait();
                            }
                            tmem_st_32x32b_x16(lanes + ACCS * RP + j0, v);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_empty[b]);
                        ++count;
                        left -= STRETCH;
                        if (left <= 0) break;
                        b = count % ACCS;
                        ok = mx4_wait_warp(&acc_full[b], (count / ACCS) & 1, guard);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (!ok) break;
                    b = ACCS;   // the item's sums
                }
                if (CODES) {
                    const uint32_t mask = nan_cols[items % MASKS][q];
                    nan = mask >> lane & 1;
                    __syncwarp();
                    if (lane == 0 && mask) nan_cols[items % MASKS][q] = 0;
                }
            }
#pragma unroll 1
            for (int j0 = 0; j0 < a.rank; j0 += 32) {
                uint32_t v[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(lanes + b * RP + j0, v);
                    tmem_ld_wait();
                }
                const int js = min(32, a.rank - j0);
                if (n == 0 || nan) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = n == 0 ? 0u : 0x7fffffffu;
                }
                if (C > 1) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < js) part[(j0 + j) * GC + 32 * q + lane] = __uint_as_float(v[j]);
                } else if (col < a.C) {
                    const long long at = (static_cast<long long>(g) * a.rank + j0) * a.C + col;
                    if (out_bf16) {
                        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.dw) + at;
#pragma unroll
                        for (int j = 0; j < 32; ++j, p += a.C)
                            if (j < js) *p = __float2bfloat16_rn(__uint_as_float(v[j]));
                    } else {
                        float* p = static_cast<float*>(a.dw) + at;
#pragma unroll
                        for (int j = 0; j < 32; ++j, p += a.C)
                            if (j < js) *p = __uint_as_float(v[j]);
                    }
                }
            }
            if (n > 0) {
                if (b < ACCS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[b]);
                    ++count;
                }
                ++items;
            }
        }
        __syncwarp();
    }
    if (C > 1) {
        // one item a cluster: this block's share of the ranks, summed over the blocks
        cluster_sync();
        const int g = first_g, cb = first_cb;
        constexpr int V = GC / 4;
        const int r1 = a.rank * (rank + 1) / C, c0 = cb * GC + 4 * (tid % V);
        for (int r = a.rank * rank / C + tid / V; r < r1; r += THREADS / V) {
            const uint32_t addr = smem_u32(smem) + (r * GC + 4 * (tid % V)) * 4;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int p = 0; p < C; ++p) {
                const float4 v = ld_shared_cluster_f4(mapa_shared(addr, p));
                s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
            }
            if (c0 >= a.C) continue;
            const long long at = (static_cast<long long>(g) * a.rank + r) * a.C + c0;
            if (out_bf16)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dw) + at) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
            else
                *reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at) = s;
        }
        cluster_sync();   // the others have read this block's sums
    }

    // ---------------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == LOADERS) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

template <int RP, bool CODES, bool ORDER>
cudaError_t launch_cfg(const LoraGradArgs& a, bool out_bf16, int C, int sm_count, uint64_t timeout_ns, cudaStream_t stream) {
    using Cfg = GradCfg<RP, CODES, ORDER>;
    auto kern = lora_grad_kernel<Cfg>;
    const int shm = Cfg::SMEM + (a.G + 1) * static_cast<int>(sizeof(int32_t));
    // one limit for every call: another thread may launch with other groups in between
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg::SMEM + (RDOT_MAX_GROUPS + 1) * static_cast<int>(sizeof(int32_t)));
    if (e != cudaSuccess) return e;
    const int blocks = (a.C + GC - 1) / GC;
    const long long items = static_cast<long long>(a.G) * blocks;
    const long long grid = C > 1 ? items * C : items < sm_count ? items : sm_count;   // a persistent block an SM
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(grid)), dim3(Cfg::THREADS), C, shm, stream, a, blocks, out_bf16, timeout_ns);
}

template <bool CODES, bool ORDER>
cudaError_t launch_rank(const LoraGradArgs& a, bool out_bf16, int C, int sm_count, uint64_t timeout_ns, cudaStream_t stream) {
    if (a.rank <= 16) return launch_cfg<16, CODES, ORDER>(a, out_bf16, C, sm_count, timeout_ns, stream);
    if (a.rank <= 32) return launch_cfg<32, CODES, ORDER>(a, out_bf16, C, sm_count, timeout_ns, stream);
    if (a.rank <= 64) return launch_cfg<64, CODES, ORDER>(a, out_bf16, C, sm_count, timeout_ns, stream);
    return launch_cfg<128, CODES, ORDER>(a, out_bf16, C, sm_count, timeout_ns, stream);
}

}  // namespace

cudaError_t launch_lora_grad(const LoraGradArgs& a, bool codes, bool out_bf16, int sm_count, uint64_t timeout_ns,
                             cudaStream_t stream) {
    const long long groups = a.G < a.M ? a.G : a.M > 0 ? a.M : 1;   // groups that can have a row
    const long long items = groups * ((a.C + GC - 1) / GC);
    const int stages = static_cast<int>((a.M + groups * GR - 1) / (groups * GR));
    // Few items: clusters as large as the SMs hold (one group, rank 16, 16384 rows of 1024 columns: C = 1 79 us, C = 8 20; of
    // 2048: C = 4 30, C = 6 27, C = 8 39; of 4736: C = 2 49, C = 3 43, C = 4 61), unless they save fewer stages than the
    // join costs (8 groups, rank 64, 4096 x 640: C = 1 12.3, C = 2 14.4).
    int C = lora_cluster(items, 1, sm_count);
    while (C > 1 && 2 * C > stages) --C;
    if (stages * (C - 1) < (a.rank <= 64 ? 6 : 10) * C) C = 1;
    if (codes) return a.order ? launch_rank<true, true>(a, out_bf16, C, sm_count, timeout_ns, stream) : launch_rank<true, false>(a, out_bf16, C, sm_count, timeout_ns, stream);
    return a.order ? launch_rank<false, true>(a, out_bf16, C, sm_count, timeout_ns, stream) : launch_rank<false, false>(a, out_bf16, C, sm_count, timeout_ns, stream);
}

cudaError_t lora_grad_status(int32_t** word) {
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_status);
    *word = static_cast<int32_t*>(p);
    return e;
}

}  // namespace rdot
