// lora_grad.cu -- the gradients of low-rank adapters: dw[g] = t_g^T z_g, a contraction over a group's rows.
//
// With t = scale x down^T the gradient of up is t^T dy, and with dt = scale dy up^T that of down is dt^T x: one
// kernel, [rank x C] sums for each group. z is bf16 or an 8-bit checkpoint (E4M3 codes with a scale per row
// and 32 columns): the codes are widened to bf16 in registers, exactly, between shared memory and the MMA, so
// the activation is never written in 16 bits. The scales do not run along the contraction, so the
// block-scaled MMAs cannot take them.
//
// A block takes 128 columns of a group (each z element is read once; t, C/128 times from L2), a cluster
// divides the group's rows. The fp32 partial sums of its blocks are added through distributed shared memory
// in rank order: no atomics, the same result every time. HBM bounds it.
#include <cuda_bf16.h>

#include "kernels.h"
#include "lora.cuh"
#include "pdl.cuh"

namespace rdot {

namespace {

constexpr int GC = 128;    // columns of a block
constexpr int GR = 64;     // rows of a stage

template <int RP_, bool CODES_>
struct GradCfg {
    static constexpr int RP = RP_;
    static constexpr bool CODES = CODES_;
    static constexpr int ZP = (CODES ? GC : 2 * GC) + 16;   // pitches in bytes, 16 off a multiple of 128
    static constexpr int TP = 2 * RP + 16;
    static constexpr int SCALES = CODES ? GR * 9 + 64 : 0;  // a row: two aligned words that hold its four scales, their place
    static constexpr int SLOT = GR * (ZP + TP) + SCALES;
    static constexpr int STAGES = RP <= 32 ? 4 : 3;
    static constexpr int PP = GC + 4;                       // pitch of the sums (fp32)
    static constexpr int RING = STAGES * SLOT;
    static constexpr int SMEM = RING > RP * PP * 4 ? RING : RP * PP * 4;
};

// Two E4M3 codes (bytes 1 and 3 of v) as bf16 times 2^-120: the exponent and mantissa bits move to the
// bf16 field's low end, subnormals and all.
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t v) { return (v & 0x80008000u) | ((v >> 4) & 0x07f007f0u); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Nonzero where one of four codes is NaN.
__device__ __forceinline__ uint32_t nan_code(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// 2^(s - 127) as bf16, 255 NaN.
__device__ __forceinline__ uint32_t scale_bf16(uint32_t s) { return s == 0u ? 0x0040u : s == 255u ? 0x7fffu : s << 7; }

template <class Cfg>
__global__ void __launch_bounds__(LORA_THREADS) lora_grad_kernel(LoraGradArgs a, int blocks, bool out_bf16) {
    constexpr int RP = Cfg::RP, ZP = Cfg::ZP, TP = Cfg::TP, S = Cfg::STAGES, PP = Cfg::PP;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan_part[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = static_cast<int>(cluster_ctas()), rank = static_cast<int>(cluster_ctarank());
    const int item = static_cast<int>(blockIdx.x) / C;
    const int g = item / blocks, cb = item % blocks;

    grid_dependency_enter();
    // the group's first position: the sizes before it, each at least 0
    long long before = 0;
    for (int i = tid; i < g; i += LORA_THREADS) before += max(__ldg(a.group_sizes + i), 0);
    long long total;
    block_scan128(before, scan_part, &total);
    const int p0 = static_cast<int>(min(total, static_cast<long long>(a.M)));
    const int n = static_cast<int>(min(static_cast<long long>(max(__ldg(a.group_sizes + g), 0)), static_cast<long long>(a.M - p0)));
    const long long all = (static_cast<long long>(n) + GR - 1) / GR;   // stages of the group
    const long long s0 = all * rank / C, s1 = all * (rank + 1) / C;
    const int stages = static_cast<int>(s1 - s0);
    const uint32_t ring = smem_u32(smem);
    const int sb = a.C / 32;   // scales of a row

    // row of z at place q of the group, -1 for none
    const auto row_at = [&](long long q) -> long long {
        if (q >= n) return -1;
        if (!a.order) return p0 + q;
        const int row = __ldg(a.order + p0 + q);
        return row >= 0 && row < a.M ? row : -1;
    };
    const auto load = [&](int i) {
        if (i < stages) {
            constexpr int V = Cfg::CODES ? GC / 16 : GC / 8;   // 16-byte pieces of a row of z
            const uint32_t slot = ring + (i % S) * Cfg::SLOT;
            const long long q0 = (s0 + i) * GR;                // the stage's first row of the group
            const int c0 = cb * GC + (tid % V) * (Cfg::CODES ? 16 : 8);
            constexpr int ESIZE = Cfg::CODES ? 1 : 2;
#pragma unroll
            for (int r = tid / V; r < GR; r += LORA_THREADS / V) {
                const long long row = row_at(q0 + r);
                const bool ok = row >= 0 && c0 < a.C;
                cp_async16(slot + r * ZP + (tid % V) * 16,
                           static_cast<const uint8_t*>(a.z) + (ok ? (row * a.C + c0) * ESIZE : 0), ok);
            }
            constexpr int W = RP / 8;
            for (int e = tid; e < GR * W; e += LORA_THREADS) {
                const int r = e / W, j = 8 * (e % W);
                const bool ok = j < a.rank && row_at(q0 + r) >= 0;
                cp_async16(slot + GR * ZP + r * TP + 2 * j,
                           static_cast<const uint16_t*>(a.t) + (ok ? (p0 + q0 + r) * a.rank + j : 0), ok);
            }
            if (Cfg::CODES) {
                // a row's scales start at any byte: the two aligned words around them, cut at the tensor's end
                const int r = tid >> 1, w = tid & 1;
                const long long row = row_at(q0 + r);
                const long long at = ((row * sb + 4 * cb) & ~3LL) + 4 * w;
                const long long left = static_cast<long long>(a.M) * sb - at;
                const int bytes = row < 0 || left <= 0 ? 0 : left < 4 ? static_cast<int>(left) : 4;
                cp_async4(slot + GR * (ZP + TP) + r * 8 + 4 * w, a.z_scale + (bytes ? at : 0), bytes);
                if (w == 0) smem[(i % S) * Cfg::SLOT + GR * (ZP + TP + 8) + r] = static_cast<uint8_t>((row * sb) & 3);
            }
        }
        cp_async_commit();
    };

    float acc[RP / 16][4][4] = {};
    if (all > 0) {
#pragma unroll
        for (int i = 0; i < S - 1; ++i) load(i);
        for (int i = 0; i < stages; ++i) {
            cp_async_wait<S - 2>();
            __syncthreads();
            load(i + S - 1);
            const uint8_t* slot = smem + (i % S) * Cfg::SLOT;
            const uint32_t zs = smem_u32(slot), ts = zs + GR * ZP;
#pragma unroll
            for (int kk = 0; kk < GR / 16; ++kk) {
                uint32_t fb[4][2];   // z: 16 rows x 32 columns, four tiles of 8
                if (Cfg::CODES) {
                    // lane (q, c): rows 2q, 2q + 1, 2q + 8, 2q + 9; columns 4c .. 4c + 3, column 4c + j in tile j
                    const int q = lane & 3, c = lane >> 2;
                    const uint8_t* p = slot + (16 * kk + 2 * q) * ZP + 32 * warp + 4 * c;
                    uint32_t w[4], sc[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 16 * kk + 2 * q + (j & 1) + 8 * (j >> 1);
                        w[j] = *reinterpret_cast<const uint32_t*>(p + ((j & 1) + 8 * (j >> 1)) * ZP);
                        const int off = (sb & 3) != 0 ? slot[GR * (ZP + TP + 8) + r] : 0;
                        sc[j] = scale_bf16(slot[GR * (ZP + TP) + r * 8 + off + warp]);
                    }
                    const uint32_t up = 0x7b807b80u;   // 2^120 twice
                    const uint32_t sa = sc[0] | sc[1] << 16, sd = sc[2] | sc[3] << 16;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // byte j of two rows to bytes 1 and 3
                        const uint32_t sel = j | j << 4 | (4 + j) << 8 | (4 + j) << 12;
                        fb[j][0] = mul_bf16x2(mul_bf16x2(widen_e4m3x2(__byte_perm(w[0], w[1], sel)), up), sa);
                        fb[j][1] = mul_bf16x2(mul_bf16x2(widen_e4m3x2(__byte_perm(w[2], w[3], sel)), up), sd);
                    }
                    if (nan_code(w[0]) | nan_code(w[1]) | nan_code(w[2]) | nan_code(w[3])) {
                        // code 0x7f or 0xff is NaN (the quantiser writes none)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if ((w[k] >> (8 * j) & 0x7fu) == 0x7fu) fb[j][k >> 1] |= 0x7fffu << (16 * (k & 1));
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t f[4];
                        ldmatrix_x4_trans(f, zs + (16 * kk + (lane & 15)) * ZP + (32 * warp + 16 * h + 8 * (lane >> 4)) * 2);
                        fb[2 * h][0] = f[0];
                        fb[2 * h][1] = f[1];
                        fb[2 * h + 1][0] = f[2];
                        fb[2 * h + 1][1] = f[3];
                    }
                }
#pragma unroll
                for (int m = 0; m < RP / 16; ++m) {
                    // t^T: 16 ranks x 16 rows
                    uint32_t fa[4];
                    ldmatrix_x4_trans(fa, ts + (16 * kk + (lane & 7) + ((lane >> 4) << 3)) * TP +
                                              (16 * m + 8 * ((lane >> 3) & 1)) * 2);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_16816(acc[m][j], fa, fb[j][0], fb[j][1]);
                }
            }
        }
        cp_async_wait<0>();
        __syncthreads();   // the ring becomes the sums
        float* sums = reinterpret_cast<float*>(smem);
        const int q = lane & 3;
#pragma unroll
        for (int m = 0; m < RP / 16; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float* row = sums + (16 * m + (lane >> 2) + 8 * half) * PP + 32 * warp;
                if (Cfg::CODES) {   // columns 2q and 2q + 1 of tile j: 8q + j, 8q + 4 + j
                    *reinterpret_cast<float4*>(row + 8 * q) =
                        make_float4(acc[m][0][2 * half], acc[m][1][2 * half], acc[m][2][2 * half], acc[m][3][2 * half]);
                    *reinterpret_cast<float4*>(row + 8 * q + 4) = make_float4(
                        acc[m][0][2 * half + 1], acc[m][1][2 * half + 1], acc[m][2][2 * half + 1], acc[m][3][2 * half + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float2*>(row + 8 * j + 2 * q) = make_float2(acc[m][j][2 * half], acc[m][j][2 * half + 1]);
                }
            }
        if (C > 1) cluster_sync();
        else __syncthreads();
    }
    // this block's share of the rows of dw[g], zeros for an empty group
    constexpr int V = GC / 4;
    const int r0 = a.rank * rank / C, r1 = a.rank * (rank + 1) / C;
    const int c0 = cb * GC + 4 * (tid % V);
    for (int r = r0 + tid / V; r < r1; r += LORA_THREADS / V) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (all > 0) {
            const uint32_t addr = smem_u32(smem) + (r * PP + 4 * (tid % V)) * 4;
#pragma unroll 4
            for (int q = 0; q < C; ++q) {
                const float4 v = ld_shared_cluster_f4(mapa_shared(addr, q));
                s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
            }
        }
        if (c0 >= a.C) continue;
        const long long at = (static_cast<long long>(g) * a.rank + r) * a.C + c0;
        if (out_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dw) + at) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at) = s;
    }
    if (all > 0 && C > 1) cluster_sync();   // the others have read this block's sums
}

template <int RP, bool CODES>
cudaError_t launch_cfg(const LoraGradArgs& a, bool out_bf16, int C, cudaStream_t stream) {
    using Cfg = GradCfg<RP, CODES>;
    auto kern = lora_grad_kernel<Cfg>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    const int blocks = (a.C + GC - 1) / GC;
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(static_cast<long long>(a.G) * blocks * C)),
                              dim3(LORA_THREADS), C, Cfg::SMEM, stream, a, blocks, out_bf16);
}

template <bool CODES>
cudaError_t launch_codes(const LoraGradArgs& a, bool out_bf16, int C, cudaStream_t stream) {
    if (a.rank <= 16) return launch_cfg<16, CODES>(a, out_bf16, C, stream);
    if (a.rank <= 32) return launch_cfg<32, CODES>(a, out_bf16, C, stream);
    if (a.rank <= 64) return launch_cfg<64, CODES>(a, out_bf16, C, stream);
    return launch_cfg<128, CODES>(a, out_bf16, C, stream);
}

}  // namespace

cudaError_t launch_lora_grad(const LoraGradArgs& a, bool codes, bool out_bf16, int sm_count, cudaStream_t stream) {
    const long long groups = a.G < a.M ? a.G : a.M > 0 ? a.M : 1;   // groups that can have a row
    const long long items = groups * ((a.C + GC - 1) / GC);
    const long long stages = (a.M + groups * GR - 1) / (groups * GR);
    int C = 1;
    while (C < 8 && items * C * 2 <= 4LL * sm_count && 2 * C <= stages) C *= 2;
    return codes ? launch_codes<true>(a, out_bf16, C, stream) : launch_codes<false>(a, out_bf16, C, stream);
}

}  // namespace rdot
