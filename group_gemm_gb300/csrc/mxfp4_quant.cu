// mxfp4_quant.cu -- MXFP4 quantisation of activation rows and of a layer's weights.
//
// Rule (OCP Microscaling Formats v1.0): a block of 32 elements along the contraction with largest
// magnitude amax gets the scale 2^(floor(log2 amax) - 2), at least 2^-127 (2 = the largest E2M1
// exponent); each element is divided by it (exact: a power of two), rounded to E2M1 to nearest even
// and saturated at 6, its sign kept. With E the biased fp32 exponent of amax the scale byte is
// max(E - 2, 0). A block with a NaN or an infinity has no finite scale: byte 255, codes 0, values NaN.
// The optional values, code x scale, are bf16 without rounding: two significant bits and exponents
// from -128 to 127 fit it (its subnormals reach 2^-133).
//
// Both kernels are one-pass streams: each element is read once. HBM bounds rows (16384 x 4096 bf16 with
// values 47.1 us, 6.5 TB/s, codes alone 28.6 us) and fp32 weights; bf16 weights stay below it (figures at
// the kernel).
#include <cuda_bf16.h>

#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace rdot {

namespace {

// Scale byte of a block from the largest |x| as fp32 bits (NaN and infinity compare above all numbers).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    const uint32_t e = amax_bits >> 23;
    return e > 2u ? e - 2u : 0u;
}

// 2^(127 - s) as fp32; s <= 252.
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Eight elements (already divided by the scale) as E2M1 codes, element 0 in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The values of the four E2M1 codes in the low 16 bits of c as bf16 pairs (codes 0, 1 and 2, 3). The
// magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6 are the bf16 words 0000 3F00 3F80 3FC0 4000 4040 4080 40C0: a byte
// permute picks four high bytes, another four low bytes, by the codes' low three bits.
__device__ __forceinline__ uint2 e2m1x4_bf16(uint32_t c) {
    const uint32_t m = c & 0x7777u;
    const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, m), lo = __byte_perm(0xc0800000u, 0xc0804000u, m);
    return make_uint2(__byte_perm(lo, hi, 0x5140u) | ((c << 12) & 0x8000u) | ((c << 24) & 0x80000000u),
                      __byte_perm(lo, hi, 0x7362u) | ((c << 4) & 0x8000u) | ((c << 16) & 0x80000000u));
}

// A bf16 pair times 2^(s-127) (NaN for s = 255), exact: the products have two significant bits and
// bf16 multiplication keeps subnormals.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t v, uint32_t scale2) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(scale2));
    return r;
}

// 2^(s-127) twice as a bf16 pair: the exponent field is s, 2^-127 a subnormal, 255 NaN.
__device__ __forceinline__ uint32_t scale_pair(uint32_t s) {
    const uint32_t w = s == 0u ? 0x0040u : s == 255u ? 0x7fffu : s << 7;
    return w | (w << 16);
}

__device__ __forceinline__ float unpack_bf16(uint32_t w, int hi) {
    return __uint_as_float(hi ? (w & 0xffff0000u) : (w << 16));
}

// Rows: the blocks of all rows are consecutive, so the tensor is one array of 32-element blocks. Four
// lanes hold a block, 8 elements each.
constexpr int QR_UNROLL = 4;   // vectors of 8 elements in flight per lane

template <bool BF16>
__device__ __forceinline__ void load_vec8(const uint4* __restrict__ x, long long i, uint4 (&u)[2]) {
    if (BF16) {
        u[0] = __ldg(x + i);
    } else {
        u[0] = __ldg(x + 2 * i);
        u[1] = __ldg(x + 2 * i + 1);
    }
}

// CHUNKS: a block takes QR_UNROLL * 256 consecutive vectors a pass, so that its loads and stores share DRAM
// pages (16384 x 4096 bf16 with values: 47.1 against 48.6 us, codes alone 28.6 / 30.2); without, they are spread over
// the grid, so that more blocks share a small input (37 x 1408 fp32: 1.3 against 2.3 us). The launch takes
// chunks where they fill the grid, from 4864 rows of 4096: there 16.1 against 15.7 us, at 5500 rows 17.3 / 17.7.
// They also win below that (2432 rows 9.4 / 9.7, 1216 rows 5.9 / 6.4), so the border could lie lower.
template <bool BF16, bool VALUES, bool CHUNKS>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint4* __restrict__ x, long long vecs,
                                                            uint32_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales,
                                                            uint4* __restrict__ values) {
    grid_dependency_enter();
    const long long pass = static_cast<long long>(gridDim.x) * QR_UNROLL * 256;
    const long long step = CHUNKS ? 256 : static_cast<long long>(gridDim.x) * 256;
    const uint32_t group = 0xfu << (threadIdx.x & 28);   // the four lanes of a block; vecs is a multiple of 4
    for (long long i0 = static_cast<long long>(blockIdx.x) * (CHUNKS ? QR_UNROLL * 256 : 256) + threadIdx.x; i0 < vecs;
         i0 += pass) {
        uint4 u[QR_UNROLL][2];
#pragma unroll
        for (int r = 0; r < QR_UNROLL; ++r)
            if (i0 + r * step < vecs) load_vec8<BF16>(x, i0 + r * step, u[r]);
#pragma unroll
        for (int r = 0; r < QR_UNROLL; ++r) {
            const long long i = i0 + r * step;
            if (i >= vecs) break;
            const uint32_t q[8] = {u[r][0].x, u[r][0].y, u[r][0].z, u[r][0].w, u[r][1].x, u[r][1].y, u[r][1].z, u[r][1].w};
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = BF16 ? unpack_bf16(q[j >> 1], j & 1) : __uint_as_float(q[j]);
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
            amax = max(amax, __shfl_xor_sync(group, amax, 1));
            amax = max(amax, __shfl_xor_sync(group, amax, 2));
            const uint32_t s = scale_byte(amax);
            const bool nan = s == 255u;
            const float inv = nan ? 0.f : inverse_scale(s);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= inv;
            const uint32_t c = nan ? 0u : e2m1x8(v);
            codes[i] = c;
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(s);
            if (VALUES) {
                const uint32_t sv = scale_pair(s);
                const uint2 lo = e2m1x4_bf16(c), hi = e2m1x4_bf16(c >> 16);
                values[i] = make_uint4(scale_bf16x2(lo.x, sv), scale_bf16x2(lo.y, sv), scale_bf16x2(hi.x, sv),
                                       scale_bf16x2(hi.y, sv));
            }
        }
    }
}

// Weights [G, K, N] -> codes [G, N, K/2] and scale atoms. A block of 4 warps takes 64 columns x 128 rows of
// one group: warp w the 32 rows of scale block w, lane l columns 2l and 2l + 1, so a scale block of a
// column lies in one thread's registers (all 32 loads in flight); the codes are turned through shared
// memory into rows of up to 64 bytes, the scales into one atom's words. Four such blocks share an SM and
// so load, compute and store at different times: 456 us (6.7 TB/s) for 8 x 4096 x 14336 fp32 with
// values, against 568 us for two blocks of 8 warps, 642 us for one of 16, and 599 us for five of 4. With values
// the kernel uses the 128 registers that four blocks leave and spills 52 bytes a thread (bf16: 48); five
// blocks leave 96 and spill 240. Codes alone (no spills): fp32 304 us, bf16 209 (floor 175). bf16 with values
// is the form farthest from its floor: 499 us against 313; a lane loads 4 bytes there, half the bytes in flight.
constexpr int QW_COLS = 64;
constexpr int QW_BLOCKS = 4;    // scale blocks (32 rows each) per thread block
constexpr int QW_THREADS = 32 * QW_BLOCKS;
constexpr int QW_PITCH = 16 * QW_BLOCKS + 16;   // shared bytes of a column's codes plus 16 against bank conflicts

template <bool BF16, bool VALUES>
__global__ void __launch_bounds__(QW_THREADS, 512 / QW_THREADS) quantize_weight_kernel(const void* __restrict__ w, int K, int N, int NT, int KC,
                                                              uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales,
                                                              uint32_t* __restrict__ values) {
    __shared__ __align__(16) uint8_t tile[QW_COLS * QW_PITCH];
    __shared__ __align__(8) uint8_t sc[QW_COLS][QW_BLOCKS];   // read as words of 4
    grid_dependency_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kc = blockIdx.x % KC;
    const int nt = (blockIdx.x / KC) % NT;
    const long long g = blockIdx.x / KC / NT;
    const int KB = K / 32;
    const int kb = kc * QW_BLOCKS + warp;
    const int n = nt * QW_COLS + 2 * lane;   // N is even: both columns are inside or both past it
    const bool live = kb < KB && n < N;
    uint32_t s0 = 0, s1 = 0;
    if (live) {
        const long long base = (g * K + 32LL * kb) * N + n;   // element index of (row 0, column n)
        float c0[32], c1[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            if (BF16) {
                const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(w) + ((base + static_cast<long long>(r) * N) >> 1));
                c0[r] = unpack_bf16(u, 0);
                c1[r] = unpack_bf16(u, 1);
            } else {
                const float2 u = __ldg(reinterpret_cast<const float2*>(w) + ((base + static_cast<long long>(r) * N) >> 1));
                c0[r] = u.x;
                c1[r] = u.y;
            }
        }
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            m0 = max(m0, __float_as_uint(c0[r]) & 0x7fffffffu);
            m1 = max(m1, __float_as_uint(c1[r]) & 0x7fffffffu);
        }
        s0 = scale_byte(m0);
        s1 = scale_byte(m1);
        const bool nan0 = s0 == 255u, nan1 = s1 == 255u;
        const float i0 = nan0 ? 0.f : inverse_scale(s0), i1 = nan1 ? 0.f : inverse_scale(s1);
        const uint32_t sv = __byte_perm(scale_pair(s0), scale_pair(s1), 0x5410u);   // column 0's, column 1's
        uint32_t q0[4], q1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a[8], b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] = c0[8 * i + j] * i0;
                b[j] = c1[8 * i + j] * i1;
            }
            q0[i] = nan0 ? 0u : e2m1x8(a);
            q1[i] = nan1 ? 0u : e2m1x8(b);
            if (VALUES) {
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    // four rows of each column, then turned into (column 0, column 1) pairs
                    const uint2 x0 = e2m1x4_bf16(q0[i] >> (4 * j)), x1 = e2m1x4_bf16(q1[i] >> (4 * j));
                    const uint32_t rows[4] = {__byte_perm(x0.x, x1.x, 0x5410u), __byte_perm(x0.x, x1.x, 0x7632u),
                                              __byte_perm(x0.y, x1.y, 0x5410u), __byte_perm(x0.y, x1.y, 0x7632u)};
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        values[(base + static_cast<long long>(8 * i + j + r) * N) >> 1] = scale_bf16x2(rows[r], sv);
                }
            }
        }
        *reinterpret_cast<uint4*>(tile + (2 * lane) * QW_PITCH + 16 * warp) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
        *reinterpret_cast<uint4*>(tile + (2 * lane + 1) * QW_PITCH + 16 * warp) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
    }
    sc[2 * lane][warp] = static_cast<uint8_t>(s0);       // 0 past K and N
    sc[2 * lane + 1][warp] = static_cast<uint8_t>(s1);
    __syncthreads();
    // codes: 32 bytes (two scale blocks of a column) a thread
    {
        const int c = threadIdx.x / (QW_BLOCKS / 2), part = threadIdx.x % (QW_BLOCKS / 2);
        const int col = nt * QW_COLS + c;
        if (col < N) {
            uint4* dst = reinterpret_cast<uint4*>(codes + ((g * N + col) * KB + kc * QW_BLOCKS) * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int b = 2 * part + i;
                if (kc * QW_BLOCKS + b < KB) dst[b] = *reinterpret_cast<const uint4*>(tile + c * QW_PITCH + 16 * b);
            }
        }
    }
    // scales: one 4-byte word per column and atom of 4 blocks
    if (threadIdx.x < QW_BLOCKS / 4 * QW_COLS) {
        const int c = threadIdx.x & (QW_COLS - 1), half = threadIdx.x / QW_COLS;
        const int KA = (KB + 3) / 4, NB = (N + 127) / 128;
        const int ka = kc * (QW_BLOCKS / 4) + half;
        const int col = (nt * QW_COLS + c) & 127;
        if (ka < KA) {
            uint8_t* atom = scales + ((g * NB + nt / 2) * KA + ka) * 512;
            *reinterpret_cast<uint32_t*>(atom + 16 * (col & 31) + 4 * (col >> 5)) =
                *reinterpret_cast<const uint32_t*>(&sc[c][4 * half]);
        }
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, bool bf16, long long elements, uint8_t* codes, uint8_t* scales,
                                 void* values, int sm_count, cudaStream_t stream) {
    const long long vecs = elements / 8;
    const long long want = (vecs + 255) / 256;
    const int grid = static_cast<int>(want < 16LL * sm_count ? want : 16LL * sm_count);
    const auto launch = [&](auto kern) {
        return launch_pdl(kern, dim3(grid), dim3(256), 0, stream, static_cast<const uint4*>(x), vecs,
                          reinterpret_cast<uint32_t*>(codes), scales, static_cast<uint4*>(values));
    };
    if (vecs >= static_cast<long long>(grid) * QR_UNROLL * 256) {
        if (bf16) return values ? launch(quantize_rows_kernel<true, true, true>) : launch(quantize_rows_kernel<true, false, true>);
        return values ? launch(quantize_rows_kernel<false, true, true>) : launch(quantize_rows_kernel<false, false, true>);
    }
    if (bf16) return values ? launch(quantize_rows_kernel<true, true, false>) : launch(quantize_rows_kernel<true, false, false>);
    return values ? launch(quantize_rows_kernel<false, true, false>) : launch(quantize_rows_kernel<false, false, false>);
}

cudaError_t launch_quantize_weight(const void* w, bool bf16, int groups, int K, int N, uint8_t* codes, uint8_t* scales,
                                   void* values, cudaStream_t stream) {
    const int NT = 2 * ((N + 127) / 128);   // both halves of every 128-column atom
    const int KC = (K / 32 + QW_BLOCKS - 1) / QW_BLOCKS;
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(groups) * NT * KC));
    auto kern = bf16 ? (values ? quantize_weight_kernel<true, true> : quantize_weight_kernel<true, false>)
                     : (values ? quantize_weight_kernel<false, true> : quantize_weight_kernel<false, false>);
    return launch_pdl(kern, grid, dim3(QW_THREADS), 0, stream, w, K, N, NT, KC, codes, scales, static_cast<uint32_t*>(values));
}

}  // namespace rdot
