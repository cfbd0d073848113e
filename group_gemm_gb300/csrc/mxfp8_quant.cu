// mxfp8_quant.cu -- MXFP8 rows: activations kept in 8 bits, quantised and restored.
//
// A block of 32 elements along a row with largest magnitude amax gets the scale 2^e, the smallest power of two
// with amax / 2^e <= 448 (the largest E4M3 number), at least 2^-127; each element is divided by it (exact: a
// power of two) and rounded to E4M3 to nearest even. No element saturates: amax / 2^e lies in (224, 448].
// With E the biased fp32 exponent of amax and m its mantissa, 448 = 1.75 x 2^8 makes the scale byte
// max(E - 8 + (m > 0.75), 0). A block with a NaN or an infinity gets byte 255 and codes 0; it restores as NaN.
//
// One pass each way, HBM-bound: an element is read once, its code or its value written once (16384 x 4096 bf16 and back:
// 65 us, 92 % of a copy's rate).
#include <cuda_bf16.h>

#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace rdot {

namespace {

constexpr int Q8_UNROLL = 4;   // vectors of 8 elements in flight per lane

__device__ __forceinline__ uint32_t scale_byte8(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    const uint32_t e = (amax_bits >> 23) + ((amax_bits & 0x7fffffu) > 0x600000u ? 1u : 0u);
    return e > 8u ? e - 8u : 0u;
}

// Four elements as E4M3 codes, element 0 in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Four lanes hold a block, 8 elements each. A thread block takes Q8_UNROLL * 256 consecutive vectors a pass.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_mxfp8_kernel(const uint4* __restrict__ x, long long vecs, long long step,
                                                             uint2* __restrict__ codes, uint8_t* __restrict__ scales) {
    grid_dependency_enter();
    const long long pass = static_cast<long long>(gridDim.x) * Q8_UNROLL * 256;
    const uint32_t group = 0xfu << (threadIdx.x & 28);   // the four lanes of a block; vecs is a multiple of 4
    const long long first = step == 256 ? static_cast<long long>(blockIdx.x) * Q8_UNROLL * 256 : static_cast<long long>(blockIdx.x) * 256;
    for (long long i0 = first + threadIdx.x; i0 < vecs; i0 += pass) {
        uint4 u[Q8_UNROLL][2];
#pragma unroll
        for (int r = 0; r < Q8_UNROLL; ++r) {
            const long long i = i0 + r * step;
            if (i >= vecs) continue;
            if (BF16) {
                u[r][0] = __ldg(x + i);
            } else {
                u[r][0] = __ldg(x + 2 * i);
                u[r][1] = __ldg(x + 2 * i + 1);
            }
        }
#pragma unroll
        for (int r = 0; r < Q8_UNROLL; ++r) {
            const long long i = i0 + r * step;
            if (i >= vecs) break;
            const uint32_t q[8] = {u[r][0].x, u[r][0].y, u[r][0].z, u[r][0].w, u[r][1].x, u[r][1].y, u[r][1].z, u[r][1].w};
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __uint_as_float(BF16 ? (j & 1 ? q[j >> 1] & 0xffff0000u : q[j >> 1] << 16) : q[j]);
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
            amax = max(amax, __shfl_xor_sync(group, amax, 1));
            amax = max(amax, __shfl_xor_sync(group, amax, 2));
            const uint32_t s = scale_byte8(amax);
            const float inv = s == 255u ? 0.f : __uint_as_float((254u - s) << 23);
            uint2 c = make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                 e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
            if (s == 255u) c = make_uint2(0u, 0u);
            codes[i] = c;
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(s);
        }
    }
}

// 2^(s - 127), 255 NaN; 2^-127 is a subnormal.
__device__ __forceinline__ float scale_f32(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fffffffu : s << 23);
}

// Two E4M3 codes (the low 16 bits) as floats.
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t c) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(c));
    float2 r;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}

template <bool BF16>
__global__ void __launch_bounds__(256) dequantize_mxfp8_kernel(const uint2* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, long long vecs,
                                                               long long step, uint4* __restrict__ out) {
    grid_dependency_enter();
    const long long pass = static_cast<long long>(gridDim.x) * Q8_UNROLL * 256;
    const long long first = step == 256 ? static_cast<long long>(blockIdx.x) * Q8_UNROLL * 256 : static_cast<long long>(blockIdx.x) * 256;
    for (long long i0 = first + threadIdx.x; i0 < vecs; i0 += pass) {
        uint2 u[Q8_UNROLL];
        uint32_t s[Q8_UNROLL];
#pragma unroll
        for (int r = 0; r < Q8_UNROLL; ++r) {
            const long long i = i0 + r * step;
            if (i >= vecs) continue;
            u[r] = __ldg(codes + i);
            s[r] = __ldg(scales + (i >> 2));
        }
#pragma unroll
        for (int r = 0; r < Q8_UNROLL; ++r) {
            const long long i = i0 + r * step;
            if (i >= vecs) break;
            const float f = scale_f32(s[r]);
            float2 v[4] = {e4m3x2_f32(u[r].x), e4m3x2_f32(u[r].x >> 16), e4m3x2_f32(u[r].y), e4m3x2_f32(u[r].y >> 16)};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_float2(v[j].x * f, v[j].y * f);
            if (BF16) {
                out[i] = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                                    pack_bf16x2(v[3].x, v[3].y));
            } else {
                reinterpret_cast<float4*>(out)[2 * i] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
                reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
            }
        }
    }
}

// Blocks of 256 threads for `vecs` vectors, and the distance between a lane's vectors: 256 (a block's vectors are
// consecutive, so that its accesses share DRAM pages) where that fills the grid, else the grid's width.
int grid_for(long long vecs, int sm_count, long long* step) {
    const long long want = (vecs + 255) / 256;
    const int grid = static_cast<int>(want < 16LL * sm_count ? want : 16LL * sm_count);
    *step = vecs >= static_cast<long long>(grid) * Q8_UNROLL * 256 ? 256 : static_cast<long long>(grid) * 256;
    return grid;
}

}  // namespace

cudaError_t launch_quantize_mxfp8(const void* x, bool bf16, long long elements, uint8_t* codes, uint8_t* scales,
                                  int sm_count, cudaStream_t stream) {
    long long step;
    const int grid = grid_for(elements / 8, sm_count, &step);
    auto kern = bf16 ? quantize_mxfp8_kernel<true> : quantize_mxfp8_kernel<false>;
    return launch_pdl(kern, dim3(grid), dim3(256), 0, stream, static_cast<const uint4*>(x), elements / 8, step,
                      reinterpret_cast<uint2*>(codes), scales);
}

cudaError_t launch_dequantize_mxfp8(const uint8_t* codes, const uint8_t* scales, long long elements, void* out,
                                    bool bf16, int sm_count, cudaStream_t stream) {
    long long step;
    const int grid = grid_for(elements / 8, sm_count, &step);
    auto kern = bf16 ? dequantize_mxfp8_kernel<true> : dequantize_mxfp8_kernel<false>;
    return launch_pdl(kern, dim3(grid), dim3(256), 0, stream, reinterpret_cast<const uint2*>(codes), scales, elements / 8,
                      step, static_cast<uint4*>(out));
}

}  // namespace rdot
