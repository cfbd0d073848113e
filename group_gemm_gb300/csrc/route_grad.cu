// route_grad.cu -- the gradients of the routing steps of route.cu: permute, un-permute, router top-k.
//
// With order / inv the index outputs of the permute (row p of the sorted order holds copy order[p] =
// t*k + j, inv the other way round, -1 for none):
//   un-permute  out[t] = sum_j w[t,j] y[inv[t,j]]    dy[p] = w[order[p]] dout[order[p] / k]
//                                                   dw[t,j] = <dout[t], y[inv[t,j]]>
//   permute     x_sorted[p] = x[order[p] / k]        dx[t] = sum_j dx_sorted[inv[t,j]]
//   router      w = top-k logits, or their softmax   dlogits, see router_topk_grad_kernel
// HBM bounds the first two: rows move as 16-byte vectors, each row of y and dx_sorted is read once and each
// output row written once; dout[t] is read for each of its k copies, again from L2. Latency bounds the router's:
// 4096 x 256 takes 2.8 us for 1.3 us of HBM time. Sums are kept in fp32 in a fixed order (no atomics).
#include <cuda_bf16.h>

#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace rdot {

namespace {

constexpr int VEC_UNROLL = 4;   // 16-byte loads in flight per lane and operand

// One 16-byte vector of E elements as fp32: 8 bf16 or 4 fp32.
template <bool BF16>
struct Vec {
    static constexpr int E = BF16 ? 8 : 4;
    __device__ __forceinline__ static void unpack(uint4 u, float (&f)[E]) {
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                f[2 * i] = __uint_as_float(q[i] << 16);
                f[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
            } else {
                f[i] = __uint_as_float(q[i]);
            }
        }
    }
    // fp32 sums or products, rounded to the output type once, to nearest even
    __device__ __forceinline__ static uint4 pack(const float (&f)[E]) {
        if constexpr (BF16)
            return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                              pack_bf16x2(f[6], f[7]));
        else
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

int warps_grid(long long warps, int sm_count) {
    const long long want = (warps + 7) / 8;
    return static_cast<int>(want < 8LL * sm_count ? want : 8LL * sm_count);
}

// WARPS warps per J copies f = t*k + j, j + 1, ...: reads dout[t] and y[inv[f]], writes dy[inv[f]] and dw[f];
// then zeroes row f of dy if no copy is placed there. Index values outside [0, T*k) count as none. One warp
// a copy streams best when the copies fill the GPU (8192 tokens top-2, rows of 4096: 51.0 us, 6.6 TB/s), two
// copies at once where a row gives a lane fewer than four vectors (rows of 512, 16384 tokens top-8: 52.6
// against 67.2 us); a whole block a copy when they do not (61 tokens top-8, rows of 7168: 3.4 against
// 7.4 us).
template <int WARPS, int U, int J>
__global__ void __launch_bounds__(256) unpermute_grad_kernel(const uint4* __restrict__ dout,
                                                             const uint4* __restrict__ y,
                                                             const int32_t* __restrict__ order,
                                                             const int32_t* __restrict__ inv,
                                                             const float* __restrict__ w, long long total, int k,
                                                             int vec_per_row, uint4* __restrict__ dy,
                                                             float* __restrict__ dw) {
    static_assert(WARPS == 1 || (WARPS == 8 && J == 1), "a warp per J copies or a block per copy");
    __shared__ float part[8];
    grid_dependency_enter();
    constexpr int STEP = 32 * WARPS;   // threads of a copy
    const int lane = threadIdx.x & 31;
    const int sub = threadIdx.x % STEP;
    const long long first = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / STEP * J;
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x / STEP * J;
    // the next copies' indices and weights are in flight while these copies' rows move
    int32_t pn[J], on[J];
    float wn[J];
    const auto fetch = [&](long long f0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            pn[j] = on[j] = -1;
            wn[j] = 0.f;
            if (f0 + j >= total) continue;
            pn[j] = __ldg(inv + f0 + j);
            on[j] = __ldg(order + f0 + j);
            wn[j] = __ldg(w + f0 + j);
        }
    };
    fetch(first);
    for (long long f0 = first; f0 < total; f0 += stride) {
        int32_t p[J], o[J];
        float wf[J], dot[J];
        bool kept[J], any = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            p[j] = pn[j];
            o[j] = on[j];
            wf[j] = wn[j];
            dot[j] = 0.f;
            kept[j] = p[j] >= 0 && p[j] < total;
            any = any || kept[j];
        }
        fetch(f0 + stride);
        if (any) {
            for (int i0 = sub; i0 < vec_per_row; i0 += STEP * U) {
                uint4 a[J][U], b[J][U];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const uint4* d = dout + (f0 + j) / k * vec_per_row;
                    const uint4* src = y + static_cast<long long>(p[j]) * vec_per_row;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (kept[j] && i0 + STEP * u < vec_per_row) {
                            a[j][u] = __ldg(d + i0 + STEP * u);
                            b[j][u] = __ldg(src + i0 + STEP * u);
                        }
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (!kept[j]) continue;
                    uint4* dst = dy + static_cast<long long>(p[j]) * vec_per_row;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (i0 + STEP * u >= vec_per_row) continue;
                        float x[8], v[8];
                        Vec<true>::unpack(a[j][u], x);
                        Vec<true>::unpack(b[j][u], v);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            dot[j] += x[c] * v[c];
                            x[c] *= wf[j];
                        }
                        dst[i0 + STEP * u] = Vec<true>::pack(x);
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < J; ++j) dot[j] = warp_sum(dot[j]);
        }
        if constexpr (WARPS > 1) {   // f0 is the same for the whole block
            if (lane == 0) part[threadIdx.x >> 5] = dot[0];
            __syncthreads();
            dot[0] = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) dot[0] += part[i];
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (f0 + j >= total) continue;
            if (sub == 0) dw[f0 + j] = dot[j];
            if (o[j] < 0 || o[j] >= total)
                for (int i = sub; i < vec_per_row; i += STEP) dy[(f0 + j) * vec_per_row + i] = make_uint4(0, 0, 0, 0);
        }
    }
}

template <int WARPS, int U, int J>
cudaError_t launch_unpermute_grad(const void* dout, const void* y_sorted, const int32_t* order, const int32_t* inv,
                                  const float* weights, long long total, int k, int vec, void* dy_sorted,
                                  float* dweights, int sm_count, cudaStream_t stream) {
    const int grid = warps_grid((total + J - 1) / J * WARPS, sm_count);
    return launch_pdl(unpermute_grad_kernel<WARPS, U, J>, dim3(grid), dim3(256), 0, stream,
                      static_cast<const uint4*>(dout), static_cast<const uint4*>(y_sorted), order, inv, weights, total, k,
                      vec, static_cast<uint4*>(dy_sorted), dweights);
}

// One warp per (token, 32 U vectors of its row): sums the kept copies' vectors in fp32, J copies' loads in
// flight together. Rows of 4096 bf16: U = 2, J = 4 takes 88.9 us for 8192 tokens top-8 (6.8 TB/s) against
// 95.2 with U = 4, J = 1, but 56.1 against 42.5 for 16384 tokens top-1; U = 2, J = 2 59.2 against 62.4 for top-2.
template <bool BF16, int U, int J>
__global__ void __launch_bounds__(256) permute_grad_kernel(const uint4* __restrict__ dxs,
                                                           const int32_t* __restrict__ inv, long long tokens, int k,
                                                           int vec_per_row, uint4* __restrict__ dx) {
    using V = Vec<BF16>;
    grid_dependency_enter();
    const int lane = threadIdx.x & 31;
    const long long warp = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
    const long long chunks = (vec_per_row + 32 * U - 1) / (32 * U);
    const long long total = tokens * k;
    for (long long it = warp; it < tokens * chunks; it += nwarps) {
        const long long t = it / chunks;
        const int i0 = static_cast<int>(it - t * chunks) * 32 * U + lane;
        float a[U][V::E];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < V::E; ++c) a[u][c] = 0.f;
        for (int j0 = 0; j0 < k; j0 += J) {
            uint4 v[J][U];
            bool live[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int32_t p = j0 + j < k ? __ldg(inv + t * k + j0 + j) : -1;
                live[j] = p >= 0 && p < total;
                const uint4* src = dxs + static_cast<long long>(live[j] ? p : 0) * vec_per_row + i0;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (live[j] && i0 + 32 * u < vec_per_row) v[j][u] = __ldg(src + 32 * u);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!live[j]) continue;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i0 + 32 * u >= vec_per_row) continue;
                    float x[V::E];
                    V::unpack(v[j][u], x);
#pragma unroll
                    for (int c = 0; c < V::E; ++c) a[u][c] += x[c];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + 32 * u < vec_per_row) dx[t * vec_per_row + i0 + 32 * u] = V::pack(a[u]);
    }
}

template <bool BF16, int U, int J>
cudaError_t launch_permute_grad(const void* dx_sorted, const int32_t* inv, long long tokens, int k, int vec, void* dx,
                                int sm_count, cudaStream_t stream) {
    const long long warps = tokens * ((vec + 32 * U - 1) / (32 * U));
    return launch_pdl(permute_grad_kernel<BF16, U, J>, dim3(warps_grid(warps, sm_count)), dim3(256), 0, stream,
                      static_cast<const uint4*>(dx_sorted), inv, tokens, k, vec, static_cast<uint4*>(dx));
}

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* p, long long i) {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short*>(p) + i)) << 16);
    return __ldg(static_cast<const float*>(p) + i);
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void* p, long long i, float v) {
    if (BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
}

// One warp per token. With e_j the token's k experts, w_j the router's weights, g_j their gradients
// and s = sum_j w_j g_j:
//   values        dl[e_j] = g_j
//   softmax       dl[e]   = [e = e_j] w_j g_j - p_e s,  p = softmax over all E logits (recomputed)
//   softmax_topk  dl[e_j] = w_j (g_j - s)
// and zero for the other experts. Lane j holds copy j's expert and its term; lane l the logits of
// experts l, l + 32, ..., IPL of them, read once. Above 64 experts the terms reach their experts' lanes
// through a row of shared memory per warp (comparing every expert with every copy's takes most of the
// instructions: 8192 tokens x 1024, top-32: 19.0 against 33.3 us); copies of the same expert, which the
// router never makes, are added up in copy order. Above 256 experts the kernel is far from HBM (8192 x 1024
// fp32: 19.0 us against 10.4): 101 registers a thread and 32 KB of shared memory a block leave two blocks an
// SM, and the next token's logits are not fetched ahead.
template <int IPL, bool BF16>
__global__ void __launch_bounds__(256) router_topk_grad_kernel(const void* __restrict__ logits,
                                                               const int32_t* __restrict__ ids,
                                                               const float* __restrict__ w,
                                                               const float* __restrict__ dw, long long tokens, int E,
                                                               int k, int mode, void* __restrict__ dlogits) {
    constexpr bool SCATTER = IPL > 2;
    constexpr bool AHEAD = IPL <= 8;   // more logits a lane ahead cost the occupancy (E = 1024: 27.1 us against 19.0)
    __shared__ float rows[8][SCATTER ? 32 * IPL : 1];
    grid_dependency_enter();
    const int lane = threadIdx.x & 31;
    float* row = rows[threadIdx.x >> 5];
    const long long warp = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
    if (SCATTER) {
#pragma unroll
        for (int i = 0; i < IPL; ++i) row[lane + 32 * i] = 0.f;
    }
    // the next token's inputs are in flight while this one is worked on
    float vn[AHEAD ? IPL : 1], wn = 0.f, gn = 0.f;
    int idn = -1;
    const auto fetch = [&](long long t) {
        if (t >= tokens) return;
        if (AHEAD && mode == RDOT_ROUTER_SOFTMAX) {
#pragma unroll
            for (int i = 0; i < (AHEAD ? IPL : 1); ++i)
                vn[i] = lane + 32 * i < E ? load_elem<BF16>(logits, t * E + lane + 32 * i) : -INFINITY;
        }
        if (lane < k) {
            idn = __ldg(ids + t * k + lane);
            wn = __ldg(w + t * k + lane);
            gn = __ldg(dw + t * k + lane);
        }
    };
    fetch(warp);
    for (long long t = warp; t < tokens; t += nwarps) {
        float v[IPL];
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            v[i] = 0.f;
            if (mode != RDOT_ROUTER_SOFTMAX) continue;
            if constexpr (AHEAD) v[i] = vn[i];
            else v[i] = lane + 32 * i < E ? load_elem<BF16>(logits, t * E + lane + 32 * i) : -INFINITY;
        }
        const int id = idn;
        const float wj = wn, gj = gn;
        fetch(t + nwarps);
        const float s = mode == RDOT_ROUTER_VALUES ? 0.f : warp_sum(wj * gj);
        const float term = mode == RDOT_ROUTER_VALUES ? gj : mode == RDOT_ROUTER_SOFTMAX ? wj * gj : wj * (gj - s);
        if (mode == RDOT_ROUTER_SOFTMAX) {
            float m = v[0];
#pragma unroll
            for (int i = 1; i < IPL; ++i) m = fmaxf(m, v[i]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < IPL; ++i) {
                v[i] = lane + 32 * i < E ? expf(v[i] - m) : 0.f;
                sum += v[i];
            }
            const float scale = -s / warp_sum(sum);
#pragma unroll
            for (int i = 0; i < IPL; ++i) v[i] *= scale;
        }
        if (SCATTER) {
            const bool inside = id >= 0 && id < E;
            // a copy whose lane number another copy of the same expert has overwritten: add them up in order
            __syncwarp();
            if (inside) row[id] = __int_as_float(lane);
            __syncwarp();
            const bool alone = !inside || __float_as_int(row[id]) == lane;
            float sum = term;
            if (!__all_sync(0xffffffffu, alone)) {
                sum = 0.f;
                for (int j = 0; j < k; ++j) {
                    const int ej = __shfl_sync(0xffffffffu, id, j);
                    const float tj = __shfl_sync(0xffffffffu, term, j);
                    if (ej == id) sum += tj;
                }
            }
            if (inside) row[id] = sum;   // the same value from every copy of one expert
            __syncwarp();
#pragma unroll
            for (int i = 0; i < IPL; ++i) v[i] += row[lane + 32 * i];
            __syncwarp();
            if (inside) row[id] = 0.f;   // zero again for the next token
        } else {
            for (int j = 0; j < k; ++j) {
                const int ej = __shfl_sync(0xffffffffu, id, j);
                const float tj = __shfl_sync(0xffffffffu, term, j);
#pragma unroll
                for (int i = 0; i < IPL; ++i)
                    if (ej == lane + 32 * i) v[i] += tj;
            }
        }
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            if (lane + 32 * i < E) store_elem<BF16>(dlogits, t * E + lane + 32 * i, v[i]);
    }
}

template <int IPL>
cudaError_t launch_topk_grad_ipl(const void* logits, bool bf16, const int32_t* ids, const float* weights,
                                 const float* dweights, long long tokens, int E, int k, int mode, void* dlogits, int grid,
                                 cudaStream_t stream) {
    auto kern = bf16 ? router_topk_grad_kernel<IPL, true> : router_topk_grad_kernel<IPL, false>;
    return launch_pdl(kern, dim3(grid), dim3(256), 0, stream, logits, ids, weights, dweights, tokens, E, k, mode, dlogits);
}

}  // namespace

cudaError_t launch_moe_unpermute_grad(const void* dout, const void* y_sorted, const int32_t* order, const int32_t* inv,
                                      const float* weights, long long tokens, int k, long long n, void* dy_sorted,
                                      float* dweights, int sm_count, cudaStream_t stream) {
    const long long total = tokens * k;
    // a block per copy while the copies are few for the length of their rows (measured on both sides:
    // rows of 7168, 2048 copies 12.8 against 14.9 us; of 4096, 122 copies 2.2 / 4.2, 2048 copies 10.4 / 9.3; of
    // 1024, 3200 copies 6.9 / 3.1)
    const int vec = static_cast<int>(n / 8);
    const bool block = total * 64 < static_cast<long long>(vec) * sm_count;
    const auto launch = block       ? launch_unpermute_grad<8, VEC_UNROLL, 1>
                        : vec < 128 ? launch_unpermute_grad<1, 2, 2>
                                    : launch_unpermute_grad<1, VEC_UNROLL, 1>;
    return launch(dout, y_sorted, order, inv, weights, total, k, vec, dy_sorted, dweights, sm_count, stream);
}

cudaError_t launch_moe_permute_grad(const void* dx_sorted, bool bf16, const int32_t* inv, long long tokens, int k,
                                    long long n, void* dx, int sm_count, cudaStream_t stream) {
    const int vec = static_cast<int>(n / (bf16 ? 8 : 4));
    if (k == 1)
        return bf16 ? launch_permute_grad<true, 4, 1>(dx_sorted, inv, tokens, k, vec, dx, sm_count, stream)
                    : launch_permute_grad<false, 4, 1>(dx_sorted, inv, tokens, k, vec, dx, sm_count, stream);
    if (k == 2)
        return bf16 ? launch_permute_grad<true, 2, 2>(dx_sorted, inv, tokens, k, vec, dx, sm_count, stream)
                    : launch_permute_grad<false, 2, 2>(dx_sorted, inv, tokens, k, vec, dx, sm_count, stream);
    return bf16 ? launch_permute_grad<true, 2, 4>(dx_sorted, inv, tokens, k, vec, dx, sm_count, stream)
                : launch_permute_grad<false, 2, 4>(dx_sorted, inv, tokens, k, vec, dx, sm_count, stream);
}

cudaError_t launch_router_topk_grad(const void* logits, bool bf16, const int32_t* ids, const float* weights,
                                    const float* dweights, long long tokens, int E, int k, int mode, void* dlogits,
                                    int sm_count, cudaStream_t stream) {
    const int grid = warps_grid(tokens, sm_count);
    const auto launch = E <= 32    ? launch_topk_grad_ipl<1>
                        : E <= 64  ? launch_topk_grad_ipl<2>
                        : E <= 128 ? launch_topk_grad_ipl<4>
                        : E <= 256 ? launch_topk_grad_ipl<8>
                        : E <= 512 ? launch_topk_grad_ipl<16>
                                   : launch_topk_grad_ipl<32>;
    return launch(logits, bf16, ids, weights, dweights, tokens, E, k, mode, dlogits, grid, stream);
}

}  // namespace rdot
