// Backward pass of the router: from the gradients of the gate weights and of the logits to the
// gradients of the hidden states, the router weights and the bias.
//
//   dl[t][e] = dlogits[t][e] + sum over slots k with topk_idx[t][k] = e of
//              w_k (dw_k - sum_j w_j dw_j)            (softmax over the K selected logits)
//   dx = dl Wr (+ dx_add)      dWr = dl^T x      dbias = sum_t dl
// A masked token's dl is 0 whatever its inputs hold, and its row of x is not read.
#pragma once

#include "common.cuh"

namespace moe {

// dl [N][E] fp32, one warp per token.
__global__ void __launch_bounds__(256)
    router_dlogits_kernel(const int32_t *__restrict__ topk_idx, const float *__restrict__ topk_w,
                          const float *__restrict__ dtopk_w, const float *__restrict__ dlogits,
                          const uint8_t *__restrict__ mask, int N, int E, int K,
                          float *__restrict__ dl)
{
    const int lane = threadIdx.x & 31;
    for (int64_t t = (blockIdx.x * 256 + threadIdx.x) >> 5; t < N; t += gridDim.x * 8) {
        const bool live = !mask || mask[t];
        int idx = -1;
        float v = 0.0f;
        if (dtopk_w) {
            float w = 0.0f, dw = 0.0f;
            if (live && lane < K) {
                idx = topk_idx[t * K + lane];
                if ((unsigned)idx < (unsigned)E) {
                    w = topk_w[t * K + lane];
                    dw = dtopk_w[t * K + lane];
                } else {
                    set_dev_error(MOE_ERR_DEVICE_BOUNDS);
                }
            }
            const float s = warp_sum(w * dw);
            v = w * (dw - s);
        }
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            float a = (dlogits && live && e < E) ? dlogits[t * E + e] : 0.0f;
            if (dtopk_w) {
                for (int k = 0; k < K; ++k) {
                    const int ik = __shfl_sync(0xffffffffu, idx, k);
                    const float vk = __shfl_sync(0xffffffffu, v, k);
                    if (ik == e)
                        a += vk;
                }
            }
            if (e < E)
                dl[t * E + e] = a;
        }
    }
}

// dx tile of 64 tokens x 64 columns, 4 x 4 per thread.
template <bool OUT_BF16>
__global__ void __launch_bounds__(256)
    router_dx_kernel(const float *__restrict__ dl, const float *__restrict__ wr,
                     const uint16_t *add, int N, int d, int E, void *dx)
{
    __shared__ float sa[16][65], sb[16][64];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * 64;
    const int c0 = blockIdx.y * 64;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < E; k0 += 16) {
        for (int i = tid; i < 1024; i += 256) {
            const int64_t t = t0 + i / 16;
            const int k = k0 + i % 16;
            sa[i % 16][i / 16] = (t < N && k < E) ? dl[t * E + k] : 0.0f;
        }
        for (int i = tid; i < 1024; i += 256) {
            const int k = k0 + i / 64, c = c0 + i % 64;
            sb[i / 64][i % 64] = (k < E && c < d) ? wr[(size_t)k * d + c] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + ty * 4 + i;
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + tx + 16 * j;
            if (t >= N || c >= d)
                continue;
            const size_t at = (size_t)t * d + c;
            float v = acc[i][j];
            if (add)
                v += __uint_as_float((uint32_t)add[at] << 16);
            if (OUT_BF16)
                static_cast<uint16_t *>(dx)[at] = (uint16_t)pack_bf16x2(v, 0.0f);
            else
                static_cast<float *>(dx)[at] = v;
        }
    }
}

// dWr tile of 16 experts x 64 columns over all tokens (fp32 in chunks of 64 tokens, fp64 over
// the chunks).
__global__ void __launch_bounds__(256)
    router_dw_kernel(const float *__restrict__ dl, const uint16_t *__restrict__ x,
                     const uint8_t *__restrict__ mask, int N, int d, int E,
                     float *__restrict__ dw)
{
    __shared__ float sa[64][16], sb[64][64];
    const int tid = threadIdx.x, tx = tid & 63, ty = tid >> 6;
    const int e0 = blockIdx.y * 16, c0 = blockIdx.x * 64;
    double sum[4] = {};
    for (int64_t t0 = 0; t0 < N; t0 += 64) {
        for (int i = tid; i < 1024; i += 256) {
            const int64_t t = t0 + i / 16;
            const int e = e0 + i % 16;
            sa[i / 16][i % 16] = (t < N && e < E) ? dl[t * E + e] : 0.0f;
        }
        for (int i = tid; i < 4096; i += 256) {
            const int64_t t = t0 + i / 64;
            const int c = c0 + i % 64;
            sb[i / 64][i % 64] = (t < N && c < d && (!mask || mask[t]))
                                     ? __uint_as_float((uint32_t)x[t * d + c] << 16)
                                     : 0.0f;
        }
        __syncthreads();
        float acc[4] = {};
#pragma unroll 8
        for (int k = 0; k < 64; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = fmaf(sa[k][ty * 4 + i], sb[k][tx], acc[i]);
        for (int i = 0; i < 4; ++i)
            sum[i] += acc[i];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int e = e0 + ty * 4 + i, c = c0 + tx;
        if (e < E && c < d)
            dw[(size_t)e * d + c] = (float)sum[i];
    }
}

// dbias: one block per expert.
__global__ void __launch_bounds__(256)
    router_dbias_kernel(const float *__restrict__ dl, int N, int E, float *__restrict__ dbias)
{
    __shared__ double red[8];
    const int e = blockIdx.x;
    double s = 0.0;
    for (int64_t t = threadIdx.x; t < N; t += 256)
        s += dl[t * E + e];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w)
            s += red[w];
        dbias[e] = (float)s;
    }
}

}  // namespace moe
