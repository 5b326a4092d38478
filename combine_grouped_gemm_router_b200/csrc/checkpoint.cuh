// 8-bit checkpoint of the SwiGLU experts' pre-activations, and the activation's backward pass
// that reads it.
//
// A checkpoint row holds one kept row's gate values g = x W1^T and up values u = x W3^T [f]
// each, as e4m3 codes with one power of two per 32 columns (the block rule of the FP8 return
// payload): f gate codes, f up codes, f / 32 gate exponent bytes j + 127, f / 32 up exponent
// bytes, zero-padded or left as found up to a multiple of 16 bytes. 2.06 bytes per column
// instead of the 6 of bf16 g, u and h.
//
// From the decoded g, u and the gradient dh of h = silu(g) u, with s = 1 / (1 + e^-g):
//   dgate = dh u s (1 + g (1 - s))     dup = dh g s     h = g s u (recomputed)
#pragma once

#include "combine.cuh"
#include "common.cuh"

namespace moe {

__host__ __device__ constexpr int checkpoint_stride(int f)
{
    return 2 * f + ((f / 16 + 15) & ~15);
}

// A block covers TY rows at once and TX chunks of 8 columns of each; TX divides f / 8.
__global__ void __launch_bounds__(256)
    swiglu_backward_kernel(const uint8_t *__restrict__ ckpt, const int32_t *__restrict__ rows_dev,
                           int rows_alloc, int f, int tx_log2,
                           const uint16_t *dh, uint16_t *dgate,
                           uint16_t *dup, uint16_t *h)
{
    const int rows = max(0, min(*rows_dev, rows_alloc));
    const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
    const int TY = 256 >> tx_log2, chunks = f / 8, stride = checkpoint_stride(f);
    for (int64_t r = (int64_t)blockIdx.x * TY + ty; r < rows; r += (int64_t)gridDim.x * TY) {
        const uint8_t *row = ckpt + (size_t)r * stride;
        for (int c = tx; c < chunks; c += 1 << tx_log2) {
            const uint2 gc = *reinterpret_cast<const uint2 *>(row + 8 * c);
            const uint2 uc = *reinterpret_cast<const uint2 *>(row + f + 8 * c);
            const float gs = pow2f((int)row[2 * f + c / 4] - 127);
            const float us = pow2f((int)row[2 * f + f / 32 + c / 4] - 127);
            const size_t at = (size_t)r * f + 8 * c;
            const uint4 dq = *reinterpret_cast<const uint4 *>(dh + at);
            const uint32_t dw[4] = {dq.x, dq.y, dq.z, dq.w};
            float g[8], u[8], a[8], b[8], hh[8];
            decode_e4m3x8(gc.x, gc.y, gs, g);
            decode_e4m3x8(uc.x, uc.y, us, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = (j & 1) ? bf16_hi(dw[j / 2]) : bf16_lo(dw[j / 2]);
                // s and 1 - s from e^-|g| <= 1: neither overflows nor cancels for large |g|
                const float e = __expf(-fabsf(g[j]));
                const float r = __fdividef(1.0f, 1.0f + e), er = e * r;
                const float s = g[j] < 0.0f ? er : r, t = g[j] < 0.0f ? r : er;
                const float silu = g[j] * s;
                a[j] = d * u[j] * (s + silu * t);
                b[j] = d * silu;
                hh[j] = silu * u[j];
            }
            auto pack = [](const float (&v)[8]) {
                return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            };
            *reinterpret_cast<uint4 *>(dgate + at) = pack(a);
            *reinterpret_cast<uint4 *>(dup + at) = pack(b);
            if (h)
                *reinterpret_cast<uint4 *>(h + at) = pack(hh);
        }
    }
}

}  // namespace moe
