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

// A block covers TY rows at once and TX chunks of 8 columns of each (16 bytes of every bf16 row: a
// warp's accesses are whole lines; 16 columns a thread wrote half sectors and took 774 us where
// this takes 519, 196608 rows of 1536); TX = 1 << tx_log2 divides f / 8. kActItems items of a
// thread are loaded before the first is worked on (1: 611 us, 2: 519, 4: 614). With few rows the
// columns are shared out too (gridDim.y). Bound by
// memory: 3.04 GB in 519 us, 0.89 of the measured copy rate.
constexpr int kActItems = 2;

__global__ void __launch_bounds__(256)
    swiglu_backward_kernel(const uint8_t *__restrict__ ckpt, const int32_t *__restrict__ rows_dev,
                           int rows_alloc, int f, int tx_log2,
                           const uint16_t *dh, uint16_t *dgate,
                           uint16_t *dup, uint16_t *h)
{
    const int rows = max(0, min(*rows_dev, rows_alloc));
    const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
    const int TX = 1 << tx_log2, TY = 256 >> tx_log2, stride = checkpoint_stride(f);
    const int groups = (f / 8) >> tx_log2;  // groups of TX chunks of a row, and this block's
    const int g0 = groups * blockIdx.y / gridDim.y, g1 = groups * (blockIdx.y + 1) / gridDim.y;
    const int per_row = g1 - g0, first = (g0 << tx_log2) + tx, end = g1 << tx_log2;
    // item i of this thread: chunk i % per_row of its row i / per_row
    const int64_t r0 = (int64_t)blockIdx.x * TY + ty, step = (int64_t)gridDim.x * TY;
    const int64_t items = r0 < rows ? ((rows - r0 + step - 1) / step) * per_row : 0;
    int64_t r = r0;
    int c = first;
    for (int64_t i = 0; i < items; i += kActItems) {
        uint2 gc[kActItems], uc[kActItems];
        uint4 dq[kActItems];
        float gs[kActItems], us[kActItems];
        size_t at[kActItems];
#pragma unroll
        for (int k = 0; k < kActItems; ++k) {
            if (i + k < items) {
                const uint8_t *row = ckpt + (size_t)r * stride;
                at[k] = (size_t)r * f + 8 * c;
                gc[k] = *reinterpret_cast<const uint2 *>(row + 8 * c);
                uc[k] = *reinterpret_cast<const uint2 *>(row + f + 8 * c);
                dq[k] = *reinterpret_cast<const uint4 *>(dh + at[k]);
                gs[k] = pow2f((int)row[2 * f + c / 4] - 127);
                us[k] = pow2f((int)row[2 * f + f / 32 + c / 4] - 127);
                c += TX;
                if (c >= end) {
                    c = first;
                    r += step;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kActItems; ++k) {
            if (i + k < items) {
                const uint32_t dw[4] = {dq[k].x, dq[k].y, dq[k].z, dq[k].w};
                float g[8], u[8], a[8], b[8], hh[8];
                decode_e4m3x8(gc[k].x, gc[k].y, gs[k], g);
                decode_e4m3x8(uc[k].x, uc[k].y, us[k], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = (j & 1) ? bf16_hi(dw[j / 2]) : bf16_lo(dw[j / 2]);
                    // s and 1 - s from e^-|g| <= 1: neither overflows nor cancels for large |g|
                    const float e = __expf(-fabsf(g[j]));
                    const float q = __fdividef(1.0f, 1.0f + e), eq = e * q;
                    const float s = g[j] < 0.0f ? eq : q, t = g[j] < 0.0f ? q : eq;
                    const float silu = g[j] * s;
                    a[j] = d * u[j] * (s + silu * t);
                    b[j] = d * silu;
                    hh[j] = silu * u[j];
                }
                auto pack = [](const float (&v)[8]) {
                    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                };
                *reinterpret_cast<uint4 *>(dgate + at[k]) = pack(a);
                *reinterpret_cast<uint4 *>(dup + at[k]) = pack(b);
                if (h)
                    *reinterpret_cast<uint4 *>(h + at[k]) = pack(hh);
            }
        }
    }
}

}  // namespace moe
