// Backward pass of the router: from the gradients of the gate weights and of the logits to the
// gradients of the hidden states, the router weights and the bias.
//
//   dl[t][e] = dlogits[t][e] + sum over slots k with topk_idx[t][k] = e of
//              w_k (dw_k - sum_j w_j dw_j)            (softmax over the K selected logits)
//   dx = dl Wr (+ dx_add)      dWr = dl^T x      dbias = sum_t dl
// A masked token's dl is 0 whatever its inputs hold, and its row of x counts as zeros.
//
// The two contractions run on tcgen05 with 16-bit operands and fp32 accumulation. The fp32 factors
// are split into terms, each the rounding of what is left, and the products of the terms are
// accumulated together:
//   dWr, beside a bf16 x: bf16 terms hi + mid + lo (3 x 8 significant bits hold all 24 of an fp32
//       value): exact products of the fp32 dl;
//   dx, fp32: the same terms of dl and Wr, hi hi + hi mid + mid hi + mid mid + hi lo + lo hi (what
//       is left out is below 2^-23 of the product);
//   dx, bf16: fp16 terms hi + lo (2 x 11 bits), hi hi + hi lo + lo hi: half the products, and what
//       is left out is below 2^-20 of the product. (Two bf16 terms lose 2^-16 of it. That is small
//       beside the output's rounding, but not beside dx where products cancel: dl's entries sum
//       to 0, so what the rows of Wr have in common drops out of dx.) fp16 has 5 exponent bits,
//       so the terms are of dl 2^-r and Wr 2^-b, r per token and b per 64 columns of Wr such that
//       the largest value lies in [2^14, 2^15): a value is off by at most 2^-22 of itself or
//       2^-39 of that largest one. The epilogue multiplies by 2^(r + b).
// Four launches (one or two for little work, router_block_grad_kernel): the split
// (router_split_grad_kernel), dx, dWr, and the sum of dWr's and dbias's partial results in a
// fixed order; the middle two are scheduled while the one before them drains (grid_wait). No
// atomics: the same bits every run.
#pragma once

#include "balance.cuh"
#include "common.cuh"
#include "grouped_gemm.cuh"

namespace moe {
namespace rb {

constexpr int kBox = 8192;  // shared memory of a 64-row x 128-byte TMA box

// Eight values -> 16 bytes of each of the three planes: v = out[0] + out[1] + out[2].
__device__ __forceinline__ void split3x8(const float (&v)[8], uint4 (&out)[3])
{
    uint32_t w[3][4], top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        w[0][i] = pack_bf16x2(a, b);
        const float ra = a - bf16_lo(w[0][i]), rb = b - bf16_hi(w[0][i]);
        w[1][i] = pack_bf16x2(ra, rb);
        w[2][i] = pack_bf16x2(ra - bf16_lo(w[1][i]), rb - bf16_hi(w[1][i]));
        top = max(top, max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu));
    }
    if (top >= 0x7F7F8000u) {
        // infinite, NaN, or a value that rounds past the largest bf16: the first term is the
        // value truncated (a NaN stays one), the others what is left of a finite value
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t h = __float_as_uint(v[j]) >> 16, m = 0, l = 0;
            if (isnan(v[j]))
                h |= 0x40u;
            else if (!isinf(v[j])) {
                const float r = v[j] - __uint_as_float(h << 16);
                m = pack_bf16x2(r, 0.0f) & 0xFFFFu;
                l = pack_bf16x2(r - __uint_as_float(m << 16), 0.0f) & 0xFFFFu;
            }
            const uint32_t t[3] = {h, m, l};
#pragma unroll
            for (int p = 0; p < 3; ++p)
                w[p][j / 2] = (j & 1) ? (w[p][j / 2] & 0xFFFFu) | (t[p] << 16)
                                      : (w[p][j / 2] & 0xFFFF0000u) | t[p];
        }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
        out[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

// Exponent x of values whose largest finite magnitude is `top`: top 2^-x in [2^14, 2^15), 0 if
// there is none. Down to -127: what is scaled by more is below 2^-113.
__device__ __forceinline__ int f16_terms_exp(float top)
{
    return top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127 - 14, -127) : 0;
}

// |v|, 0 for an infinity or NaN.
__device__ __forceinline__ float finite_abs(float v)
{
    v = fabsf(v);
    return v <= 3.402823466e38f ? v : 0.0f;
}

// n values times `scale` -> their two fp16 terms. An infinity or NaN is the first one.
template <int n>
__device__ __forceinline__ void split_f16(const float (&v)[n], float scale, uint32_t (&w)[2][n / 2])
{
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        const float a = v[2 * i] * scale, b = v[2 * i + 1] * scale;
        w[0][i] = gg::pack_f16x2(a, b);
        const float ra = a - f16_to_f32(w[0][i] & 0xFFFFu), rb = b - f16_to_f32(w[0][i] >> 16);
        w[1][i] = gg::pack_f16x2(isfinite(a) ? ra : 0.0f, isfinite(b) ? rb : 0.0f);
    }
}

// What the gradient of the logits is made of.
struct GradIn {
    const int32_t *topk_idx;
    const float *topk_w, *dtopk_w;  // dtopk_w nullable
    const float *dlogits;           // nullable
    const uint8_t *mask;            // nullable
};

// dl of token t in the 8 neighbouring columns from 8 l, LPR lanes to a token (all lanes of the
// warp call). Zeros for a masked token (whatever its inputs hold) and past the last one. row:
// the lane group's 8 LPR floats of shared memory, where the slots' gradients meet their columns.
template <int LPR>
__device__ __forceinline__ void token_dlogits(const GradIn &in, int N, int E, int K, int64_t t,
                                              int l, float *row, float (&v)[8])
{
    const int c0 = 8 * l;
    const bool inside = t < N;
    // a masked token's inputs are read all the same (and dropped): no load waits for the mask
    const bool live = inside && (!in.mask || in.mask[t]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = 0.0f;
    if (inside && in.dlogits) {
        const float *src = in.dlogits + t * E;
        if (E % 4 == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (c0 + 4 * i < E) {
                    const float4 q = *reinterpret_cast<const float4 *>(src + c0 + 4 * i);
                    v[4 * i] = q.x;
                    v[4 * i + 1] = q.y;
                    v[4 * i + 2] = q.z;
                    v[4 * i + 3] = q.w;
                }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < E)
                    v[j] = src[c0 + j];
        }
    }
    if (!live) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = 0.0f;
    }
    if (!in.dtopk_w)
        return;
    // slot k of the token, or zeros
    auto slot = [&](int k, int &idx, float &w, float &dw) {
        idx = -1;
        w = dw = 0.0f;
        if (k < K && inside) {
            idx = in.topk_idx[t * K + k];
            w = in.topk_w[t * K + k];
            dw = in.dtopk_w[t * K + k];
            if (!live || (unsigned)idx >= (unsigned)E) {
                if (live)
                    set_dev_error(MOE_ERR_DEVICE_BOUNDS);
                idx = -1;
                w = dw = 0.0f;
            }
        }
    };
    // lane l takes the slots l, l + LPR, ...
    float s = 0.0f;
    int idx, idx0 = -1;
    float w, dw, w0 = 0.0f, dw0 = 0.0f;
    for (int k0 = 0; k0 < K; k0 += LPR) {
        slot(k0 + l, idx, w, dw);
        if (k0 == 0) {
            idx0 = idx;
            w0 = w;
            dw0 = dw;
        }
        s += w * dw;
    }
    s = row_sum<LPR>(s);
    *reinterpret_cast<float4 *>(row + c0) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(row + c0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
    __syncwarp();
    for (int k0 = 0; k0 < K; k0 += LPR) {
        if (k0 == 0) {
            idx = idx0;
            w = w0;
            dw = dw0;
        } else {
            slot(k0 + l, idx, w, dw);
        }
        const float g = w * (dw - s);
        // an expert twice among these slots (no router's top-K, but allowed): one after another
        const int self = threadIdx.x & 31;
        const int key = idx < 0 ? -1 - self : idx + ((self / LPR) << 16);
        const uint32_t same = __match_any_sync(0xffffffffu, key);
        const bool lone = (same & (same - 1)) == 0;
        if (__all_sync(0xffffffffu, lone)) {
            if (idx >= 0)
                row[idx] += g;
            __syncwarp();
        } else {
            for (int o = 0; o < LPR; ++o) {
                if (l == o && idx >= 0)
                    row[idx] += g;
                __syncwarp();
            }
        }
    }
    const float4 a = *reinterpret_cast<const float4 *>(row + c0);
    const float4 b = *reinterpret_cast<const float4 *>(row + c0 + 4);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
    __syncwarp();
}

struct SplitArgs {
    GradIn in;
    const float *wr;  // nullable: no planes of the router weights wanted
    int N, E, K, d;
    int pitch;        // columns of a row of dl's planes, the ones past E zeros
    uint16_t *dl;     // bf16 terms, [3][N][pitch]; nullable
    uint16_t *dl16;   // F16: fp16 terms of dl 2^-row_exp, [2][N][pitch]
    int32_t *row_exp; // F16: [N]
    // terms of the router weights, [d / 64 rounded up][E][64] each: a box of 64 columns of x in
    // one piece. F16: two of fp16, of wr 2^-box_exp, else three of bf16
    uint16_t *wp;
    int32_t *box_exp; // F16: [d / 64 rounded up]
    float *bias_part; // [E][token_blocks]
    int token_blocks;
};

constexpr int kSplitThreads = 256;

// The last token_blocks blocks: dl of their tokens, in planes, and its sum over them; LPR lanes per
// token, 8 neighbouring columns each (one 16-byte store per plane). The blocks before them: the
// planes of the router weights (first, because fp16 terms take longer).
// F16: the fp16 terms of a bf16 dx are wanted.
template <int LPR, bool F16>
__global__ void __launch_bounds__(kSplitThreads) router_split_grad_kernel(const SplitArgs a)
{
    constexpr int GW = 32 / LPR, WARPS = kSplitThreads / 32;
    const int tid = threadIdx.x;
    grid_go();
    const int w_blocks = (int)gridDim.x - a.token_blocks;
    if (F16 && (int)blockIdx.x < w_blocks) {
        __shared__ float s_top[WARPS];
        const int boxes = (a.d + 63) / 64;
        constexpr int NI = LPR < 2 ? 1 : LPR / 2;  // E <= 8 LPR: a thread's quarter rows of a box
        for (int box = blockIdx.x; box < boxes; box += w_blocks) {
            const float *src = a.wr + box * 64;
            const int c = 4 * (tid & 15), c_end = a.d - box * 64;  // a multiple of 8
            float4 q[NI];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = (tid >> 4) + i * (kSplitThreads / 16);
                q[i] = e < a.E && c < c_end
                           ? *reinterpret_cast<const float4 *>(src + (size_t)e * a.d + c)
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
                top = fmaxf(top, fmaxf(fmaxf(finite_abs(q[i].x), finite_abs(q[i].y)),
                                       fmaxf(finite_abs(q[i].z), finite_abs(q[i].w))));
            top = row_max<32>(top);
            __syncthreads();  // the box before is done with
            if ((tid & 31) == 0)
                s_top[tid >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                top = fmaxf(top, s_top[w]);
            const int x = f16_terms_exp(top);
            const float scale = pow2f(-x);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = (tid >> 4) + i * (kSplitThreads / 16);
                const float v[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
                uint32_t w[2][2];
                split_f16<4>(v, scale, w);
                if (e < a.E && c < c_end) {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        *reinterpret_cast<uint2 *>(
                            a.wp + (((size_t)p * boxes + box) * a.E + e) * 64 + c) =
                            make_uint2(w[p][0], w[p][1]);
                }
            }
            if (tid == 0)
                a.box_exp[box] = x;
        }
        return;
    }
    if ((int)blockIdx.x < w_blocks) {
        const int64_t n = (int64_t)a.E * a.d / 8;  // d % 8 == 0
        const int64_t step = (int64_t)w_blocks * kSplitThreads;
        for (int64_t i = (int64_t)blockIdx.x * kSplitThreads + tid; i < n; i += step) {
            const float4 lo = reinterpret_cast<const float4 *>(a.wr)[2 * i];
            const float4 hi = reinterpret_cast<const float4 *>(a.wr)[2 * i + 1];
            const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint4 out[3];
            split3x8(v, out);
            const int e = (int)(i / (a.d / 8)), c = (int)(i - (int64_t)e * (a.d / 8));  // 8 columns
            const int blocks = (a.d + 63) / 64;
#pragma unroll
            for (int p = 0; p < 3; ++p)
                reinterpret_cast<uint4 *>(a.wp)[(((size_t)p * blocks + c / 8) * a.E + e) * 8 +
                                                (c & 7)] = out[p];
        }
        return;
    }
    __shared__ float s_sum[WARPS * LPR * 8];
    __shared__ __align__(16) float s_row[WARPS * 256];
    const int warp = tid >> 5, lane = tid & 31, l = lane % LPR, grp = lane / LPR;
    const int c0 = 8 * l, E = a.E;
    const size_t plane = (size_t)a.N * a.pitch;
    float sum[8] = {};
    const int64_t stride = (int64_t)a.token_blocks * WARPS * GW;
    const int block = (int)blockIdx.x - w_blocks;
    for (int64_t t0 = ((int64_t)block * WARPS + warp) * GW; t0 < a.N; t0 += stride) {
        const int64_t t = t0 + grp;
        float v[8];
        token_dlogits<LPR>(a.in, a.N, E, a.K, t, l, s_row + warp * 256 + grp * (8 * LPR), v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[j] += v[j];
        const bool stored = t < a.N && c0 < a.pitch;
        if (a.dl && stored) {
            uint4 out[3];
            split3x8(v, out);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint4 *>(a.dl + p * plane + t * a.pitch + c0) = out[p];
        }
        if constexpr (F16) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = fmaxf(top, finite_abs(v[j]));
            const int x = f16_terms_exp(row_max<LPR>(top));
            uint32_t w[2][4];
            split_f16<8>(v, pow2f(-x), w);
            if (stored) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    *reinterpret_cast<uint4 *>(a.dl16 + p * plane + t * a.pitch + c0) =
                        make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
                if (l == 0)
                    a.row_exp[t] = x;
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
    }
    if (grp == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s_sum[warp * (LPR * 8) + c0 + j] = sum[j];
    }
    __syncthreads();
    if (tid < E) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            s += s_sum[w * (LPR * 8) + tid];
        a.bias_part[(size_t)tid * a.token_blocks + block] = s;
    }
}

// ---------------------------------------------------------------- shared by the two GEMMs

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor of an operand whose rows of shared memory run along K (the
// M or N index is the contiguous one): boxes of [K][64 elements], 128-byte swizzle; 8 K rows are
// 1024 bytes, the next 64 elements of M or N are one box of `box_bytes` further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t box_bytes)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// bf16 (or both fp16) operands, fp32 accumulate; which operand is the M- or N-contiguous kind.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn, bool b_mn, bool f16 = false)
{
    return (f16 ? gg::instr_desc_f16(M, N) : gg::instr_desc_bf16(M, N)) | ((uint32_t)a_mn << 15) |
           ((uint32_t)b_mn << 16);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------- dWr = dl^T x

// D[e][d'] over a chunk of kChunk tokens: M = e (128 rows), N = d' (256 columns of x), K =
// tokens. Both operands lie in memory with the token as the slow index, so both are the
// M/N-contiguous kind. e is M and d' is N because an M = 128 MMA costs 64 cycles however small
// N is (measured: 70 at N = 64 and 128, 130 at 256: its A operand is read at 64 bytes a
// cycle), so the wide side has to be N. Up to 64 experts (FOLD), the M tile holds two planes
// (rows e: hi and lo, rows 64 + e: mid), which router_sum_kernel adds; the fourth quarter of A is a
// box of zeros. More experts: a CTA takes 128 of them. A chunk's sum is read back and added to
// fp32 registers before it is longer than 128 tokens: the tensor core's accumulator truncates,
// and a truncation per step over tens of thousands of tokens would cost the low bits that the
// split keeps. 32768 x 4096 x 64, mask: 60 us, 4.8 TB/s, MMA 0.67 of it.
// The CTAs of one share of the tokens walk over them together, one column tile each, so that
// rows of x are read whole within a short time.
constexpr int kChunk = 128;  // tokens accumulated in TMEM
constexpr int kDwThreads = 384;

template <bool FOLD>
struct DwTile {
    static constexpr int NE = FOLD ? 1 : 2;     // boxes of 64 experts
    static constexpr int XB = 4;                // boxes of 64 columns of x
    // Tokens of a shared-memory stage. With 64, two (FOLD: three) stages fit, and a stage that
    // waits for its masked rows is missed: 64 -> 58 us with a mask at 32768 x 4096 x 64, 57 ->
    // 46 us at 16384 x 4096 x 128.
    static constexpr int TOK = 32;
    static constexpr int BOX = TOK * 128;       // a box of them: 64 columns
    static constexpr int STAGE = (XB + 3 * NE) * BOX;
    static constexpr int ZERO = FOLD ? BOX : 0;
    static constexpr int STAGES = (231168 - ZERO) / STAGE;  // within 227 KB
    static constexpr int SMEM = STAGES * STAGE + ZERO + 1024 + 256;
    static_assert(STAGES >= 2 && STAGES <= 8, "tile");
};

struct DwArgs {
    int N, d, E;
    int tiles;       // column tiles of 64 XB
    int groups;      // groups of 128 experts (FOLD: 1)
    int chunks;      // chunks of kChunk tokens
    int parts;       // equal shares of the chunks, one CTA each for every tile
    int x_boxes;     // tm_x is [d / 64][N][64] (d % 64 == 0), else [N][d]
    const uint8_t *mask;
    float *part;     // [tiles][groups][parts][columns / 8][128 rows][8]
    uint64_t timeout_ns;
};

// Warps: 0 TMA, 1 MMA, 2 and 3 zero the rows of x of masked tokens (a masked row may hold NaN,
// and 0 * NaN would reach every sum), 4..11 the running sums.
template <bool FOLD>
__global__ void __launch_bounds__(kDwThreads, 1)
    router_dw_kernel(const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_dl, const DwArgs a)
{
    using T = DwTile<FOLD>;
    constexpr int S = T::STAGES, NE = T::NE, XB = T::XB, TOK = T::TOK, BOX = T::BOX;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S * T::STAGE + T::ZERO);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 3 * S + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t base = smem_u32(smem), zero = base + S * T::STAGE, bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto clean = [&](int s) { return bar0 + 8u * (S + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 * S + s); };
    auto tfull = [&](int i) { return bar0 + 8u * (3 * S + i); };
    auto tempty = [&](int i) { return bar0 + 8u * (3 * S + 2 + i); };
    const uint32_t done = bar0 + 8u * (3 * S + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the CTAs that read the same tokens are neighbours, and of them those of the same columns
    const int group = blockIdx.x % a.groups, tile = blockIdx.x / a.groups % a.tiles;
    const int part = blockIdx.x / (a.groups * a.tiles);
    const int c0 = (int)((int64_t)a.chunks * part / a.parts);
    const int c1 = (int)((int64_t)a.chunks * (part + 1) / a.parts);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(clean(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            mbar_init(tempty(i), 8);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    if (T::ZERO) {
        for (int i = threadIdx.x; i < T::ZERO / 16; i += kDwThreads)
            reinterpret_cast<uint4 *>(smem + S * T::STAGE)[i] = make_uint4(0, 0, 0, 0);
        gg::fence_proxy_async_smem();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_go();
    // The planes are the work of the kernel before dx's: nothing but this wait says that they can be
    // seen here (dx's having waited for them says so to dx's blocks only), so dWr's loads start
    // when dx is done, and only its setup overlaps dx's end.
    grid_wait();
    gg::tc_fence_before();
    __syncthreads();
    gg::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // stages of chunk c: the last one may have tokens for some only
    auto stages_of = [&](int c) {
        const int64_t left = a.N - (int64_t)c * kChunk;
        return left >= kChunk ? kChunk / TOK : (int)((left + TOK - 1) / TOK);
    };

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, last[S];
            bool issued[S];
            for (int s = 0; s < S; ++s)
                issued[s] = false;
            bool ok = true;
            for (int c = c0; c < c1 && ok; ++c) {
                for (int q = 0; q < stages_of(c); ++q) {
                    if (!gg::mbar_wait(empty(stage), phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + stage * T::STAGE;
                    const int t0 = c * kChunk + q * TOK;
                    mbar_arrive_expect_tx(full(stage), T::STAGE);
                    if (a.x_boxes)  // [box of columns][token][64]: all of them in one copy
                        tma_load_3d(dst, &tm_x, 0, t0, tile * XB, full(stage));
                    else
                        for (int b = 0; b < XB; ++b)
                            gg::tma_load_2d(dst + b * BOX, &tm_x, (tile * XB + b) * 64, t0,
                                            full(stage));
                    // [plane][box of experts][token][64]
                    tma_load_4d(dst + XB * BOX, &tm_dl, 0, t0, NE * group, 0, full(stage));
                    issued[stage] = true;
                    last[stage] = phase;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < S; ++s)  // every copy has landed before the CTA may exit
                if (issued[s])
                    gg::mbar_wait(full(s), last[s], abort_flag, a.timeout_ns, false);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t id = idesc(128, 64 * XB, true, true);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int c = c0; c < c1 && ok; ++c) {
                if (!gg::mbar_wait(tempty(acc), acc_phase ^ 1u, abort_flag, a.timeout_ns))
                    break;
                gg::tc_fence_after();
                const uint32_t d0 = tmem + (uint32_t)(acc * 256);
                const int ns = stages_of(c);
                for (int q = 0; q < ns; ++q) {
                    if (!gg::mbar_wait(a.mask ? clean(stage) : full(stage), phase, abort_flag,
                                       a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    gg::tc_fence_after();
                    const uint32_t xa = base + stage * T::STAGE, pb = xa + XB * BOX;
                    const uint64_t bdesc = smem_desc_mn_sw128(xa, BOX);
                    // 16 tokens are 2048 bytes: 128 of the descriptor's address units
                    if constexpr (FOLD) {
                        const uint64_t lo = smem_desc_mn_sw128(pb + 2 * BOX, zero - pb - 2 * BOX);
                        const uint64_t him = smem_desc_mn_sw128(pb, BOX);
#pragma unroll
                        for (int k = 0; k < TOK / 16; ++k)  // the small terms first
                            gg::tc_mma<0>(d0, lo + 128 * k, bdesc + 128 * k, id,
                                          (q > 0 || k > 0) ? 1u : 0u);
#pragma unroll
                        for (int k = 0; k < TOK / 16; ++k)
                            gg::tc_mma<0>(d0, him + 128 * k, bdesc + 128 * k, id, 1u);
                    } else {
#pragma unroll
                        for (int p = 2; p >= 0; --p) {
                            const uint64_t adesc = smem_desc_mn_sw128(pb + p * NE * BOX, BOX);
#pragma unroll
                            for (int k = 0; k < TOK / 16; ++k)
                                gg::tc_mma<0>(d0, adesc + 128 * k, bdesc + 128 * k, id,
                                              (q > 0 || p < 2 || k > 0) ? 1u : 0u);
                        }
                    }
                    gg::tc_commit(empty(stage));
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                gg::tc_commit(tfull(acc));
                acc ^= 1;
                if (acc == 0)
                    acc_phase ^= 1u;
            }
            gg::tc_commit(done);
            gg::mbar_wait(done, 0, abort_flag, a.timeout_ns, false);
        }
    } else if (warp < 4) {
        if (a.mask) {
            // Two warps, every other stage of the ring each, and a stage the same warp's at every
            // use: loads land in any order, and a wait by parity tells a phase from its
            // neighbours only, so whoever waits for a stage must have seen its use before.
            // The mask bytes of a warp's next stage are loaded while this one is awaited.
            const int64_t t_end = min((int64_t)c1 * kChunk, (int64_t)a.N);
            auto masked = [&](int64_t t0) {  // bit i: token t0 + 32 i + lane
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < TOK / 32; ++i)
                    if (t0 + 32 * i + lane < t_end)
                        m |= (uint32_t)(a.mask[t0 + 32 * i + lane] == 0) << i;
                return m;
            };
            int ok = 1;
            int stage = warp - 2;
            uint32_t phase = 0;
            int64_t t0 = (int64_t)c0 * kChunk + stage * TOK;
            uint32_t next = masked(t0);
            while (t0 < t_end) {
                const bool wraps = stage + 2 >= S;
                const int64_t t1 = t0 + (wraps ? S - stage + warp - 2 : 2) * TOK;
                const uint32_t now = next;
                next = masked(t1);
                if (lane == 0)
                    ok = gg::mbar_wait(full(stage), phase, abort_flag, a.timeout_ns) ? 1 : 0;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok)
                    break;
                if (__any_sync(0xffffffffu, now)) {
#pragma unroll
                    for (int i = 0; i < TOK / 32; ++i) {
                        uint32_t m = __ballot_sync(0xffffffffu, now >> i & 1u);
                        for (; m; m &= m - 1) {
                            // a row of each of the XB boxes: 128 bytes, 8 lanes
                            const int row = 32 * i + __ffs(m) - 1;
                            if (lane < 8 * XB) {
                                const uint32_t at = base + stage * T::STAGE + (lane >> 3) * BOX +
                                                    row * 128 + (lane & 7) * 16;
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at),
                                             "r"(0)
                                             : "memory");
                            }
                        }
                    }
                    gg::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0)
                    mbar_arrive(clean(stage));
                t0 = t1;
                stage = wraps ? warp - 2 : stage + 2;
                phase ^= (uint32_t)wraps;
            }
        }
    } else if (warp >= 4) {
        // lane quadrant of TMEM: rows of D; the two warps of a quadrant take 128 of an
        // accumulator's 256 columns each
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        float sum[128];
#pragma unroll
        for (int j = 0; j < 128; ++j)
            sum[j] = 0.0f;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int c = c0; c < c1; ++c) {
            int ok = 0;
            if (lane == 0)
                ok = gg::mbar_wait(tfull(acc), acc_phase, abort_flag, a.timeout_ns) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok)
                break;
            gg::tc_fence_after();
            const uint32_t ta = tmem + lanes + (uint32_t)(acc * 256 + half * 128);
#pragma unroll
            for (int j = 0; j < 128; j += 16) {
                uint32_t v[16];
                gg::tmem_ld16(ta + j, v);
                gg::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sum[j + i] += __uint_as_float(v[i]);
            }
            gg::tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(tempty(acc));
            acc ^= 1;
            if (acc == 0)
                acc_phase ^= 1u;
        }
        // 8 columns of a row are 32 bytes, and neighbouring rows are neighbours in memory: a warp
        // writes 1 KB in one piece
        const int row = q * 32 + lane;
        if ((FOLD ? (row & 63) : group * 128 + row) < a.E) {
            const size_t result = (size_t)(tile * a.groups + group) * a.parts + part;
            float *dst = a.part + result * (128 * 64 * XB) + half * 16 * 1024 + row * 8;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float4 *o = reinterpret_cast<float4 *>(dst + j * 1024);
                o[0] = make_float4(sum[8 * j], sum[8 * j + 1], sum[8 * j + 2], sum[8 * j + 3]);
                o[1] = make_float4(sum[8 * j + 4], sum[8 * j + 5], sum[8 * j + 6], sum[8 * j + 7]);
            }
        }
    }
    __syncwarp();
    gg::tc_fence_before();
    __syncthreads();
    gg::tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

struct SumArgs {
    int d, E;
    // dWr's partial results: [column tiles][groups][parts][32][128][8] (router_dw_kernel; with
    // fold, rows e and e + 64 of each are both expert e's), or, with groups = 0, [parts][E][d]
    int groups, parts, fold;
    const float *part;
    float *dw;
    int dw_blocks;
    const float *bias_part;  // [E][bias_parts]
    int bias_parts;
    float *dbias;
};

// dWr and dbias from their partial results, each element in a fixed order. SL threads share an
// element group (4 neighbouring columns, as the results lie), every SL-th result each: 8 where
// there are few groups (24634 x 152 x 9: 296 results of 342 groups), 1 where there are many.
template <int SL>
__global__ void __launch_bounds__(256) router_sum_kernel(const SumArgs a)
{
    if ((int)blockIdx.x < a.dw_blocks) {
        constexpr int GROUPS = 256 / SL;
        __shared__ float4 s_sum[SL][GROUPS];
        const int slot = threadIdx.x % GROUPS, share = threadIdx.x / GROUPS;
        const int n = a.fold ? 2 * a.parts : a.parts;
        const int64_t i = (int64_t)blockIdx.x * GROUPS + slot;
        const bool inside = i < (int64_t)a.E * a.d / 4;
        size_t at = 4 * (size_t)i, to = at;  // of the result's first part; of dw
        if (a.groups && inside) {
            // 8 columns of an expert, half by half, then the next expert
            const int c8 = (int)(i / (2 * a.E)), r = (int)(i - (int64_t)c8 * (2 * a.E)), e = r >> 1;
            const int tile = c8 / 32, group = e / 128;
            at = (size_t)(tile * a.groups + group) * a.parts * 32768 +
                 (size_t)(c8 - tile * 32) * 1024 + (e - group * 128) * 8 + (r & 1) * 4;
            to = (size_t)e * a.d + 8 * c8 + (r & 1) * 4;
        }
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (inside) {
            const size_t step = a.groups ? 32768 : (size_t)a.E * a.d;
#pragma unroll 8
            for (int k = share; k < n; k += SL) {
                const size_t off = a.fold ? (size_t)(k >> 1) * 32768 + (k & 1) * 512 : k * step;
                const float4 q = *reinterpret_cast<const float4 *>(a.part + at + off);
                s.x += q.x;
                s.y += q.y;
                s.z += q.z;
                s.w += q.w;
            }
        }
        if constexpr (SL > 1) {
            s_sum[share][slot] = s;
            __syncthreads();
            if (share == 0) {
#pragma unroll
                for (int w = 1; w < SL; ++w) {
                    const float4 q = s_sum[w][slot];
                    s.x += q.x;
                    s.y += q.y;
                    s.z += q.z;
                    s.w += q.w;
                }
            }
        }
        if (share == 0 && inside)
            *reinterpret_cast<float4 *>(a.dw + to) = s;
        return;
    }
    // dbias: a warp per expert
    const int e = ((int)blockIdx.x - a.dw_blocks) * 8 + (threadIdx.x >> 5);
    if (e >= a.E)
        return;
    float s = 0.0f;
#pragma unroll 8
    for (int b = threadIdx.x & 31; b < a.bias_parts; b += 32)
        s += a.bias_part[(size_t)e * a.bias_parts + b];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0)
        a.dbias[e] = s;
}

// ---------------------------------------------------------------- dx = dl Wr (+ dx_add)

// D[t][d']: M = 128 tokens, N = 64 nb columns, K = e.
// Up to 64 experts (router_dx_kernel) the pass is bound by memory: a CTA keeps its columns of
// the router weights' planes in shared memory and walks over token tiles, whose planes of dl stream
// through a ring of [128 tokens][64 experts] units; a unit of plane i meets the planes
// j <= PLANES - 1 - i of the weights; eight epilogue warps. The CTAs of a group hold the column
// slices of x and walk over the tokens together, so rows of dx are written whole within a
// short time (measured against CTAs that each walk a strip of their own: 90 -> 74 us at
// 32768 x 4096 x 64; 55 us now, 88 with dx_add: 541 MB at 6.1 TB/s).
// More experts (router_dx_pair_kernel): the weights' planes do not fit beside the rest, so both
// operands stream, 32 experts a stage. A pair of CTAs computes 256 tokens x 256 columns
// (cta_group::2): each loads its 128 tokens of dl and half of the columns of the weights, which
// both read. 4001 x 7168 x 256: 40 us, fp32 79 with the matrix pipe 0.7 busy over all; the tiles
// are 6.05 rounds of the pairs there, so the last of 7 rounds keeps few of them busy. 8192 x
// 2048 x 128: 20 us, 3.5 rounds paid as 4.
constexpr int kUnit = 16384;   // 128 tokens x 64 experts, bf16
constexpr int kPiece = 4096;   // 32 tokens x 128 bytes of dx: what one warp stores at a time
constexpr int kDxMaxUnits = 6;
constexpr int kDxMaxSmem = 231424;

template <bool BF16, bool PAIR, bool ADD>
struct DxTile {
    static constexpr int PLANES = BF16 ? 2 : 3;                // fp16 terms, bf16 terms
    static constexpr int EW = 8;                               // epilogue warps
    static constexpr int THREADS = 32 * (2 + EW);
    // pieces of a warp in flight. fp32, up to 64 experts: two and 256 columns a slice, with
    // dx_add three and 128 (32768 x 4096: 97 against 119 us, 190 against 236)
    static constexpr int SLOTS = BF16 || (!PAIR && ADD) ? 3 : 2;
    static constexpr int CP = BF16 ? 64 : 32;                  // columns of a piece
    static constexpr int NB = !BF16 && !PAIR && ADD ? 2 : 4;   // boxes of a slice, at most
    // dx_add's piece: loaded into the slot it leaves from (bf16), or beside it (half as wide)
    static constexpr int ADD_SLOT = BF16 ? kPiece : kPiece / 2;
    static constexpr int SLOT_AREA = EW * SLOTS * (kPiece + (ADD && !BF16 ? ADD_SLOT : 0));
    __host__ __device__ static constexpr int unit(int nb)  // bytes of a ring unit
    {
        return PAIR ? PLANES * (8192 + nb / 2 * 4096) : kUnit;
    }
    __host__ __device__ static constexpr int weights(int nb)  // bytes of the weights kept
    {
        return PAIR ? 0 : PLANES * nb * kBox;
    }
};

struct DxArgs {
    int N, d, E;
    int nb;         // boxes of 64 columns in a slice (pairs: even)
    int slices;     // column slices
    int tiles;      // token tiles of 128 (pairs: 256)
    int units;      // ring units
    const int32_t *row_exp, *box_exp;  // bf16 dx: the exponents of its factors (SplitArgs)
    uint64_t timeout_ns;
};

// The epilogue warps of both forms (warps 2 ..): TMEM lane quadrant = warp % 4; the warps of a
// quadrant take turns at the pieces of a tile. item(i, tile, slice): this CTA's i-th tile of
// `mine`; release(acc): the accumulator has been read.
template <typename T, bool ADD, typename Item, typename Release>
__device__ __forceinline__ void dx_epilogue(const DxArgs &a, uint32_t tmem, uint32_t p_base,
                                            int mine, const CUtensorMap &tm_dx,
                                            const CUtensorMap &tm_add,
                                            uint32_t tfull0, uint32_t addfull0,
                                            volatile int *abort_flag, const Item &item,
                                            const Release &release)
{
    constexpr bool BF16 = T::PLANES == 2;
    constexpr int CP = T::CP, SLOTS = T::SLOTS, EW = T::EW;
    auto tfull = [&](int i) { return tfull0 + 8u * i; };
    auto addfull = [&](int w, int s) { return addfull0 + 8u * (w * SLOTS + s); };
    constexpr int TURNS = EW / 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, turn = (warp - 2) >> 2, w = warp - 2;
    const int nb = a.nb;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t slots = p_base + w * SLOTS * kPiece;
    const uint32_t adds = BF16 ? slots : p_base + EW * SLOTS * kPiece + w * SLOTS * T::ADD_SLOT;
    const int pieces = 64 * nb / CP;                      // of a tile
    const int own = (pieces - turn + TURNS - 1) / TURNS;  // of them, this warp's
    // a piece's column and first token (of the warp's 32); the pieces of a warp follow one
    // another over the tiles, and their slots and barrier phases with them
    struct Piece {
        int n, pc, tile, slice, slot;
        uint32_t phase;
    };
    auto col_of = [&](const Piece &p) { return p.slice * 64 * nb + (p.pc * TURNS + turn) * CP; };
    auto row_of = [&](const Piece &p) { return p.tile * 128 + q * 32; };
    auto next = [&](Piece &p) {
        if (++p.slot == SLOTS) {
            p.slot = 0;
            p.phase ^= 1u;
        }
        if (++p.pc == own) {
            p.pc = 0;
            if (++p.n < mine)
                item(p.n, p.tile, p.slice);
        }
    };
    Piece now = {0, 0, 0, 0, 0, 0}, ahead;
    item(0, now.tile, now.slice);
    ahead = now;  // dx_add's piece to be fetched next (lane 0)
    auto fetch = [&]() {
        const uint32_t bar = addfull(w, ahead.slot);
        mbar_arrive_expect_tx(bar, T::ADD_SLOT);
        gg::tma_load_2d(adds + ahead.slot * T::ADD_SLOT, &tm_add, col_of(ahead), row_of(ahead),
                        bar);
        next(ahead);
    };
    int fetched = 0, used = 0;
    if (ADD && lane == 0 && own > 0)
        for (; ahead.n < mine && fetched < SLOTS - 1; ++fetched)
            fetch();
    int acc = 0;
    uint32_t acc_phase = 0;
    int ok = 1;
    // bf16: exponents of this lane's row in the warp's pieces of a tile, loaded a tile ahead
    static_assert(!BF16 || T::NB <= 2 * TURNS, "box exponents of a warp");
    int row_x = 0, box_x[2] = {0, 0};
    auto load_exps = [&](int n) {
        if (!BF16 || n >= mine)
            return;
        int tile, slice;
        item(n, tile, slice);
        const int row = tile * 128 + q * 32 + lane, boxes = (a.d + 63) / 64;
        row_x = row < a.N ? __ldcg(a.row_exp + row) : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int box = slice * nb + i * TURNS + turn;
            box_x[i] = i < own && box < boxes ? __ldcg(a.box_exp + box) : 0;
        }
    };
    load_exps(0);
    for (int n = 0; n < mine && ok; ++n) {
        const int exps[2] = {row_x + box_x[0], row_x + box_x[1]};
        load_exps(n + 1);
        if (lane == 0)
            ok = gg::mbar_wait(tfull(acc), acc_phase, abort_flag, a.timeout_ns) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok)
            break;
        gg::tc_fence_after();
        for (int pc = 0; pc < own; ++pc) {
            const uint32_t slot = slots + now.slot * kPiece;
            uint32_t v[CP];
#pragma unroll
            for (int c = 0; c < CP / 16; ++c)
                gg::tmem_ld16(tmem + lanes + acc * 256 + (pc * TURNS + turn) * CP + 16 * c,
                              *reinterpret_cast<uint32_t(*)[16]>(v + 16 * c));
            if (lane == 0) {
                if constexpr (ADD) {
                    ok = gg::mbar_wait(addfull(w, now.slot), now.phase, abort_flag, a.timeout_ns)
                             ? 1 : 0;
                    if (ok)
                        ++used;
                } else {
                    // the store that last read this slot has done so
                    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(SLOTS - 1) : "memory");
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            gg::tmem_ld_wait();
            if (!ok)
                break;
            float scale = 1.0f;
            if constexpr (BF16) {  // 2^(r + b), in two factors where one cannot hold it
                const int x = exps[pc ? 1 : 0], x0 = max(-126, min(127, x));
                scale = pow2f(x0);
                if (__any_sync(0xffffffffu, x != x0)) {
                    const float rest = pow2f(max(-126, min(127, x - x0)));
#pragma unroll
                    for (int c = 0; c < CP; ++c)
                        v[c] = __float_as_uint(__uint_as_float(v[c]) * rest);
                }
                if constexpr (!ADD) {
#pragma unroll
                    for (int c = 0; c < CP; c += 2) {
                        float lo, hi;
                        mul2(Pair(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                             Pair(scale, scale))
                            .get(lo, hi);
                        v[c] = __float_as_uint(lo);
                        v[c + 1] = __float_as_uint(hi);
                    }
                }
            }
            if constexpr (ADD) {
#pragma unroll
                for (int c = 0; c < CP / 8; ++c) {
                    // 16 bytes = 8 columns; rows of 128 bytes (bf16 dx) or 64 bytes
                    const uint32_t at = adds + now.slot * T::ADD_SLOT +
                                        (BF16 ? lane * 128 + ((c ^ (lane & 7)) << 4)
                                              : lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
                    uint32_t x[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                 : "r"(at));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float lo, hi;  // times scale (1 for an fp32 dx) plus dx_add
                        fma2(Pair(__uint_as_float(v[8 * c + 2 * j]),
                                  __uint_as_float(v[8 * c + 2 * j + 1])),
                             Pair(scale, scale), Pair(bf16_lo(x[j]), bf16_hi(x[j])))
                            .get(lo, hi);
                        v[8 * c + 2 * j] = __float_as_uint(lo);
                        v[8 * c + 2 * j + 1] = __float_as_uint(hi);
                    }
                }
                if (!BF16 && lane == 0)  // the slot's last store has read it
                    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(SLOTS - 1) : "memory");
                __syncwarp();
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (BF16)
                        o[j] = pack_bf16x2(__uint_as_float(v[8 * c + 2 * j]),
                                           __uint_as_float(v[8 * c + 2 * j + 1]));
                    else
                        o[j] = v[4 * c + j];
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 slot + lane * 128 + ((c ^ (lane & 7)) << 4)),
                             "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                             : "memory");
            }
            gg::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                const int col = col_of(now), row = row_of(now);
                if (col < a.d && row < a.N)
                    gg::tma_store_2d(&tm_dx, slot, col, row);
                else
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                if (ADD && ahead.n < mine) {
                    // into the slot before this one: its store has read it
                    if (BF16)
                        gg::bulk_wait_read1();
                    fetch();
                    ++fetched;
                }
            }
            next(now);
        }
        gg::tc_fence_before();
        __syncwarp();
        if (!ok)
            break;
        if (lane == 0)
            release(acc);
        acc ^= 1;
        if (acc == 0)
            acc_phase ^= 1u;
    }
    if (lane == 0) {
        for (; used < fetched; ++used)  // after a timeout: copies in flight have landed
            gg::mbar_wait(addfull(w, used % SLOTS), (uint32_t)(used / SLOTS) & 1u, abort_flag,
                          a.timeout_ns, false);
        gg::bulk_wait_all();
    }
}

template <bool BF16, bool ADD>
__global__ void __launch_bounds__((DxTile<BF16, false, ADD>::THREADS), 1)
    router_dx_kernel(const __grid_constant__ CUtensorMap tm_dl,
                     const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_dx,
                     const __grid_constant__ CUtensorMap tm_add, const DxArgs a)
{
    using T = DxTile<BF16, false, ADD>;
    constexpr int PLANES = T::PLANES, SLOTS = T::SLOTS, EW = T::EW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nb = a.nb, wbytes = T::weights(nb), ubytes = T::unit(nb);
    const uint32_t w_base = smem_u32(smem), a_base = w_base + wbytes;
    const uint32_t p_base = a_base + a.units * ubytes;  // pieces, then (fp32) dx_add's
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + wbytes + a.units * ubytes +
                                                  T::SLOT_AREA);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kDxMaxUnits + s); };
    auto tfull = [&](int i) { return bar0 + 8u * (2 * kDxMaxUnits + i); };
    auto tempty = [&](int i) { return bar0 + 8u * (2 * kDxMaxUnits + 2 + i); };
    const uint32_t wfull = bar0 + 8u * (2 * kDxMaxUnits + 4);
    const uint32_t done = bar0 + 8u * (2 * kDxMaxUnits + 5);
    const uint32_t addfull0 = bar0 + 8u * (2 * kDxMaxUnits + 6);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kDxMaxUnits + 6 + EW * SLOTS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this CTA's tiles: item i is (token tile, column slice)
    const int groups = gridDim.x / a.slices, group = blockIdx.x / a.slices;
    const int mine = (a.tiles - group + groups - 1) / groups;
    auto item = [&](int i, int &tile, int &slice) {
        tile = group + i * groups;
        slice = blockIdx.x % a.slices;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kDxMaxUnits; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            mbar_init(tempty(i), EW);
        }
        mbar_init(wfull, 1);
        mbar_init(done, 1);
        for (int i = 0; i < EW * SLOTS; ++i)
            mbar_init(addfull0 + 8u * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_go();
    grid_wait();  // the planes of the kernel before
    gg::tc_fence_before();
    __syncthreads();
    gg::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, last[kDxMaxUnits];
            bool issued[kDxMaxUnits];
            for (int s = 0; s < kDxMaxUnits; ++s)
                issued[s] = false;
            bool ok = true;
            mbar_arrive_expect_tx(wfull, wbytes);
            tma_load_4d(w_base, &tm_w, 0, 0, (int)(blockIdx.x % a.slices) * nb, 0, wfull);
            for (int i = 0; i < mine && ok; ++i) {
                int tile, slice;
                item(i, tile, slice);
                for (int u = 0; u < PLANES; ++u) {
                    if (!gg::mbar_wait(empty(stage), phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = a_base + stage * ubytes;
                    mbar_arrive_expect_tx(full(stage), ubytes);
                    tma_load_3d(dst, &tm_dl, 0, tile * 128, PLANES - 1 - u, full(stage));
                    issued[stage] = true;
                    last[stage] = phase;
                    if (++stage == a.units) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < a.units; ++s)
                if (issued[s])
                    gg::mbar_wait(full(s), last[s], abort_flag, a.timeout_ns, false);
            gg::mbar_wait(wfull, 0, abort_flag, a.timeout_ns, false);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t id = idesc(128, 64 * nb, false, true, BF16);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = gg::mbar_wait(wfull, 0, abort_flag, a.timeout_ns);
            for (int i = 0; i < mine && ok; ++i) {
                if (!gg::mbar_wait(tempty(acc), acc_phase ^ 1u, abort_flag, a.timeout_ns))
                    break;
                gg::tc_fence_after();
                const uint32_t d0 = tmem + (uint32_t)(acc * 256);
                uint32_t accumulate = 0;
                for (int u = 0; u < PLANES; ++u) {
                    if (!gg::mbar_wait(full(stage), phase, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    gg::tc_fence_after();
                    const uint32_t at = a_base + stage * ubytes;
                    // the small products first; 16 experts are 32 bytes of a row of A and 2048
                    // bytes of B (descriptor address units of 16 bytes)
                    const int ks = (a.E + 15) / 16;
                    const uint64_t ad = gg::smem_desc_sw128(at);
                    for (int j = u; j >= 0; --j) {
                        const uint64_t bd = smem_desc_mn_sw128(w_base + j * nb * kBox, kBox);
                        for (int k = 0; k < ks; ++k) {
                            gg::tc_mma<0>(d0, ad + 2 * k, bd + 128 * k, id, accumulate);
                            accumulate = 1;
                        }
                    }
                    gg::tc_commit(empty(stage));
                    if (++stage == a.units) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                gg::tc_commit(tfull(acc));
                acc ^= 1;
                if (acc == 0)
                    acc_phase ^= 1u;
            }
            gg::tc_commit(done);
            gg::mbar_wait(done, 0, abort_flag, a.timeout_ns, false);
        }
    } else {
        dx_epilogue<T, ADD>(a, tmem, p_base, mine, tm_dx, tm_add, tfull(0), addfull0, abort_flag,
                            item, [&](int acc) { mbar_arrive(tempty(acc)); });
    }
    __syncwarp();
    gg::tc_fence_before();
    __syncthreads();
    gg::tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

// K-major operand in 64-byte swizzled rows (8 rows x 64 bytes, atoms 512 bytes apart).
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1u << 16) |
           ((uint64_t)(512u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)4u << 61);
}

// TMA loads and commits of a pair (no multicast): each CTA loads into its own shared memory, and
// the bytes count on the first CTA's barrier.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                                 int z, uint32_t bar_cluster_addr)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster_addr)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                                 int z, int w, uint32_t bar_cluster_addr)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar_cluster_addr)
        : "memory");
}

// A stage of a tile (chunk = 32 experts). Products of two planes i, j: those below fp32's
// rounding, i + j >= PLANES, are left out. bf16 dx: stage u holds both fp16 planes of chunk u and
// gives all three products. fp32 dx: stages 0 .. C-1 hold the three planes of a chunk and give the
// five products below hi hi; the stages after them hold the hi planes of three chunks each and
// give hi hi. So the accumulator, which the tensor core truncates at every step, holds small
// values until E / 16 steps before the end (all six products chunk by chunk left a relative
// error of 1.5e-6 with 256 experts).
template <bool BF16, bool ADD>
__global__ void __launch_bounds__((DxTile<BF16, true, ADD>::THREADS), 1)
    router_dx_pair_kernel(const __grid_constant__ CUtensorMap tm_dl,
                          const __grid_constant__ CUtensorMap tm_w,
                          const __grid_constant__ CUtensorMap tm_dl1,
                          const __grid_constant__ CUtensorMap tm_w1,
                          const __grid_constant__ CUtensorMap tm_dx,
                          const __grid_constant__ CUtensorMap tm_add, const DxArgs a)
{
    using T = DxTile<BF16, true, ADD>;
    constexpr int PLANES = T::PLANES, SLOTS = T::SLOTS, EW = T::EW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int hb = a.nb / 2, ubytes = T::unit(a.nb);  // boxes of columns this CTA loads
    const uint32_t a_base = smem_u32(smem), p_base = a_base + a.units * ubytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + a.units * ubytes + T::SLOT_AREA);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kDxMaxUnits + s); };
    auto tfull = [&](int i) { return bar0 + 8u * (2 * kDxMaxUnits + i); };
    auto tempty = [&](int i) { return bar0 + 8u * (2 * kDxMaxUnits + 2 + i); };
    const uint32_t done = bar0 + 8u * (2 * kDxMaxUnits + 4);
    const uint32_t addfull0 = bar0 + 8u * (2 * kDxMaxUnits + 5);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kDxMaxUnits + 5 + EW * SLOTS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = gg::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int mine = (a.tiles * a.slices - pair + pairs - 1) / pairs;
    // tiles in token order over the pairs: rows of dx are written whole within a short time
    auto pair_item = [&](int i, int &tile, int &slice) {
        const int u = pair + i * pairs;  // tiles * slices is about N d / 65536
        tile = u / a.slices;
        slice = u - tile * a.slices;
    };
    auto item = [&](int i, int &tile, int &slice) {  // in tiles of 128 tokens
        pair_item(i, tile, slice);
        tile = 2 * tile + (int)rank;
    };
    const int chunks = (a.E + 31) / 32;
    const int per_tile = BF16 ? chunks : chunks + (chunks + 2) / 3;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kDxMaxUnits; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            mbar_init(tempty(i), 2 * EW);
        }
        mbar_init(done, 1);
        for (int i = 0; i < EW * SLOTS; ++i)
            mbar_init(addfull0 + 8u * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    grid_go();
    grid_wait();  // the planes of the kernel before
    gg::tc_fence_before();
    gg::cluster_sync_all();  // barriers initialised in both CTAs before any remote use
    gg::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA (both CTAs)
            int stage = 0;
            uint32_t phase = 0, last[kDxMaxUnits];
            bool issued[kDxMaxUnits];
            for (int s = 0; s < kDxMaxUnits; ++s)
                issued[s] = false;
            bool ok = true;
            for (int i = 0; i < mine && ok; ++i) {
                int tile, slice;
                pair_item(i, tile, slice);
                const int t0 = tile * 256 + (int)rank * 128, cb = slice * a.nb + (int)rank * hb;
                for (int u = 0; u < per_tile; ++u) {
                    if (!gg::mbar_wait(empty(stage), phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = a_base + stage * ubytes, wdst = dst + PLANES * 8192;
                    const uint32_t bar = gg::map_to_rank(full(stage), 0);
                    // chunks of the unit whose hi planes alone are wanted (fp32), or none
                    const int c1 = 3 * (u - chunks);
                    const int n1 = BF16 || u < chunks ? 0 : min(3, chunks - c1);
                    if (rank == 0)
                        mbar_arrive_expect_tx(full(stage),
                                              2 * (n1 ? n1 * (8192 + hb * 4096) : ubytes));
                    if (n1 == 0) {
                        tma_load_3d_pair(dst, &tm_dl, 32 * u, t0, 0, bar);
                        tma_load_4d_pair(wdst, &tm_w, 0, 32 * u, cb, 0, bar);
                    } else {
                        for (int p = 0; p < n1; ++p) {
                            tma_load_3d_pair(dst + p * 8192, &tm_dl1, 32 * (c1 + p), t0, 0, bar);
                            tma_load_4d_pair(wdst + p * hb * 4096, &tm_w1, 0, 32 * (c1 + p), cb, 0,
                                             bar);
                        }
                    }
                    issued[stage] = true;
                    last[stage] = phase;
                    if (++stage == a.units) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (rank == 0)  // its barriers count both CTAs' copies
                for (int s = 0; s < a.units; ++s)
                    if (issued[s])
                        gg::mbar_wait(full(s), last[s], abort_flag, a.timeout_ns, false);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // ---------------- MMA (first CTA of the pair)
            const uint32_t id = idesc(256, 64 * a.nb, false, true, BF16);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int i = 0; i < mine && ok; ++i) {
                if (!gg::mbar_wait(tempty(acc), acc_phase ^ 1u, abort_flag, a.timeout_ns))
                    break;
                gg::tc_fence_after();
                const uint32_t d0 = tmem + (uint32_t)(acc * 256);
                uint32_t accumulate = 0;
                // one product: slot i of dl with slot j of the weights, ks steps of 16 experts (32
                // bytes of a row of A, 2048 bytes of B)
                for (int u = 0; u < per_tile; ++u) {
                    if (!gg::mbar_wait(full(stage), phase, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    gg::tc_fence_after();
                    const uint32_t at = a_base + stage * ubytes;
                    auto product = [&](int x, int y, int ks) {
                        const uint64_t ad = smem_desc_sw64(at + x * 8192);
                        const uint64_t bd =
                            smem_desc_mn_sw128(at + PLANES * 8192 + y * hb * 4096, 4096);
                        gg::tc_mma_pair<0>(d0, ad, bd, id, accumulate);
                        accumulate = 1;
                        if (ks > 1)
                            gg::tc_mma_pair<0>(d0, ad + 2, bd + 128, id, 1u);
                    };
                    if (BF16 || u < chunks) {
                        const int ks = min(2, (a.E - 32 * u + 15) / 16);
#pragma unroll
                        for (int order = PLANES - 1; order >= (BF16 ? 0 : 1); --order)
#pragma unroll
                            for (int p = order; p >= 0; --p)
                                product(p, order - p, ks);
                    } else {
                        const int c1 = 3 * (u - chunks), n1 = min(3, chunks - c1);
                        for (int p = 0; p < n1; ++p)
                            product(p, p, min(2, (a.E - 32 * (c1 + p) + 15) / 16));
                    }
                    gg::tc_commit_pair(gg::map_to_rank(empty(stage), 0));
                    gg::tc_commit_pair(gg::map_to_rank(empty(stage), 1));
                    if (++stage == a.units) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                gg::tc_commit_pair(gg::map_to_rank(tfull(acc), 0));
                gg::tc_commit_pair(gg::map_to_rank(tfull(acc), 1));
                acc ^= 1;
                if (acc == 0)
                    acc_phase ^= 1u;
            }
            gg::tc_commit_pair(gg::map_to_rank(done, 0));
            gg::mbar_wait(done, 0, abort_flag, a.timeout_ns, false);
        }
    } else {
        dx_epilogue<T, ADD>(a, tmem, p_base, mine, tm_dx, tm_add, tfull(0), addfull0, abort_flag,
                            item, [&](int acc) {
                                gg::mbar_arrive_cluster(gg::map_to_rank(tempty(acc), 0));
                            });
    }
    __syncwarp();
    gg::tc_fence_before();
    if (*abort_flag) {
        // after a timeout, give copies already in flight time to land before the pair leaves
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    gg::cluster_sync_all();  // neither CTA leaves while its partner may still use its memory
    gg::tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
}

// ---------------------------------------------------------------- little work

// A call of little work (N E d <= kBlockWork) is bound by its launches and the latency of each: one
// kernel makes dl, dx and dWr of 64 columns in fp32 on the FMA pipes, without planes and tensor
// maps, and a second one adds the blocks' shares of dWr and dbias where there is more than one.
// A block holds its 64 columns of the router weights and of 64 tokens at a time, makes dl of
// those tokens for itself, and keeps its sums of dWr in registers over all its tokens (64
// tokens in one run of additions, then those sums). Measured against the tensor-core path:
// 64 x 128 x 8 13 against 26 us, 2575 x 136 x 11 15 against 19, 1000 x 1000 x 32
// 18.5 against 20.5, 1024 x 2048 x 32 29 against 21.
constexpr int64_t kBlockWork = (int64_t)1 << 25;

__host__ __device__ inline bool block_path(int N, int E, int d)
{
    return (int64_t)N * E * d <= kBlockWork;
}

struct BlockArgs {
    GradIn in;
    const uint16_t *x;
    const float *wr;
    const uint16_t *add;
    void *dx;
    float *dw;    // [parts][E][d]
    float *bias;  // [E][parts]
    int N, E, K, d, bf16;
    int cols, tiles, parts;  // tiles of 64 columns, of 64 tokens; shares of the latter
};

// dl [64][E + 1] (a row's neighbours in other banks), x [64][64], Wr [E][64].
constexpr int block_smem(int E) { return 4 * (64 * (E + 1) + 64 * 64 + 64 * E); }

template <int LPR>
__global__ void __launch_bounds__(256) router_block_grad_kernel(const BlockArgs a)
{
    constexpr int GW = 32 / LPR, NI = LPR < 2 ? 1 : LPR / 2;  // experts of a thread: 16 apart
    extern __shared__ __align__(16) float block_mem[];
    __shared__ __align__(16) float s_row[8 * 256];
    const int N = a.N, E = a.E, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *xs = block_mem, *ws = xs + 64 * 64, *dl = ws + 64 * E;
    const int tx = tid & 15, ty = tid >> 4, pitch = E + 1;
    const int tile_c = blockIdx.x % a.cols, part = blockIdx.x / a.cols;
    const int c0 = tile_c * 64, col = c0 + 4 * tx;  // this thread's 4 columns
    const int t_first = (int)((int64_t)a.tiles * part / a.parts);
    const int t_last = (int)((int64_t)a.tiles * (part + 1) / a.parts);
    if (a.dx)
        for (int i = tid; i < E * 16; i += 256) {
            const int e = i >> 4, c = c0 + 4 * (i & 15);
            *reinterpret_cast<float4 *>(ws + e * 64 + 4 * (i & 15)) =
                c < a.d ? *reinterpret_cast<const float4 *>(a.wr + (size_t)e * a.d + c)
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    float sum[NI][4] = {}, bias = 0.0f;
    for (int tile = t_first; tile < t_last; ++tile) {
        const int t0 = tile * 64;
        __syncthreads();  // the tile before is done with
        for (int r = warp * GW; r < 64; r += 8 * GW) {
            const int l = lane % LPR, t = r + lane / LPR;
            float v[8];
            float *row = s_row + warp * 256 + (lane / LPR) * (8 * LPR);
            token_dlogits<LPR>(a.in, N, E, a.K, t0 + t, l, row, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * l + j < E)
                    dl[t * pitch + 8 * l + j] = v[j];
        }
        if (a.dw)
            for (int i = tid; i < 64 * 8; i += 256) {  // 8 columns of a token
                const int t = t0 + (i >> 3), c = c0 + 8 * (i & 7);
                uint4 q = make_uint4(0, 0, 0, 0);
                if (t < N && c < a.d && (!a.in.mask || a.in.mask[t]))
                    q = *reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.d + c);
                float4 *o = reinterpret_cast<float4 *>(xs + (i >> 3) * 64 + 8 * (i & 7));
                o[0] = make_float4(bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y));
                o[1] = make_float4(bf16_lo(q.z), bf16_hi(q.z), bf16_lo(q.w), bf16_hi(q.w));
            }
        __syncthreads();
        if (a.dx) {
            float acc[4][4] = {};  // tokens ty + 16 i
#pragma unroll 4
            for (int e = 0; e < E; ++e) {
                const float4 w = *reinterpret_cast<const float4 *>(ws + e * 64 + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float g = dl[(ty + 16 * i) * pitch + e];
                    acc[i][0] = fmaf(g, w.x, acc[i][0]);
                    acc[i][1] = fmaf(g, w.y, acc[i][1]);
                    acc[i][2] = fmaf(g, w.z, acc[i][2]);
                    acc[i][3] = fmaf(g, w.w, acc[i][3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + ty + 16 * i;
                if (t >= N || col >= a.d)
                    continue;
                const size_t at = (size_t)t * a.d + col;
                if (a.add) {
                    const uint2 q = *reinterpret_cast<const uint2 *>(a.add + at);
                    acc[i][0] += bf16_lo(q.x);
                    acc[i][1] += bf16_hi(q.x);
                    acc[i][2] += bf16_lo(q.y);
                    acc[i][3] += bf16_hi(q.y);
                }
                if (a.bf16)
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dx) + at) = make_uint2(
                        pack_bf16x2(acc[i][0], acc[i][1]), pack_bf16x2(acc[i][2], acc[i][3]));
                else
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.dx) + at) =
                        make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            }
        }
        if (a.dw) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = min(ty + 16 * i, E - 1);
                float acc[4] = {};
#pragma unroll 8
                for (int t = 0; t < 64; ++t) {
                    const float g = dl[t * pitch + e];
                    const float4 q = *reinterpret_cast<const float4 *>(xs + t * 64 + 4 * tx);
                    acc[0] = fmaf(g, q.x, acc[0]);
                    acc[1] = fmaf(g, q.y, acc[1]);
                    acc[2] = fmaf(g, q.z, acc[2]);
                    acc[3] = fmaf(g, q.w, acc[3]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum[i][j] += acc[j];
            }
        }
        if (a.bias && tile_c == 0 && tid < E) {
            float acc = 0.0f;
#pragma unroll 8
            for (int t = 0; t < 64; ++t)
                acc += dl[t * pitch + tid];
            bias += acc;
        }
    }
    if (a.dw && col < a.d) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = ty + 16 * i;
            if (e < E)
                *reinterpret_cast<float4 *>(a.dw + ((size_t)part * E + e) * a.d + col) =
                    make_float4(sum[i][0], sum[i][1], sum[i][2], sum[i][3]);
        }
    }
    if (a.bias && tile_c == 0 && tid < E)
        a.bias[(size_t)tid * a.parts + part] = bias;
}

}  // namespace rb
}  // namespace moe
