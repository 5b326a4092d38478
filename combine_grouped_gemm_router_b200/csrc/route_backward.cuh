// Backward pass of the router: from the gradients of the gate weights and of the logits to the
// gradients of the hidden states, the router weights and the bias.
//
//   dl[t][e] = dlogits[t][e] + sum over slots k with topk_idx[t][k] = e of
//              w_k (dw_k - sum_j w_j dw_j)            (softmax over the K selected logits)
//   dx = dl Wr (+ dx_add)      dWr = dl^T x      dbias = sum_t dl
// A masked token's dl is 0 whatever its inputs hold, and its row of x counts as zeros.
//
// The two contractions run on tcgen05 with bf16 operands and fp32 accumulation. x is bf16
// already; the fp32 factors are split into bf16 terms, v = hi + mid + lo (each the rounding of
// what is left: 3 x 8 significant bits hold all 24 of an fp32 value), and the products of the
// terms are accumulated together:
//   dWr: x (hi + mid + lo): exact products of the fp32 dl;
//   dx, fp32: hi hi + hi mid + mid hi + mid mid + hi lo + lo hi (what is left out is below
//       2^-23 of the product); bf16: hi hi + hi mid + mid hi (below 2^-14, against the output's
//       own rounding of 2^-8).
// Four launches: the split (router_split_grad_kernel), dx, dWr, and the sum of dWr's and dbias's
// partial results in a fixed order. No atomics: the same bits every run.
#pragma once

#include "common.cuh"
#include "grouped_gemm.cuh"

namespace moe {
namespace rb {

constexpr int kBox = 8192;  // shared memory of a 64-row x 128-byte TMA box

// v = p[0] + p[1] + p[2] in bf16 terms (bits). Not finite: all of it in p[0].
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3])
{
    uint32_t h = pack_bf16x2(v, 0.0f) & 0xFFFFu;
    if (!isfinite(__uint_as_float(h << 16))) {
        if (!isfinite(v)) {
            p[0] = h;
            p[1] = p[2] = 0;
            return;
        }
        h = __float_as_uint(v) >> 16;  // rounds past the largest bf16: truncated instead
    }
    const float r = v - __uint_as_float(h << 16);
    const uint32_t m = pack_bf16x2(r, 0.0f) & 0xFFFFu;
    p[0] = h;
    p[1] = m;
    p[2] = pack_bf16x2(r - __uint_as_float(m << 16), 0.0f) & 0xFFFFu;
}

// Eight values -> 16 bytes of each of the three planes.
__device__ __forceinline__ void split3x8(const float (&v)[8], uint4 (&out)[3])
{
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a[3], b[3];
        split3(v[2 * i], a);
        split3(v[2 * i + 1], b);
#pragma unroll
        for (int p = 0; p < 3; ++p)
            w[p][i] = a[p] | (b[p] << 16);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
        out[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

struct SplitArgs {
    const int32_t *topk_idx;
    const float *topk_w, *dtopk_w;  // dtopk_w nullable
    const float *dlogits;           // nullable
    const uint8_t *mask;            // nullable
    const float *wr;                // nullable: no planes of the router weights wanted
    int N, E, K, d;
    int pitch;        // E rounded up to 8: columns of a row of the planes
    uint16_t *dl;     // [3][N][pitch]
    uint16_t *wp;     // [3][E][d]
    float *bias_part; // [token_blocks][E]
    int token_blocks;
};

constexpr int kSplitThreads = 256;

// Blocks [0, token_blocks): dl of their tokens, in planes, and its sum over them; LPR lanes per
// token, 8 neighbouring columns each (one 16-byte store per plane). The other blocks: the
// planes of the router weights.
template <int LPR>
__global__ void __launch_bounds__(kSplitThreads) router_split_grad_kernel(const SplitArgs a)
{
    constexpr int GW = 32 / LPR, WARPS = kSplitThreads / 32;
    const int tid = threadIdx.x;
    if ((int)blockIdx.x >= a.token_blocks) {
        const int64_t n = (int64_t)a.E * a.d / 8;  // d % 8 == 0
        const int64_t step = (int64_t)(gridDim.x - a.token_blocks) * kSplitThreads;
        for (int64_t i = (int64_t)(blockIdx.x - a.token_blocks) * kSplitThreads + tid; i < n;
             i += step) {
            const float4 lo = reinterpret_cast<const float4 *>(a.wr)[2 * i];
            const float4 hi = reinterpret_cast<const float4 *>(a.wr)[2 * i + 1];
            const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint4 out[3];
            split3x8(v, out);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                reinterpret_cast<uint4 *>(a.wp)[p * n + i] = out[p];
        }
        return;
    }
    __shared__ float s_sum[WARPS * LPR * 8];
    const int warp = tid >> 5, lane = tid & 31, l = lane % LPR, grp = lane / LPR;
    const int c0 = 8 * l, E = a.E, K = a.K;
    const size_t plane = (size_t)a.N * a.pitch;
    float sum[8] = {};
    const int64_t stride = (int64_t)a.token_blocks * WARPS * GW;
    for (int64_t t = ((int64_t)blockIdx.x * WARPS + warp) * GW + grp; t < a.N; t += stride) {
        const bool live = !a.mask || a.mask[t];
        float v[8] = {};
        if (live && a.dlogits) {
            const float *row = a.dlogits + t * E;
            if (E % 4 == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (c0 + 4 * i < E) {
                        const float4 q = *reinterpret_cast<const float4 *>(row + c0 + 4 * i);
                        v[4 * i] = q.x;
                        v[4 * i + 1] = q.y;
                        v[4 * i + 2] = q.z;
                        v[4 * i + 3] = q.w;
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + j < E)
                        v[j] = row[c0 + j];
            }
        }
        if (live && a.dtopk_w) {
            const int32_t *idx = a.topk_idx + t * K;
            const float *w = a.topk_w + t * K, *dw = a.dtopk_w + t * K;
            float s = 0.0f;
            for (int k = 0; k < K; ++k) {
                if ((unsigned)idx[k] < (unsigned)E)
                    s += w[k] * dw[k];
                else if (l == 0)
                    set_dev_error(MOE_ERR_DEVICE_BOUNDS);
            }
            for (int k = 0; k < K; ++k) {
                const int c = idx[k] - c0;
                if ((unsigned)idx[k] < (unsigned)E && (unsigned)c < 8u) {
                    const float g = w[k] * (dw[k] - s);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] += j == c ? g : 0.0f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[j] += v[j];
        if (c0 < a.pitch) {
            uint4 out[3];
            split3x8(v, out);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint4 *>(a.dl + p * plane + t * a.pitch + c0) = out[p];
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
        a.bias_part[(size_t)blockIdx.x * E + tid] = s;
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

// Shared-memory matrix descriptor of an operand whose rows of shared memory run along K (the
// M or N index is the contiguous one): boxes of [K][64 elements], 128-byte swizzle; 8 K rows are
// 1024 bytes, the next 64 elements of M or N are one box of `box_bytes` further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t box_bytes)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// bf16 operands, fp32 accumulate; which operand is the M- or N-contiguous kind.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn, bool b_mn)
{
    return gg::instr_desc_bf16(M, N) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
}

struct Span {  // work items [u0, u1) of CTA c of G: an even, contiguous share of U
    int64_t u0, u1;
    __host__ __device__ Span(int64_t U, int G, int c) : u0(U * c / G), u1(U * (c + 1) / G) {}
};
// The CTA whose span holds item v.
__host__ __device__ inline int span_owner(int64_t U, int G, int64_t v)
{
    return (int)(((v + 1) * G - 1) / U);
}

// ---------------------------------------------------------------- dWr = dl^T x

// D[d'][e] over a chunk of kChunk tokens: M = d' (MT tiles of 128 columns of x), N = e, K =
// tokens. Both operands lie in memory with the token as the slow index, so both are the
// M/N-contiguous kind. A chunk's sum is read back and added to fp32 registers before it is
// longer than 128 tokens: the tensor core's accumulator truncates, and a truncation per step
// over tens of thousands of tokens would cost the low bits that the split keeps.
constexpr int kTok = 64;     // tokens of a shared-memory stage
constexpr int kChunk = 128;  // tokens of a work item (accumulated in TMEM)
constexpr int kDwThreads = 384;

template <int NE, int MT>
struct DwTile {
    static constexpr int STAGE = (2 * MT + 3 * NE) * kBox;
    static constexpr int STAGES = 231168 / STAGE > 4 ? 4 : 231168 / STAGE;  // within 227 KB
    static constexpr int SMEM = STAGES * STAGE + 1024 + 256;
    static constexpr int REGS = MT == 2 ? 64 * NE : 32 * NE;  // columns of one epilogue thread
    static_assert(STAGES >= 2 && 2 * MT * 64 * NE <= 512, "tile");
};

struct DwArgs {
    int N, d, E;
    int tiles;       // column tiles of 128 MT
    int chunks;      // chunks of kChunk tokens
    int kmax;        // partial results kept per tile, at most
    const uint8_t *mask;
    float *part;     // [tiles][kmax][E][128 MT]
    uint64_t timeout_ns;
};

// Warps: 0 TMA, 1 MMA, 2 zeroes the rows of x of masked tokens (a masked row may hold NaN, and
// 0 * NaN would reach every sum), 4..11 the running sums.
template <int NE, int MT>
__global__ void __launch_bounds__(kDwThreads, 1)
    router_dw_kernel(const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_dl, const DwArgs a)
{
    using T = DwTile<NE, MT>;
    constexpr int S = T::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S * T::STAGE);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 3 * S + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t base = smem_u32(smem), bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto clean = [&](int s) { return bar0 + 8u * (S + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 * S + s); };
    auto tfull = [&](int i) { return bar0 + 8u * (3 * S + i); };
    auto tempty = [&](int i) { return bar0 + 8u * (3 * S + 2 + i); };
    const uint32_t done = bar0 + 8u * (3 * S + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Span span((int64_t)a.tiles * a.chunks, gridDim.x, blockIdx.x);

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
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    gg::tc_fence_before();
    __syncthreads();
    gg::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // stages of chunk c: the last one may have tokens for one stage only
    auto stages_of = [&](int64_t c) {
        const int64_t left = a.N - c * kChunk;
        return left > kTok ? 2 : 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, last[S];
            bool issued[S];
            for (int s = 0; s < S; ++s)
                issued[s] = false;
            bool ok = true;
            for (int64_t u = span.u0; u < span.u1 && ok; ++u) {
                const int64_t tile = u / a.chunks, c = u - tile * a.chunks;
                for (int q = 0; q < stages_of(c); ++q) {
                    if (!gg::mbar_wait(empty(stage), phase ^ 1u, abort_flag, a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + stage * T::STAGE;
                    const int t0 = (int)(c * kChunk) + q * kTok;
                    mbar_arrive_expect_tx(full(stage), T::STAGE);
#pragma unroll
                    for (int b = 0; b < 2 * MT; ++b)
                        gg::tma_load_2d(dst + b * kBox, &tm_x, (int)tile * 128 * MT + 64 * b, t0,
                                        full(stage));
#pragma unroll
                    for (int p = 0; p < 3; ++p)
#pragma unroll
                        for (int b = 0; b < NE; ++b)
                            tma_load_3d(dst + (2 * MT + p * NE + b) * kBox, &tm_dl, 64 * b, t0, p,
                                        full(stage));
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
        if (lane == 0) {
            const int n = (a.E + 15) & ~15;
            const uint32_t id = idesc(128, n, true, true);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t u = span.u0; u < span.u1 && ok; ++u) {
                const int64_t c = u % a.chunks;
                if (!gg::mbar_wait(tempty(acc), acc_phase ^ 1u, abort_flag, a.timeout_ns))
                    break;
                gg::tc_fence_after();
                const uint32_t d0 = tmem + (uint32_t)(acc * MT * 64 * NE);
                const int ns = stages_of(c);
                for (int q = 0; q < ns; ++q) {
                    if (!gg::mbar_wait(a.mask ? clean(stage) : full(stage), phase, abort_flag,
                                       a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    gg::tc_fence_after();
                    const uint32_t xa = base + stage * T::STAGE, pb = xa + 2 * MT * kBox;
#pragma unroll
                    for (int p = 2; p >= 0; --p)  // the small terms first
#pragma unroll
                        for (int k = 0; k < kTok / 16; ++k)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                gg::tc_mma<0>(d0 + mt * 64 * NE,
                                              smem_desc_mn_sw128(xa + 2 * mt * kBox + k * 2048, kBox),
                                              smem_desc_mn_sw128(pb + p * NE * kBox + k * 2048, kBox),
                                              id, (q > 0 || p < 2 || k > 0) ? 1u : 0u);
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
    } else if (warp == 2) {
        if (a.mask) {
            int stage = 0;
            uint32_t phase = 0;
            int ok = 1;
            for (int64_t u = span.u0; u < span.u1 && ok; ++u) {
                const int64_t c = u % a.chunks;
                const int ns = stages_of(c);
                for (int q = 0; q < ns; ++q) {
                    const int64_t t0 = c * kChunk + q * kTok;
                    uint32_t gone[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int64_t t = t0 + 32 * i + lane;
                        gone[i] = __ballot_sync(0xffffffffu, t < a.N && !a.mask[t]);
                    }
                    if (lane == 0)
                        ok = gg::mbar_wait(full(stage), phase, abort_flag, a.timeout_ns) ? 1 : 0;
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok)
                        break;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        for (uint32_t m = gone[i]; m; m &= m - 1) {
                            // a row of each of the 2 MT boxes: 128 bytes, 8 lanes
                            const int row = 32 * i + __ffs(m) - 1;
                            if (lane < 16 * MT) {
                                const uint32_t at = base + stage * T::STAGE + (lane >> 3) * kBox +
                                                    row * 128 + (lane & 7) * 16;
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at),
                                             "r"(0)
                                             : "memory");
                            }
                        }
                    gg::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(clean(stage));
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= 4) {
        // lane quadrant of TMEM: rows d'; the two warps of a quadrant take an M tile each
        // (MT = 2) or half of the columns
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int mt = MT == 2 ? half : 0, col0 = MT == 2 ? 0 : half * T::REGS;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        float sum[T::REGS];
#pragma unroll
        for (int j = 0; j < T::REGS; ++j)
            sum[j] = 0.0f;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int64_t u = span.u0; u < span.u1; ++u) {
            int ok = 0;
            if (lane == 0)
                ok = gg::mbar_wait(tfull(acc), acc_phase, abort_flag, a.timeout_ns) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok)
                break;
            gg::tc_fence_after();
            const uint32_t ta = tmem + lanes + (uint32_t)(acc * MT * 64 * NE + mt * 64 * NE + col0);
#pragma unroll
            for (int j = 0; j < T::REGS; j += 16) {
                if (col0 + j >= a.E)
                    break;  // columns no MMA has written
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
            const int64_t tile = u / a.chunks;
            if (u + 1 == span.u1 || (u + 1) / a.chunks != tile) {
                const int k = (int)blockIdx.x - span_owner((int64_t)a.tiles * a.chunks, gridDim.x,
                                                           tile * a.chunks);
                float *dst = a.part + ((size_t)tile * a.kmax + k) * a.E * (128 * MT) + mt * 128 +
                             q * 32 + lane;
#pragma unroll
                for (int j = 0; j < T::REGS; ++j) {
                    if (col0 + j < a.E)
                        dst[(size_t)(col0 + j) * (128 * MT)] = sum[j];
                    sum[j] = 0.0f;
                }
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
    int tile_cols, tiles, chunks, kmax, G;  // dWr's partial results (part null: dWr not wanted)
    const float *part;
    float *dw;
    int dw_blocks;
    const float *bias_part;  // [bias_parts][E]
    int bias_parts;
    float *dbias;
};

// dWr and dbias from their partial results, each element in the order of the tokens.
__global__ void __launch_bounds__(256) router_sum_kernel(const SumArgs a)
{
    if ((int)blockIdx.x < a.dw_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 4 columns of one expert
        const int64_t per_row = a.d / 4;
        if (i >= per_row * a.E)
            return;
        const int e = (int)(i / per_row), c = 4 * (int)(i - e * per_row);
        const int tile = c / a.tile_cols;
        const int64_t U = (int64_t)a.tiles * a.chunks, v0 = (int64_t)tile * a.chunks;
        const int n = span_owner(U, a.G, v0 + a.chunks - 1) - span_owner(U, a.G, v0) + 1;
        const float *p = a.part + ((size_t)tile * a.kmax * a.E + e) * a.tile_cols +
                         (c - tile * a.tile_cols);
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = 0; k < n; ++k) {
            const float4 q = *reinterpret_cast<const float4 *>(p + (size_t)k * a.E * a.tile_cols);
            s.x += q.x;
            s.y += q.y;
            s.z += q.z;
            s.w += q.w;
        }
        *reinterpret_cast<float4 *>(a.dw + (size_t)e * a.d + c) = s;
        return;
    }
    // dbias: 32 experts a block, 8 threads of each
    __shared__ double red[8][32];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int e = ((int)blockIdx.x - a.dw_blocks) * 32 + lane;
    double s = 0.0;
    if (e < a.E)
        for (int b = row; b < a.bias_parts; b += 8)
            s += a.bias_part[(size_t)b * a.E + e];
    red[row][lane] = s;
    __syncthreads();
    if (row == 0 && e < a.E) {
        for (int r = 1; r < 8; ++r)
            s += red[r][lane];
        a.dbias[e] = (float)s;
    }
}

// ---------------------------------------------------------------- dx = dl Wr (+ dx_add)

// D[t][d']: M = 128 tokens, N = BN columns, K = e. A CTA keeps its BN columns of the router
// weights' planes in shared memory (BN: as many of 256, 128, 64 as fit) and walks over token
// tiles, whose planes of dl stream through a ring of [128 tokens][64 experts] units. A unit of
// plane i meets the planes j <= planes - 1 - i of the weights. The work items are ordered columns
// first, then tokens, and split evenly over the CTAs, so a CTA loads its weights once or twice.
constexpr int kDxThreads = 192;
constexpr int kUnit = 16384;   // 128 tokens x 64 experts, bf16
constexpr int kPiece = 4096;   // 32 tokens x 128 bytes of dx: what one warp stores at a time
constexpr int kSlots = 3;      // pieces of a warp in flight
constexpr int kDxMaxB = 131072;
constexpr int kDxUnits = 2;    // ring units, at least (as many as fit, at most kDxMaxUnits)
constexpr int kDxMaxUnits = 6;
constexpr int kDxMaxSmem = 231424;

struct DxArgs {
    int N, d, E;
    int chunks;     // of 64 experts
    int bn;         // columns of a slice
    int slices;     // column slices
    int tiles;      // token tiles
    int units;      // ring units
    int add;        // dx_add is given
    uint64_t timeout_ns;
};

__host__ __device__ inline int dx_piece_area(bool bf16)
{
    // a slot: the piece stored, and with fp32 dx the bf16 piece of dx_add beside it
    return 4 * kSlots * (bf16 ? kPiece : kPiece + kPiece / 2);
}

template <bool BF16>
__global__ void __launch_bounds__(kDxThreads, 1)
    router_dx_kernel(const __grid_constant__ CUtensorMap tm_dl,
                     const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_dx,
                     const __grid_constant__ CUtensorMap tm_add, const DxArgs a)
{
    constexpr int PLANES = BF16 ? 2 : 3;
    constexpr int CP = BF16 ? 64 : 32;  // columns of a piece
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nb = a.bn / 64, wbytes = PLANES * a.chunks * nb * kBox;
    const uint32_t w_base = smem_u32(smem), a_base = w_base + wbytes;
    const uint32_t p_base = a_base + a.units * kUnit;  // kPiece areas, then (fp32) dx_add's
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + wbytes + a.units * kUnit +
                                                  dx_piece_area(BF16));
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kDxMaxUnits + s); };
    auto tfull = [&](int i) { return bar0 + 8u * (2 * kDxMaxUnits + i); };
    auto tempty = [&](int i) { return bar0 + 8u * (2 * kDxMaxUnits + 2 + i); };
    const uint32_t wfull = bar0 + 8u * (2 * kDxMaxUnits + 4);
    const uint32_t wfree = bar0 + 8u * (2 * kDxMaxUnits + 5);
    const uint32_t done = bar0 + 8u * (2 * kDxMaxUnits + 6);
    auto addfull = [&](int w, int s) { return bar0 + 8u * (2 * kDxMaxUnits + 7 + w * kSlots + s); };
    uint32_t *tmem_slot =
        reinterpret_cast<uint32_t *>(bars + 2 * kDxMaxUnits + 7 + 4 * kSlots);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Span span((int64_t)a.slices * a.tiles, gridDim.x, blockIdx.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kDxMaxUnits; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            mbar_init(tempty(i), 4);
        }
        mbar_init(wfull, 1);
        mbar_init(wfree, 1);
        mbar_init(done, 1);
        for (int i = 0; i < 4 * kSlots; ++i)
            mbar_init(addfull(i / kSlots, i % kSlots), 1);
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
            int64_t have = -1;
            int loads = 0;  // slices loaded
            for (int64_t u = span.u0; u < span.u1 && ok; ++u) {
                const int64_t slice = u / a.tiles, tile = u - slice * a.tiles;
                if (slice != have) {
                    // the weights of the next slice, once the MMAs of the last one are done
                    if (loads > 0 && !gg::mbar_wait(wfree, (uint32_t)(loads - 1) & 1u, abort_flag,
                                                    a.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    have = slice;
                    ++loads;
                    mbar_arrive_expect_tx(wfull, wbytes);
                    for (int p = 0; p < PLANES; ++p)
                        for (int c = 0; c < a.chunks; ++c)
                            for (int b = 0; b < nb; ++b)
                                tma_load_3d(w_base + ((p * a.chunks + c) * nb + b) * kBox, &tm_w,
                                            (int)slice * a.bn + 64 * b, 64 * c, p, wfull);
                }
                for (int p = PLANES - 1; p >= 0 && ok; --p)
                    for (int c = 0; c < a.chunks; ++c) {
                        if (!gg::mbar_wait(empty(stage), phase ^ 1u, abort_flag, a.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(full(stage), kUnit);
                        tma_load_3d(a_base + stage * kUnit, &tm_dl, 64 * c, (int)tile * 128, p,
                                    full(stage));
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
            if (loads > 0)
                gg::mbar_wait(wfull, (uint32_t)(loads - 1) & 1u, abort_flag, a.timeout_ns, false);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id = idesc(128, a.bn, false, true);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            int64_t have = -1;
            int loads = 0;
            for (int64_t u = span.u0; u < span.u1 && ok; ++u) {
                const int64_t slice = u / a.tiles;
                if (slice != have) {
                    if (!gg::mbar_wait(wfull, (uint32_t)loads & 1u, abort_flag, a.timeout_ns))
                        break;
                    have = slice;
                    ++loads;
                }
                if (!gg::mbar_wait(tempty(acc), acc_phase ^ 1u, abort_flag, a.timeout_ns))
                    break;
                gg::tc_fence_after();
                const uint32_t d0 = tmem + (uint32_t)(acc * 256);
                uint32_t accumulate = 0;
                for (int p = PLANES - 1; p >= 0 && ok; --p)
                    for (int c = 0; c < a.chunks; ++c) {
                        if (!gg::mbar_wait(full(stage), phase, abort_flag, a.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        gg::tc_fence_after();
                        const int ks = min(4, (a.E - 64 * c + 15) / 16);
                        for (int j = PLANES - 1 - p; j >= 0; --j)
                            for (int k = 0; k < ks; ++k) {
                                gg::tc_mma<0>(
                                    d0, gg::smem_desc_sw128(a_base + stage * kUnit + k * 32),
                                    smem_desc_mn_sw128(
                                        w_base + (j * a.chunks + c) * nb * kBox + k * 2048, kBox),
                                    id, accumulate);
                                accumulate = 1;
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
                if (u + 1 < span.u1 && (u + 1) / a.tiles != slice)
                    gg::tc_commit(wfree);
            }
            gg::tc_commit(done);
            gg::mbar_wait(done, 0, abort_flag, a.timeout_ns, false);
        }
    } else {
        // ---------------- epilogue: warps 2..5, TMEM lane quadrant = warp % 4
        const int q = warp & 3;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const uint32_t slots = p_base + q * kSlots * kPiece;
        const uint32_t adds = BF16 ? slots : p_base + 4 * kSlots * kPiece + q * kSlots * (kPiece / 2);
        constexpr int ADD_SLOT = BF16 ? kPiece : kPiece / 2;
        const int pieces = a.bn / CP;
        const int64_t total = (span.u1 - span.u0) * pieces;
        // piece i of this CTA: its column and its first token (of this warp's 32)
        auto place = [&](int64_t i, int &col, int &row) {
            const int64_t u = span.u0 + i / pieces, slice = u / a.tiles;
            col = (int)slice * a.bn + (int)(i % pieces) * CP;
            row = (int)(u - slice * a.tiles) * 128 + q * 32;
        };
        auto fetch = [&](int64_t i) {  // lane 0: dx_add's piece i into its slot
            int col, row;
            place(i, col, row);
            const int s = (int)(i % kSlots);
            mbar_arrive_expect_tx(addfull(q, s), ADD_SLOT);
            gg::tma_load_2d(adds + s * ADD_SLOT, &tm_add, col, row, addfull(q, s));
        };
        int64_t fetched = 0, used = 0;
        if (a.add && lane == 0)
            for (; fetched < total && fetched < kSlots - 1; ++fetched)
                fetch(fetched);
        int acc = 0;
        uint32_t acc_phase = 0;
        int ok = 1;
        for (int64_t u = span.u0; u < span.u1 && ok; ++u) {
            if (lane == 0)
                ok = gg::mbar_wait(tfull(acc), acc_phase, abort_flag, a.timeout_ns) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok)
                break;
            gg::tc_fence_after();
            for (int pc = 0; pc < pieces; ++pc) {
                const int64_t i = (u - span.u0) * pieces + pc;
                const int s = (int)(i % kSlots);
                const uint32_t slot = slots + s * kPiece;
                uint32_t v[CP];
#pragma unroll
                for (int c = 0; c < CP / 16; ++c)
                    gg::tmem_ld16(tmem + lanes + acc * 256 + pc * CP + 16 * c,
                                  *reinterpret_cast<uint32_t(*)[16]>(v + 16 * c));
                if (lane == 0) {
                    if (a.add) {
                        ok = gg::mbar_wait(addfull(q, s), (uint32_t)(i / kSlots) & 1u, abort_flag,
                                           a.timeout_ns) ? 1 : 0;
                        if (ok)
                            ++used;
                    } else {
                        // the store that last read this slot has done so
                        asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kSlots - 1) : "memory");
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                gg::tmem_ld_wait();
                if (!ok)
                    break;
                if (a.add) {
#pragma unroll
                    for (int c = 0; c < CP / 8; ++c) {
                        // 16 bytes = 8 columns; rows of 128 bytes (bf16 dx) or 64 bytes
                        const uint32_t at = adds + s * ADD_SLOT +
                                            (BF16 ? lane * 128 + ((c ^ (lane & 7)) << 4)
                                                  : lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(at));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[8 * c + 2 * j] = __float_as_uint(
                                __uint_as_float(v[8 * c + 2 * j]) + bf16_lo(w[j]));
                            v[8 * c + 2 * j + 1] = __float_as_uint(
                                __uint_as_float(v[8 * c + 2 * j + 1]) + bf16_hi(w[j]));
                        }
                    }
                    if (!BF16 && lane == 0)  // the slot's last store has read it
                        asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kSlots - 1) : "memory");
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (BF16)
                            w[j] = pack_bf16x2(__uint_as_float(v[8 * c + 2 * j]),
                                               __uint_as_float(v[8 * c + 2 * j + 1]));
                        else
                            w[j] = v[4 * c + j];
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     slot + lane * 128 + ((c ^ (lane & 7)) << 4)),
                                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
                gg::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    int col, row;
                    place(i, col, row);
                    if (col < a.d && row < a.N)
                        gg::tma_store_2d(&tm_dx, slot, col, row);
                    else
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    if (a.add && fetched < total) {
                        // into the slot before this one: its store has read it
                        if (BF16)
                            gg::bulk_wait_read1();
                        fetch(fetched++);
                    }
                }
            }
            gg::tc_fence_before();
            __syncwarp();
            if (!ok)
                break;
            if (lane == 0)
                mbar_arrive(tempty(acc));
            acc ^= 1;
            if (acc == 0)
                acc_phase ^= 1u;
        }
        if (lane == 0) {
            for (; used < fetched; ++used)  // after a timeout: copies in flight have landed
                gg::mbar_wait(addfull(q, (int)(used % kSlots)), (uint32_t)(used / kSlots) & 1u,
                              abort_flag, a.timeout_ns, false);
            gg::bulk_wait_all();
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

}  // namespace rb
}  // namespace moe
