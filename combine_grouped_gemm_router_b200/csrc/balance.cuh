// Balance loss of the router with the per-expert counts it rests on, and its gradient.
//
// With p_t the softmax of token t's E logits, lse_t their log-sum-exp, M the counted tokens
// (token_mask != 0), counts[e] the counted assignments to expert e and f_e = counts[e] / (M K):
//   P_e     = (1/M) sum_t p_te
//   balance = E sum_e f_e P_e          z = (1/M) sum_t lse_t^2
//   loss    = cb balance + cz z
//   dloss/dl_te = p_te (cb E / M (f_e - sum_j f_j p_tj) + cz 2 / M lse_t)
// (the counts are constants: no gradient passes through the selection).
//
// Both passes read the [N][E] logits once. A row is held by LPR lanes, up to 16 columns each, so
// the softmax's maximum and sum are log2(LPR) shuffles and a lane owns the same columns in every
// row it sees: the sums over tokens stay in its registers until the end of the block. With 8
// columns a lane the shuffles were a third of the instructions. The sums (131072 x 256 with a
// mask: 33 us, of which 4 in balance_finish_kernel) read the next row's logits while a row is
// worked on; their loop streams at about 6 TB/s, the rest is the start and the end of the two
// kernels. The gradient (30011 x 160: 10 us, its bytes 6) waits for memory: a row is loaded, worked
// on and stored before the next one is loaded (issue slots half busy, 7 warps of an issue waiting
// for loads), and the grid's 3.2 passes over the rows cost 4.
#pragma once

#include "common.cuh"

namespace moe {

// Registers for two rows a lane; 131072 x 256: 33.0 us, 33.7 with 768, 36.6 with 1024 (64
// registers a thread are too few), 36.8 with 640. A ring of rows in shared memory instead of
// the registers: 35.4.
constexpr int kBalThreads = 896;

// Lane l of the LPR lanes of a row holds C = 4 NC columns col(j): NC 16-byte chunks (VEC,
// E % 4 == 0) or C columns LPR apart. A column at or past E reads as -inf (probability 0).
template <int LPR, int NC, bool VEC>
struct RowSlice {
    static constexpr int C = 4 * NC;
    static __device__ __forceinline__ int col(int l, int j)
    {
        return VEC ? 4 * (l + LPR * (j / 4)) + (j & 3) : l + LPR * j;
    }
    static __device__ __forceinline__ void load(const float *row, int E, int l, float (&v)[C])
    {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = 4 * (l + LPR * i);
                const float4 q = c < E ? *reinterpret_cast<const float4 *>(row + c)
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                v[4 * i] = q.x;
                v[4 * i + 1] = q.y;
                v[4 * i + 2] = q.z;
                v[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c = l + LPR * j;
                v[j] = c < E ? row[c] : -INFINITY;
            }
        }
    }
    static __device__ __forceinline__ void store(float *row, int E, int l, const float (&v)[C])
    {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = 4 * (l + LPR * i);
                if (c < E)
                    *reinterpret_cast<float4 *>(row + c) =
                        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int c = l + LPR * j;
                if (c < E)
                    row[c] = v[j];
            }
        }
    }
};

// Two fp32 values in a register pair: one instruction for both.
struct Pair {
    unsigned long long r;
    __device__ __forceinline__ Pair(float lo, float hi)
    {
        asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    }
    __device__ __forceinline__ void get(float &lo, float &hi) const
    {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
    }
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)  // a b + c
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c.r) : "l"(a.r), "l"(b.r));
    return c;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.r) : "l"(b.r));
    return a;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.r) : "l"(b.r));
    return a;
}

template <int LPR>
__device__ __forceinline__ float row_max(float v)
{
#pragma unroll
    for (int off = LPR / 2; off; off >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int off = LPR / 2; off; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Softmax of the row in v, in place: exponentials relative to the row's maximum, not yet divided
// by their sum. Returns the sum; lse: the log-sum-exp. With L = log2(e), e^(v - m) is
// 2^(v L - m L), one fused multiply-add: the rounding of m L is common to the row and cancels in
// the probabilities. That holds while it is small against 1: a row whose maximum is past 2^20
// (m L off by up to 2^-4 there, by infinity at the type's lowest value) subtracts m first.
// Results below fp32's normal range are 0.
template <int LPR, int C>
__device__ __forceinline__ float row_softmax(float (&v)[C], float &lse)
{
    constexpr float kL = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
    float m = v[0];
#pragma unroll
    for (int j = 1; j < C; ++j)
        m = fmaxf(m, v[j]);
    m = row_max<LPR>(m);
    float c = -m * kL;
    if (fabsf(m) > 1048576.0f) {
#pragma unroll
        for (int j = 0; j < C; ++j)
            v[j] -= m;
        c = 0.0f;
    }
    __syncwarp();
    Pair sum(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < C; j += 2) {
        float a, b;
        fma2(Pair(v[j], v[j + 1]), Pair(kL, kL), Pair(c, c)).get(a, b);
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[j]) : "f"(a));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[j + 1]) : "f"(b));
        sum = add2(sum, Pair(v[j], v[j + 1]));
    }
    float s, s1;
    sum.get(s, s1);
    s = row_sum<LPR>(s + s1);
    float l2;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(l2) : "f"(s));
    lse = fmaf(l2, kLn2, m);
    return s;
}

// One block's share of the sums, in the workspace: probability sums [blocks][E], counts
// [blocks][E], then {sum of lse^2, counted tokens} per block.
struct BalanceParts {
    float *prob;
    int32_t *count;
    float2 *zm;  // {sum of lse^2, tokens as int bits}
};

struct BalanceOut {
    float *loss;         // [3]: loss, balance, z
    int32_t *counts;     // [E]
    float *prob_mean;    // [E]
    int32_t *tokens;     // [1]
    float cb, cz;
    int E, K;
};

// The totals of a whole call -> its outputs. Thread e < E of the block brings expert e's sums.
__device__ __forceinline__ void balance_outputs(const BalanceOut &o, double prob, int count,
                                                double z, int tokens, double *red)
{
    const int e = threadIdx.x;
    const double inv_m = tokens > 0 ? 1.0 / tokens : 0.0;
    double term = 0.0;
    if (e < o.E) {
        o.counts[e] = count;
        o.prob_mean[e] = (float)(prob * inv_m);
        term = (double)count / o.K * inv_m * (prob * inv_m);
    }
    term = warp_sum(term);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        double bal = 0.0;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w)
            bal += red[w];
        bal *= o.E;
        const double zz = z * inv_m;
        o.loss[0] = (float)(o.cb * bal + (o.cz != 0.0f ? o.cz * zz : 0.0));  // zz may be inf
        o.loss[1] = (float)bal;
        o.loss[2] = (float)zz;
        o.tokens[0] = tokens;
    }
}

// Sums over this block's tokens. A grid of one block also writes the outputs.
template <int LPR, int NC, bool VEC>
__global__ void __launch_bounds__(kBalThreads, 1)
    balance_sums_kernel(const float *__restrict__ logits, const int32_t *__restrict__ topk_idx,
                        const uint8_t *__restrict__ mask, int N, BalanceParts parts,
                        BalanceOut out)
{
    using Slice = RowSlice<LPR, NC, VEC>;
    constexpr int C = Slice::C;
    constexpr int GW = 32 / LPR;  // rows of a warp at once
    constexpr int WARPS = kBalThreads / 32;
    __shared__ float s_prob[WARPS * LPR * C];  // up to 256 columns a warp
    __shared__ int s_count[256];
    __shared__ float s_z[WARPS];
    __shared__ int s_m[WARPS];
    __shared__ double s_red[WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int l = lane % LPR, grp = lane / LPR;
    const int E = out.E, K = out.K;
    grid_go();
    if (tid < 256)
        s_count[tid] = 0;
    __syncthreads();

    float acc[C] = {};
    float zsum = 0.0f;
    int m_tok = 0;
    bool bad_index = false, bad_logit = false;
    const int64_t stride = (int64_t)gridDim.x * WARPS * GW;
    // a row is loaded while the one before it is worked on
    struct {
        float v[C];
        int e;  // this lane's first slot
        bool inside, live;
    } next;
    auto fetch = [&](int64_t base) {
        const int64_t t = base + grp;
        next.inside = t < N;
        next.live = next.inside && (!mask || mask[t]);
        Slice::load(logits + (next.inside ? t : 0) * E, next.inside ? E : 0, l, next.v);
        next.e = next.inside && l < K ? topk_idx[t * K + l] : 0;
    };
    int64_t base = ((int64_t)blockIdx.x * WARPS + warp) * GW;
    if (base < N)
        fetch(base);
    for (; base < N; base += stride) {
        const int64_t t = base + grp;
        const bool inside = next.inside, live = next.live;
        const int first = next.e;
        float v[C];
#pragma unroll
        for (int j = 0; j < C; ++j)
            v[j] = next.v[j];
        if (base + stride < N)
            fetch(base + stride);
        // counts: lane l takes the slots l, l + LPR, ... of its token
        for (int k = l; k < K; k += LPR) {
            const int e = k == l ? first : inside ? topk_idx[t * K + k] : 0;
            const bool ok = (unsigned)e < (unsigned)E;
            if (live && ok)
                atomicAdd(&s_count[e], 1);
            bad_index |= live && !ok;
        }
        if (__any_sync(0xffffffffu, !live)) {  // keeps the arithmetic of a row left out finite
#pragma unroll
            for (int j = 0; j < C; ++j)
                v[j] = live ? v[j] : 0.0f;
        }
        float lse;
        const float s = row_softmax<LPR>(v, lse);
        const float inv = live ? __fdividef(1.0f, s) : 0.0f;
#pragma unroll
        for (int j = 0; j < C; j += 2)
            fma2(Pair(v[j], v[j + 1]), Pair(inv, inv), Pair(acc[j], acc[j + 1]))
                .get(acc[j], acc[j + 1]);
        lse = live ? lse : 0.0f;
        bad_logit |= !isfinite(lse);
        zsum = fmaf(lse, lse, zsum);
        m_tok += live;
    }
    if (bad_index)
        set_dev_error(MOE_ERR_DEVICE_BOUNDS);
    if (bad_logit)
        set_dev_error(MOE_ERR_NONFINITE);
    if (l != 0) {  // every lane of a row has them
        zsum = 0.0f;
        m_tok = 0;
    }

    // over the row groups of the warp, then over the warps
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
#pragma unroll
        for (int j = 0; j < C; ++j)
            acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], off);
    }
    if (grp == 0) {
#pragma unroll
        for (int j = 0; j < C; ++j)
            s_prob[warp * (LPR * C) + Slice::col(l, j)] = acc[j];
    }
    zsum = warp_sum(zsum);
    m_tok = warp_sum(m_tok);
    if (lane == 0) {
        s_z[warp] = zsum;
        s_m[warp] = m_tok;
    }
    __syncthreads();
    float p = 0.0f;
    if (tid < E) {
#pragma unroll 8
        for (int w = 0; w < WARPS; ++w)
            p += s_prob[w * (LPR * C) + tid];
    }
    float z = 0.0f;
    int mt = 0;
    if (tid == 0 || gridDim.x == 1) {
        for (int w = 0; w < WARPS; ++w) {
            z += s_z[w];
            mt += s_m[w];
        }
    }
    if (gridDim.x == 1) {
        balance_outputs(out, p, tid < E ? s_count[tid] : 0, z, mt, s_red);
    } else {
        if (tid < E) {
            parts.prob[(size_t)blockIdx.x * E + tid] = p;
            parts.count[(size_t)blockIdx.x * E + tid] = s_count[tid];
        }
        if (tid == 0)
            parts.zm[blockIdx.x] = make_float2(z, __int_as_float(mt));
    }
}

// Adds up the blocks' shares: a cluster of 8 blocks, 32 experts each, 32 threads an expert (a
// single block took 4 us longer to read the shares of 148 blocks). Every sum in a fixed order.
constexpr int kFinishBlocks = 8;

__global__ void __cluster_dims__(kFinishBlocks, 1, 1) __launch_bounds__(1024, 1)
    balance_finish_kernel(BalanceParts parts, int blocks, BalanceOut out)
{
    __shared__ double s_prob[32][33];
    __shared__ int s_count[32][33];
    __shared__ double s_term[kFinishBlocks];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = out.E;
    const int e = blockIdx.x * 32 + lane;
    // every block of the cluster has started before one writes to another's shared memory
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    grid_wait();
    double p = 0.0, z = 0.0;
    int c = 0, m = 0;
    if (e < E)
        for (int b = warp; b < blocks; b += 32) {
            p += parts.prob[(size_t)b * E + e];
            c += parts.count[(size_t)b * E + e];
        }
    s_prob[warp][lane] = p;
    s_count[warp][lane] = c;
    if (warp == 0) {
        for (int b = lane; b < blocks; b += 32) {
            const float2 q = parts.zm[b];
            z += q.x;
            m += __float_as_int(q.y);
        }
        z = warp_sum(z);
        m = warp_sum(m);
    }
    __syncthreads();
    if (warp == 0) {
        p = 0.0;
        c = 0;
        for (int w = 0; w < 32; ++w) {
            p += s_prob[w][lane];
            c += s_count[w][lane];
        }
        const double inv_m = m > 0 ? 1.0 / m : 0.0, mean = p * inv_m;
        if (e < E) {
            out.counts[e] = c;
            out.prob_mean[e] = (float)mean;
        }
        const double term = warp_sum((double)c / out.K * inv_m * mean);
        if (lane == 0) {  // to the first block
            uint32_t at;
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                         : "=r"(at)
                         : "r"(smem_u32(&s_term[blockIdx.x])));
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(term) : "memory");
        }
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        double bal = 0.0;
        for (int r = 0; r < kFinishBlocks; ++r)
            bal += s_term[r];
        const double inv_m = m > 0 ? 1.0 / m : 0.0, zz = z * inv_m;
        bal *= E;
        out.loss[0] = (float)(out.cb * bal + (out.cz != 0.0f ? out.cz * zz : 0.0));
        out.loss[1] = (float)bal;
        out.loss[2] = (float)zz;
        out.tokens[0] = m;
    }
}

// dlogits from the logits, the counts and the number of counted tokens.
template <int LPR, int NC, bool VEC>
__global__ void __launch_bounds__(256)
    balance_grad_kernel(const float *logits, const uint8_t *__restrict__ mask,
                        const int32_t *__restrict__ counts, const int32_t *__restrict__ tokens,
                        const float *__restrict__ dloss, int N, int E, int K, float cb, float cz,
                        float *dlogits)
{
    using Slice = RowSlice<LPR, NC, VEC>;
    constexpr int C = Slice::C;
    constexpr int GW = 32 / LPR;
    const int warp = (blockIdx.x * 256 + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPR, grp = lane / LPR;
    const int M = tokens[0];
    const float inv_m = M > 0 ? 1.0f / (float)M : 0.0f, inv_mk = inv_m / (float)K;
    const float scale = (dloss ? dloss[0] : 1.0f) * inv_m;
    const float a = scale * cb * (float)E, b = scale * cz * 2.0f;
    float f[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = Slice::col(l, j);
        f[j] = c < E ? a * ((float)counts[c] * inv_mk) : 0.0f;  // a f_e
    }
    const int64_t stride = (int64_t)(gridDim.x * 256 / 32) * GW;
    for (int64_t base = (int64_t)warp * GW; base < N; base += stride) {
        const int64_t t = base + grp;
        const bool inside = t < N, live = inside && M > 0 && (!mask || mask[t]);
        float v[C];
        Slice::load(logits + (inside ? t : 0) * E, inside ? E : 0, l, v);
        const bool any_out = __any_sync(0xffffffffu, !live);
        if (any_out) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                v[j] = live ? v[j] : 0.0f;
        }
        float lse;
        const float s = row_softmax<LPR>(v, lse);
        Pair dot2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < C; j += 2)
            dot2 = fma2(Pair(f[j], f[j + 1]), Pair(v[j], v[j + 1]), dot2);
        float dot, dot1;
        dot2.get(dot, dot1);
        dot = row_sum<LPR>(dot + dot1);
        const float inv = __fdividef(1.0f, s);
        // p (a (f - inner) + b lse) = e (a f + c) / sum
        const float c = b * lse - dot * inv;
#pragma unroll
        for (int j = 0; j < C; j += 2)
            mul2(mul2(Pair(v[j], v[j + 1]), Pair(inv, inv)), add2(Pair(f[j], f[j + 1]), Pair(c, c)))
                .get(v[j], v[j + 1]);
        if (any_out) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                v[j] = live ? v[j] : 0.0f;
        }
        if (inside)
            Slice::store(dlogits + t * E, E, l, v);
    }
}

}  // namespace moe
