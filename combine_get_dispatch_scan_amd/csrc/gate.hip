// The gate on gfx950: top-K of the experts' logits with their weights, the
// counts per expert and the balance loss, and its backward pass.
//
//   softmax  p = softmax(l), r = p;   sigmoid  r = s(l), p = r / sum r
//   choice   the K largest logits (both scores grow with the logit, so the
//            choice needs no rounding), ties to the lower id
//   weight   scale * r_k / sum of the chosen r, or scale * r_k
//   loss     coef * sum_e f_e P_e,  f_e = E n_e / (K V),  P_e = sum_t p_te / V
//            over the V tokens that count
//
// A token is held by kLanes lanes of a wave, NV values a lane, so the K rounds
// of "largest value, then smallest id that has it" run for 64 / kLanes tokens at
// once.  Every lane keeps the same experts from token to token: the sums of p
// stay in its registers until the workgroup is done.  The workgroups' sums are
// then added in their order by a second launch (or, where one workgroup holds
// all tokens, by the first), so the loss does not depend on timing.
#include "expert_launch.h"

namespace moe_ep {

constexpr int kGateThreads = 256;
constexpr int kGateMaxBlocks = 256;
constexpr float kNegInf = -__builtin_inff();

// Reductions over the LANES (16, 32 or 64) lanes that hold a token.
template <int LANES>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1)
        v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

template <int LANES>
__device__ __forceinline__ int group_min(int v)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1)
        v = min(v, __shfl_xor(v, d));
    return v;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}

// Expert of value v of lane j: four neighbouring experts a lane and step.
template <int LANES>
__device__ __forceinline__ int expert_of(int v, int j)
{
    return (v >> 2) * (4 * LANES) + j * 4 + (v & 3);
}

// The token's logits (absent experts: -inf).  VEC: rows of whole, aligned fours.
template <int LANES, int NV, bool BF16, bool VEC>
__device__ __forceinline__ void load_logits(const void* logits, int64_t at, int E, int j, float (&x)[NV])
{
#pragma unroll
    for (int v = 0; v < NV; v += 4) {
        const int e = expert_of<LANES>(v, j);
        if (VEC) {
            if (e < E) {
                if (BF16) {
                    const uint2 d = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + at + e);
                    x[v] = bf16_lo(d.x);
                    x[v + 1] = bf16_hi(d.x);
                    x[v + 2] = bf16_lo(d.y);
                    x[v + 3] = bf16_hi(d.y);
                } else {
                    const u32x4 d = load16_hint<false>(static_cast<const float*>(logits) + at + e);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        x[v + c] = __uint_as_float(d[c]);
                }
            } else {
                x[v] = x[v + 1] = x[v + 2] = x[v + 3] = kNegInf;
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[v + c] = kNegInf;
                if (e + c < E)
                    x[v + c] = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at + e + c] << 16)
                                    : static_cast<const float*>(logits)[at + e + c];
            }
        }
    }
}

// Scores r of the token's experts and the factor that turns them into p.
// A token without any expert left (every logit -inf) has r = 0 and p = 0.
template <int LANES, int NV, bool SIGMOID>
__device__ __forceinline__ float scores(const float (&x)[NV], float top, float (&r)[NV])
{
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (SIGMOID)
            r[v] = 1.0f / (1.0f + expf(-x[v]));
        else
            r[v] = top == kNegInf ? 0.0f : expf(x[v] - top);
        sum += r[v];
    }
    sum = group_sum<LANES>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (!SIGMOID) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            r[v] *= inv;
        return 1.0f;
    }
    return inv;
}

__device__ __forceinline__ void gate_finish(const GateLaunch& a, int blocks, float* lds)
{
    // thread: a stripe of workgroups of one expert; LDS: [stripes][E] sums, counts
    const int E = a.E, n = blockDim.x;
    const int stripes = n / E < 1 ? 1 : n / E;
    int* lds_n = reinterpret_cast<int*>(lds + (size_t)stripes * E);
    for (int i = threadIdx.x; i < stripes * E; i += n) {
        const int e = i % E, s = i / E;
        float p = 0.0f;
        int c = 0;
#pragma unroll 8
        for (int b = s; b < blocks; b += stripes) {
            p += a.part_p[(size_t)b * E + e];
            c += a.part_n[(size_t)b * (E + 1) + e];
        }
        lds[i] = p;
        lds_n[i] = c;
    }
    __shared__ int valid;
    __shared__ float wave_sum[16];
    if (threadIdx.x < kWave) {
        int c = 0;
        for (int b = threadIdx.x; b < blocks; b += kWave)
            c += a.part_n[(size_t)b * (E + 1) + E];
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1)
            c += __shfl_xor(c, d);
        if (threadIdx.x == 0)
            valid = c;
    }
    __syncthreads();
    const float V = (float)valid;
    float sum = 0.0f;
    for (int e = threadIdx.x; e < E; e += n) {
        float p = 0.0f;
        int c = 0;
        for (int s = 0; s < stripes; ++s) {
            p += lds[s * E + e];
            c += lds_n[s * E + e];
        }
        a.counts[e] = c;
        if (valid > 0)
            sum += ((float)c * (float)E / ((float)a.K * V)) * (p / V);
    }
    sum = group_sum<64>(sum);
    if ((threadIdx.x & (kWave - 1)) == 0)
        wave_sum[threadIdx.x / kWave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.0f;
        for (int w = 0; w < n / kWave; ++w)
            s += wave_sum[w];
        *a.loss = a.coef * s;
        *a.num_valid = valid;
    }
}

__global__ __launch_bounds__(1024) void gate_finish_kernel(GateLaunch a, int blocks)
{
    extern __shared__ float lds[];
    gate_finish(a, blocks, lds);
}

template <int LANES, int NV, bool BF16, bool VEC, bool SIGMOID>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateLaunch a)
{
    constexpr int kGroups = kGateThreads / LANES;      // tokens a workgroup holds at once
    __shared__ float sum_p[kGroups * LANES * NV];
    __shared__ int cnt[LANES * NV];
    __shared__ int cnt_valid;
    const int tid = threadIdx.x, j = tid % LANES, grp = tid / LANES;
    const int E = a.E, K = a.K;
    for (int i = tid; i < LANES * NV; i += kGateThreads)
        cnt[i] = 0;
    if (tid == 0)
        cnt_valid = 0;
    __syncthreads();
    float psum[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v)
        psum[v] = 0.0f;
    for (int t = blockIdx.x * kGroups + grp; t < a.T; t += gridDim.x * kGroups) {
        const bool masked = a.token_mask && a.token_mask[t] == 0;
        float x[NV], r[NV];
        // a masked token's logits are not looked at: they may hold anything
        load_logits<LANES, NV, BF16, VEC>(a.logits, (int64_t)t * a.ld, masked ? 0 : E, j, x);
        float top = x[0];
#pragma unroll
        for (int v = 1; v < NV; ++v)
            top = fmaxf(top, x[v]);
        top = group_max<LANES>(top);
        const float pf = scores<LANES, NV, SIGMOID>(x, top, r);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            psum[v] += r[v] * pf;
        if (j == 0 && top != kNegInf)
            atomicAdd(&cnt_valid, 1);
        // lane k keeps choice k
        int my_id = -1;
        float my_r = 0.0f, total = 0.0f;
        for (int k = 0; k < K; ++k) {
            float m = x[0];
#pragma unroll
            for (int v = 1; v < NV; ++v)
                m = fmaxf(m, x[v]);
            m = group_max<LANES>(m);
            int id = 0x7FFFFFFF;
            float rv = 0.0f;
#pragma unroll
            for (int v = NV - 1; v >= 0; --v)
                if (x[v] == m) {
                    id = expert_of<LANES>(v, j);
                    rv = r[v];
                }
            const int best = group_min<LANES>(id);
            if (m == kNegInf || best >= E)      // no expert is left (or NaN)
                break;
            const bool mine = best == id;
            rv = group_sum<LANES>(mine ? rv : 0.0f);
            total += rv;
            if (j == k) {
                my_id = best;
                my_r = rv;
            }
            if (mine) {
                atomicAdd(&cnt[best], 1);
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (expert_of<LANES>(v, j) == best)
                        x[v] = kNegInf;
            }
        }
        if (j < K) {
            float w = my_r;
            if (a.normalize)
                w = total == 0.0f ? 0.0f : my_r / total;
            a.topk_idx[(int64_t)t * K + j] = my_id;
            a.topk_weights[(int64_t)t * K + j] = w * a.scale;
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
        sum_p[grp * (LANES * NV) + expert_of<LANES>(v, j)] = psum[v];
    __syncthreads();
    for (int e = tid; e < E; e += kGateThreads) {
        float p = 0.0f;
        for (int g = 0; g < kGroups; ++g)
            p += sum_p[g * (LANES * NV) + e];
        a.part_p[(size_t)blockIdx.x * E + e] = p;
        a.part_n[(size_t)blockIdx.x * (E + 1) + e] = cnt[e];
    }
    if (tid == 0)
        a.part_n[(size_t)blockIdx.x * (E + 1) + E] = cnt_valid;
}

int gate_blocks(int T, int E)
{
    const int tokens = kGateThreads / (E <= 256 ? 16 : E <= 512 ? 32 : 64);
    const int64_t need = ((int64_t)T + tokens - 1) / tokens;
    return (int)(need < 1 ? 1 : need > kGateMaxBlocks ? kGateMaxBlocks : need);
}

template <int LANES, int NV, bool BF16, bool VEC>
static void gate_run(const GateLaunch& L, int blocks, hipStream_t stream)
{
    if (L.sigmoid)
        gate_kernel<LANES, NV, BF16, VEC, true><<<blocks, kGateThreads, 0, stream>>>(L);
    else
        gate_kernel<LANES, NV, BF16, VEC, false><<<blocks, kGateThreads, 0, stream>>>(L);
}

template <bool BF16, bool VEC>
static void gate_pick(const GateLaunch& L, int blocks, hipStream_t stream)
{
    if (L.E <= 64)
        gate_run<16, 4, BF16, VEC>(L, blocks, stream);
    else if (L.E <= 128)
        gate_run<16, 8, BF16, VEC>(L, blocks, stream);
    else if (L.E <= 256)
        gate_run<16, 16, BF16, VEC>(L, blocks, stream);
    else if (L.E <= 512)
        gate_run<32, 16, BF16, VEC>(L, blocks, stream);
    else
        gate_run<64, 16, BF16, VEC>(L, blocks, stream);
}

static bool whole_fours(const void* p, bool bf16, int64_t ld, int E)
{
    return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (bf16 ? 8 : 16) == 0;
}

hipError_t launch_gate(const GateLaunch& L, hipStream_t stream)
{
    const int blocks = gate_blocks(L.T, L.E);
    debug_launch("gate", dim3(blocks), dim3(kGateThreads), 0);
    const bool vec = whole_fours(L.logits, L.bf16, L.ld, L.E);
    if (L.bf16)
        vec ? gate_pick<true, true>(L, blocks, stream) : gate_pick<true, false>(L, blocks, stream);
    else
        vec ? gate_pick<false, true>(L, blocks, stream) : gate_pick<false, false>(L, blocks, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int stripes = 1024 / L.E < 1 ? 1 : 1024 / L.E;
    const size_t lds = (size_t)stripes * L.E * 8;
    debug_launch("gate_finish", dim3(1), dim3(1024), lds);
    gate_finish_kernel<<<1, 1024, lds, stream>>>(L, blocks);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// backward: the scores again from the logits, then
//   d_e = coef * grad_loss * E * n_e / (K V^2)     (d loss / d p_te, all tokens)
//   softmax  dl = p (d - <p, d>) + ...             sigmoid  ds = (d - <p, d>) / sum r + ...
// and for the chosen experts, with g = scale * grad_weights and wn = r / sum of
// the chosen r:  normalised  (g_k - <g, wn>) / sum of the chosen r  is added to
// d/dr_k, otherwise g_k.  dl = r (dr - <r, dr>) for softmax, r (1 - r) dr for sigmoid.
// ---------------------------------------------------------------------------
template <int LANES, int NV, bool BF16, bool VEC, bool SIGMOID>
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(GateBackwardLaunch a)
{
    constexpr int kGroups = kGateThreads / LANES;
    const int tid = threadIdx.x, j = tid % LANES, grp = tid / LANES;
    const int E = a.E, K = a.K;
    float d[NV];
    {
        const float V = (float)*a.num_valid;
        const float c = a.grad_loss && V > 0.0f ? a.coef * *a.grad_loss * ((float)E / ((float)K * V)) / V : 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int e = expert_of<LANES>(v, j);
            d[v] = e < E ? c * (float)a.counts[e] : 0.0f;
        }
    }
    for (int t = blockIdx.x * kGroups + grp; t < a.T; t += gridDim.x * kGroups) {
        const bool masked = a.token_mask && a.token_mask[t] == 0;
        float x[NV], r[NV], o[NV];
        load_logits<LANES, NV, BF16, VEC>(a.logits, (int64_t)t * a.ld, masked ? 0 : E, j, x);
        float top = x[0];
#pragma unroll
        for (int v = 1; v < NV; ++v)
            top = fmaxf(top, x[v]);
        top = group_max<LANES>(top);
        const float pf = scores<LANES, NV, SIGMOID>(x, top, r);
        // d loss / d r, from the balance loss
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            dot += r[v] * d[v];
        if (SIGMOID) {
            dot = group_sum<LANES>(dot) * pf;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                o[v] = (d[v] - dot) * pf;
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                o[v] = d[v];
        }
        if (a.grad_weights) {
            // lane k holds choice k
            int id = -1;
            float g = 0.0f;
            if (j < K) {
                const int64_t i = a.topk_idx[(int64_t)t * K + j];
                id = i >= 0 && i < E ? (int)i : -1;
                g = id >= 0 ? a.grad_weights[(int64_t)t * K + j] * a.scale : 0.0f;
            }
            float total = 0.0f, gw = 0.0f;
            if (a.normalize) {
                // scores of the chosen experts, by the lanes that hold them
                for (int k = 0; k < K; ++k) {
                    const int ik = __shfl(id, k, LANES);
                    const float gk = __shfl(g, k, LANES);
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (expert_of<LANES>(v, j) == ik) {
                            total += r[v];
                            gw += gk * r[v];
                        }
                }
                total = group_sum<LANES>(total);
                gw = group_sum<LANES>(gw);
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                g = id >= 0 ? (g - gw * inv) * inv : 0.0f;
            }
            for (int k = 0; k < K; ++k) {
                const int ik = __shfl(id, k, LANES);
                const float gk = __shfl(g, k, LANES);
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (expert_of<LANES>(v, j) == ik)
                        o[v] += gk;
            }
        }
        if (SIGMOID) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                o[v] = r[v] * (1.0f - r[v]) * o[v];
        } else {
            dot = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                dot += r[v] * o[v];
            dot = group_sum<LANES>(dot);
#pragma unroll
            for (int v = 0; v < NV; ++v)
                o[v] = r[v] * (o[v] - dot);
        }
#pragma unroll
        for (int v = 0; v < NV; v += 4) {
            const int e = expert_of<LANES>(v, j);
            const int64_t at = (int64_t)t * E + e;
            if (VEC) {
                if (e < E) {
                    if (BF16) {
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.grad_logits) + at) =
                            uint2{pack_bf16x2(o[v], o[v + 1]), pack_bf16x2(o[v + 2], o[v + 3])};
                    } else {
                        store16_hint<false>(static_cast<float*>(a.grad_logits) + at,
                                            u32x4{__float_as_uint(o[v]), __float_as_uint(o[v + 1]),
                                                  __float_as_uint(o[v + 2]), __float_as_uint(o[v + 3])});
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (e + c < E) {
                        if (BF16)
                            static_cast<uint16_t*>(a.grad_logits)[at + c] = (uint16_t)f32_to_bf16_rne(o[v + c]);
                        else
                            static_cast<float*>(a.grad_logits)[at + c] = o[v + c];
                    }
            }
        }
    }
}

template <int LANES, int NV, bool BF16, bool VEC>
static void gate_backward_run(const GateBackwardLaunch& L, hipStream_t stream)
{
    const int64_t need = ((int64_t)L.T + kGateThreads / LANES - 1) / (kGateThreads / LANES);
    const int blocks = (int)(need > 2048 ? 2048 : need);
    debug_launch("gate_backward", dim3(blocks), dim3(kGateThreads), 0);
    if (L.sigmoid)
        gate_backward_kernel<LANES, NV, BF16, VEC, true><<<blocks, kGateThreads, 0, stream>>>(L);
    else
        gate_backward_kernel<LANES, NV, BF16, VEC, false><<<blocks, kGateThreads, 0, stream>>>(L);
}

template <bool BF16, bool VEC>
static void gate_backward_pick(const GateBackwardLaunch& L, hipStream_t stream)
{
    if (L.E <= 64)
        gate_backward_run<16, 4, BF16, VEC>(L, stream);
    else if (L.E <= 128)
        gate_backward_run<16, 8, BF16, VEC>(L, stream);
    else if (L.E <= 256)
        gate_backward_run<16, 16, BF16, VEC>(L, stream);
    else if (L.E <= 512)
        gate_backward_run<32, 16, BF16, VEC>(L, stream);
    else
        gate_backward_run<64, 16, BF16, VEC>(L, stream);
}

hipError_t launch_gate_backward(const GateBackwardLaunch& L, hipStream_t stream)
{
    if (L.T == 0)
        return hipSuccess;
    const bool vec = whole_fours(L.logits, L.bf16, L.ld, L.E) &&
                     reinterpret_cast<uintptr_t>(L.grad_logits) % (L.bf16 ? 8 : 16) == 0;
    if (L.bf16)
        vec ? gate_backward_pick<true, true>(L, stream) : gate_backward_pick<true, false>(L, stream);
    else
        vec ? gate_backward_pick<false, true>(L, stream) : gate_backward_pick<false, false>(L, stream);
    return hipGetLastError();
}

}  // namespace moe_ep
