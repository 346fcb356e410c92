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
// A token is held by LANES lanes of a wave, NV values a lane, so the K rounds of
// "largest value, then smallest id that has it" run for 64 / LANES tokens at once;
// reductions over 16 lanes are four DPP steps.  Every lane keeps the same experts
// from token to token: the sums of p stay in its registers until the workgroup is
// done.  The workgroups' sums are then added in their order by a second launch, so
// the loss does not depend on timing (a few tokens take one workgroup and one launch).
//
// 16384 x 256 bf16 logits, top-8 (MI355X): 15.0 us and 7.0 for the second launch,
// the backward pass 12.7.  The 19 MB they move take 4 us at the rate of a large
// copy; the rounds' instructions bound the first, the wait for the 256 workgroups'
// sums (512 KB by one CU) the second, the scores' exponentials and divisions the
// backward pass.
#include "expert_launch.h"

namespace moe_ep {

constexpr int kGateThreads = 1024;      // forward, at most
constexpr int kGateMaxBlocks = 256;
constexpr int kBackThreads = 256;
constexpr float kNegInf = -__builtin_inff();

// Reductions over the LANES (16, 32 or 64) lanes that hold a token, for all of them.
template <int CTRL>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}

template <int LANES, typename F>
__device__ __forceinline__ int group_reduce(int v, const F& f)
{
    v = f(v, dpp<0xB1>(v));              // lane ^ 1
    v = f(v, dpp<0x4E>(v));              // lane ^ 2
    v = f(v, dpp<0x141>(v));             // the other four of eight (row_half_mirror)
    v = f(v, dpp<0x140>(v));             // the other eight of sixteen (row_mirror)
    if (LANES > 16)
        v = f(v, __shfl_xor(v, 16));
    if (LANES > 32)
        v = f(v, __shfl_xor(v, 32));
    return v;
}

template <int LANES>
__device__ __forceinline__ float group_max(float v)
{
    return __int_as_float(group_reduce<LANES>(__float_as_int(v), [](int a, int b) {
        return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
    }));
}

template <int LANES>
__device__ __forceinline__ int group_min(int v)
{
    return group_reduce<LANES>(v, [](int a, int b) { return min(a, b); });
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v)
{
    return __int_as_float(group_reduce<LANES>(__float_as_int(v), [](int a, int b) {
        return __float_as_int(__int_as_float(a) + __int_as_float(b));
    }));
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

// What a token's scores are taken relative to, so that the largest is at least 1/2:
// softmax e^top, sigmoid e^min(top, 0).  A sigmoid is 0 in fp32 below -103, but the
// ratios of such scores, which is what weights and probabilities are, are not.
template <bool SIGMOID>
__device__ __forceinline__ float base_of(float top)
{
    return SIGMOID ? fminf(top, 0.0f) : top;
}

// A score over e^base, and for sigmoid 1 - s = s(-x) from the same exponential (a
// subtraction leaves 1% of it wrong at x = 12 and nothing at 17).
template <bool SIGMOID>
__device__ __forceinline__ float score(float x, float base, float& rest)
{
    if (!SIGMOID)
        return expf(x - base);
    const float e = expf(-fabsf(x));
    rest = (x > 0.0f ? e : 1.0f) / (1.0f + e);
    return (x > 0.0f ? 1.0f : base == 0.0f ? e : expf(x - base)) / (1.0f + e);
}

// Scores r of the token's experts over e^base (softmax: times `norm`), for sigmoid their
// rest 1 - s, and norm, 1 / the sum of r.  A token without any expert left (every logit
// -inf) has r = rest = norm = 0.
template <int LANES, int NV, bool SIGMOID>
__device__ __forceinline__ float scores(const float (&x)[NV], float top, float (&r)[NV], float (&rest)[NV])
{
    const float base = base_of<SIGMOID>(top);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        rest[v] = 0.0f;
        r[v] = top == kNegInf ? 0.0f : score<SIGMOID>(x[v], base, rest[v]);
        sum += r[v];
    }
    sum = group_sum<LANES>(sum);
    const float norm = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (!SIGMOID) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            r[v] *= norm;
    }
    return norm;
}

__host__ __device__ __forceinline__ int four(int E) { return (E + 3) / 4 * 4; }

// Balance loss from the sums of p (lds_p) and counts (lds_n) of all tokens; every
// thread of the workgroup calls it.
__device__ __forceinline__ void gate_loss(const GateLaunch& a, const float* lds_p, const int* lds_n, int stripes, int ld,
                                          int valid)
{
    __shared__ float wave_sum[16];
    const int E = a.E, n = blockDim.x;
    const float V = (float)valid;
    float sum = 0.0f;
    for (int e = threadIdx.x; e < E; e += n) {
        float p = 0.0f;
        int c = 0;
        for (int s = 0; s < stripes; ++s) {
            p += lds_p[s * ld + e];
            c += lds_n[s * ld + e];
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

// Stripes of workgroups that the second launch adds side by side: a thread takes
// four neighbouring experts of a stripe's workgroups.
__host__ __device__ __forceinline__ int finish_stripes(int E)
{
    const int s = kGateThreads / (four(E) / 4);
    return s > 64 ? 64 : s;
}

__global__ __launch_bounds__(kGateThreads) void gate_finish_kernel(GateLaunch a, int blocks)
{
    extern __shared__ __align__(16) float lds[];
    __shared__ int valid;
    const int ld = four(a.E), cols = ld / 4, stripes = finish_stripes(a.E);
    int* lds_n = reinterpret_cast<int*>(lds + (size_t)stripes * ld);
    if (threadIdx.x < stripes * cols) {
        const int c = threadIdx.x % cols, s = threadIdx.x / cols;
        float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        int n[4] = {0, 0, 0, 0};
#pragma unroll 8
        for (int b = s; b < blocks; b += stripes) {
            const u32x4 dp = load16_hint<false>(a.part_p + (size_t)b * ld + 4 * c);
            const u32x4 dn = load16_hint<false>(a.part_n + (size_t)b * ld + 4 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] += __uint_as_float(dp[i]);
                n[i] += (int)dn[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lds[s * ld + 4 * c + i] = p[i];
            lds_n[s * ld + 4 * c + i] = n[i];
        }
    }
    if (threadIdx.x < kWave) {
        int c = 0;
        for (int b = threadIdx.x; b < blocks; b += kWave)
            c += a.part_v[b];
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1)
            c += __shfl_xor(c, d);
        if (threadIdx.x == 0)
            valid = c;
    }
    __syncthreads();
    gate_loss(a, lds, lds_n, stripes, ld, valid);
}

template <int LANES, int NV, bool BF16, bool VEC, bool SIGMOID>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateLaunch a)
{
    constexpr int kE = LANES * NV;
    extern __shared__ __align__(16) float sum_p[];     // [waves][kE]
    __shared__ int cnt[kE];
    __shared__ int cnt_valid;
    const int threads = blockDim.x, waves = threads / kWave, groups = threads / LANES;
    const int tid = threadIdx.x, j = tid % LANES, grp = tid / LANES;
    const int E = a.E, K = a.K;
    for (int i = tid; i < kE; i += threads)
        cnt[i] = 0;
    if (tid == 0)
        cnt_valid = 0;
    __syncthreads();
    float psum[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v)
        psum[v] = 0.0f;
    for (int64_t t = (int64_t)blockIdx.x * groups + grp; t < a.T; t += (int64_t)gridDim.x * groups) {
        const bool masked = a.token_mask && a.token_mask[t] == 0;
        float x[NV], r[NV], rest[NV];
        // a masked token's logits are not looked at: they may hold anything
        load_logits<LANES, NV, BF16, VEC>(a.logits, t * a.ld, masked ? 0 : E, j, x);
        float top = x[0];
#pragma unroll
        for (int v = 1; v < NV; ++v)
            top = fmaxf(top, x[v]);
        top = group_max<LANES>(top);
        const float base = base_of<SIGMOID>(top);
        const float norm = scores<LANES, NV, SIGMOID>(x, top, r, rest);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            psum[v] += SIGMOID ? r[v] * norm : r[v];
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
#pragma unroll
            for (int v = NV - 1; v >= 0; --v)
                if (x[v] == m)
                    id = expert_of<LANES>(v, j);
            const int best = group_min<LANES>(id);
            if (m == kNegInf || best >= E)      // no expert is left (or NaN)
                break;
            // the same operations as in scores(): the same value
            float unused;
            const float rv = SIGMOID ? score<true>(m, base, unused) : score<false>(m, base, unused) * norm;
            total += rv;
            if (j == k) {
                my_id = best;
                my_r = rv;
            }
            if (best == id)
                atomicAdd(&cnt[best], 1);
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (expert_of<LANES>(v, j) == best)
                    x[v] = kNegInf;
        }
        if (j < K) {
            float w = SIGMOID ? my_r * expf(base) : my_r;
            if (a.normalize)
                w = total == 0.0f ? 0.0f : my_r / total;
            a.topk_idx[t * K + j] = my_id;
            a.topk_weights[t * K + j] = w * a.scale;
        }
    }
    // over the wave's groups, then over the waves
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float p = psum[v];
        if (LANES <= 16)
            p += __shfl_xor(p, 16);
        if (LANES <= 32)
            p += __shfl_xor(p, 32);
        if (tid % kWave < LANES)
            sum_p[tid / kWave * kE + expert_of<LANES>(v, j)] = p;
    }
    __syncthreads();
    const int ld = four(E);
    if (gridDim.x == 1) {
        for (int e = tid; e < E; e += threads) {
            float p = 0.0f;
            for (int w = 0; w < waves; ++w)
                p += sum_p[w * kE + e];
            sum_p[e] = p;               // (row 0: only this thread reads it before)
        }
        __syncthreads();
        gate_loss(a, sum_p, cnt, 1, kE, cnt_valid);
        return;
    }
    for (int e = tid; e < ld; e += threads) {
        float p = 0.0f;
        for (int w = 0; w < waves; ++w)
            p += sum_p[w * kE + e];
        a.part_p[(size_t)blockIdx.x * ld + e] = p;
        a.part_n[(size_t)blockIdx.x * ld + e] = cnt[e];
    }
    if (tid == 0)
        a.part_v[blockIdx.x] = cnt_valid;
}

// Launch shape.  A token's rounds are a chain of about 800 instructions, so tokens
// are spread over the SIMDs before any SIMD gets a second wave to fill its waits:
// 128 tokens, 256 experts, top-8 of sigmoid scores take 10.3 + 3.6 us in 32 workgroups
// of one wave and the second launch, 28.5 in one workgroup of 16 waves; 16384 tokens
// (softmax) 15.0 + 7.0 in 256 of 16 waves and 34.2 + 8.9 in 256 of four.  16 tokens (of
// 16 lanes) go in one workgroup without a second launch.
struct GateShape {
    int threads, blocks;
};

static GateShape gate_shape(int T, int E)
{
    const int lanes = E <= 256 ? 16 : E <= 512 ? 32 : 64;
    const int64_t waves = ((int64_t)T * lanes + kWave - 1) / kWave;
    if (waves <= 4)
        return GateShape{256, 1};
    const int threads = waves <= kGateMaxBlocks ? 64 : waves <= 4 * kGateMaxBlocks ? 256 : kGateThreads;
    const int64_t need = (waves * kWave + threads - 1) / threads;
    return GateShape{threads, (int)(need > kGateMaxBlocks ? kGateMaxBlocks : need)};
}

size_t gate_workspace(int T, int E)
{
    return (size_t)gate_shape(T, E).blocks * (2 * four(E) + 1) * 4;
}

template <int LANES, int NV, bool BF16, bool VEC>
static void gate_run(const GateLaunch& L, const GateShape& g, hipStream_t stream)
{
    const size_t lds = (size_t)(g.threads / kWave) * LANES * NV * 4;
    debug_launch("gate", dim3(g.blocks), dim3(g.threads), lds);
    if (L.sigmoid)
        gate_kernel<LANES, NV, BF16, VEC, true><<<g.blocks, g.threads, lds, stream>>>(L);
    else
        gate_kernel<LANES, NV, BF16, VEC, false><<<g.blocks, g.threads, lds, stream>>>(L);
}

template <bool BF16, bool VEC>
static void gate_pick(const GateLaunch& L, const GateShape& g, hipStream_t stream)
{
    if (L.E <= 64)
        gate_run<16, 4, BF16, VEC>(L, g, stream);
    else if (L.E <= 128)
        gate_run<16, 8, BF16, VEC>(L, g, stream);
    else if (L.E <= 256)
        gate_run<16, 16, BF16, VEC>(L, g, stream);
    else if (L.E <= 512)
        gate_run<32, 16, BF16, VEC>(L, g, stream);
    else
        gate_run<64, 16, BF16, VEC>(L, g, stream);
}

static bool whole_fours(const void* p, bool bf16, int64_t ld, int E)
{
    return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (bf16 ? 8 : 16) == 0;
}

hipError_t launch_gate(GateLaunch L, void* ws, hipStream_t stream)
{
    const GateShape g = gate_shape(L.T, L.E);
    L.part_p = static_cast<float*>(ws);
    L.part_n = reinterpret_cast<int32_t*>(L.part_p + (size_t)g.blocks * four(L.E));
    L.part_v = L.part_n + (size_t)g.blocks * four(L.E);
    const bool vec = whole_fours(L.logits, L.bf16, L.ld, L.E);
    if (L.bf16)
        vec ? gate_pick<true, true>(L, g, stream) : gate_pick<true, false>(L, g, stream);
    else
        vec ? gate_pick<false, true>(L, g, stream) : gate_pick<false, false>(L, g, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (g.blocks == 1)
        return e;
    const size_t lds = (size_t)finish_stripes(L.E) * four(L.E) * 8;
    debug_launch("gate_finish", dim3(1), dim3(kGateThreads), lds);
    gate_finish_kernel<<<1, kGateThreads, lds, stream>>>(L, g.blocks);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// backward: the scores again from the logits, then
//   d_e = coef * grad_loss * E * n_e / (K V^2)     (d loss / d p_te, all tokens)
//   softmax  dl = p (d - <p, d>) + ...             sigmoid  ds = (d - <p, d>) / sum r + ...
// and for the chosen experts, with g = scale * grad_weights and wn = r / sum of
// the chosen r:  normalised  (g_k - <g, wn>) / sum of the chosen r  is added to
// d/dr_k, otherwise g_k.  dl = r (dr - <r, dr>) for softmax, r (1 - r) dr for sigmoid,
// where r dr is the same with r and its sums over e^base.
// ---------------------------------------------------------------------------
template <int LANES, int NV, bool BF16, bool VEC, bool SIGMOID>
__global__ __launch_bounds__(kBackThreads) void gate_backward_kernel(GateBackwardLaunch a)
{
    constexpr int kGroups = kBackThreads / LANES;
    constexpr int kE = LANES * NV;
    // a token's scores, for the lanes that hold a choice; gradients of the chosen ones
    __shared__ __align__(16) float lds_r[kGroups][kE], lds_g[kGroups][kE];
    const int tid = threadIdx.x, j = tid % LANES, grp = tid / LANES;
    const int E = a.E, K = a.K;
    for (int i = j; i < kE; i += LANES)
        lds_g[grp][i] = 0.0f;
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
    for (int64_t t = (int64_t)blockIdx.x * kGroups + grp; t < a.T; t += (int64_t)gridDim.x * kGroups) {
        const bool masked = a.token_mask && a.token_mask[t] == 0;
        float x[NV], r[NV], rest[NV], o[NV];
        load_logits<LANES, NV, BF16, VEC>(a.logits, t * a.ld, masked ? 0 : E, j, x);
        float top = x[0];
#pragma unroll
        for (int v = 1; v < NV; ++v)
            top = fmaxf(top, x[v]);
        top = group_max<LANES>(top);
        const float norm = scores<LANES, NV, SIGMOID>(x, top, r, rest);
        // d loss / d r, from the balance loss
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            dot += r[v] * d[v];
        if (SIGMOID) {
            dot = group_sum<LANES>(dot) * norm;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                o[v] = (d[v] - dot) * norm;
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
                const int64_t i = a.topk_idx[t * K + j];
                id = i >= 0 && i < E ? (int)i : -1;
                g = id >= 0 ? a.grad_weights[t * K + j] * a.scale : 0.0f;
            }
            if (a.normalize) {
#pragma unroll
                for (int v = 0; v < NV; v += 4)
                    *reinterpret_cast<float4*>(&lds_r[grp][expert_of<LANES>(v, j)]) = float4{r[v], r[v + 1], r[v + 2], r[v + 3]};
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const float rk = id >= 0 ? lds_r[grp][id] : 0.0f;
                const float total = group_sum<LANES>(rk), gw = group_sum<LANES>(g * rk);
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                g = (g - gw * inv) * inv;
            } else if (SIGMOID) {
                g *= expf(base_of<SIGMOID>(top));      // r is over e^base
            }
            // to the lanes that hold the chosen experts, and back to zeros for the next token
            if (id >= 0)
                atomicAdd(&lds_g[grp][id], g);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int v = 0; v < NV; v += 4) {
                const float4 q = *reinterpret_cast<const float4*>(&lds_g[grp][expert_of<LANES>(v, j)]);
                o[v] += q.x;
                o[v + 1] += q.y;
                o[v + 2] += q.z;
                o[v + 3] += q.w;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (id >= 0)
                lds_g[grp][id] = 0.0f;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        if (SIGMOID) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                o[v] = r[v] * rest[v] * o[v];
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
            const int64_t at = t * E + e;
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
    const int64_t need = ((int64_t)L.T + kBackThreads / LANES - 1) / (kBackThreads / LANES);
    const int blocks = (int)(need > 2048 ? 2048 : need);
    debug_launch("gate_backward", dim3(blocks), dim3(kBackThreads), 0);
    if (L.sigmoid)
        gate_backward_kernel<LANES, NV, BF16, VEC, true><<<blocks, kBackThreads, 0, stream>>>(L);
    else
        gate_backward_kernel<LANES, NV, BF16, VEC, false><<<blocks, kBackThreads, 0, stream>>>(L);
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
