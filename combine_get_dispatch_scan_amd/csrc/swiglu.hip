// SwiGLU between the experts' two products, on gfx950, in 8 bits on the way out
// and in the checkpoint:
//   forward   h = [g | u] (bf16):  a = g * s(g) * u,  s(g) = 1 / (1 + e^-g),
//             written as E4M3FN codes with 1 x 128 scales (what the second
//             product reads), and h itself in the same format, half of its
//             bytes, for the backward pass
//   backward  from the checkpoint's g, u and da (bf16):
//             dg = da * u * s(g) * (1 + g * (1 - s(g))),  du = da * g * s(g),
//             written as bf16 (what the weight gradient reads) and as codes
//             with scales (what the product towards the input reads)
// All arithmetic is fp32; e^-g is the hardware's base-2 exponential (its error
// grows by |g| * 2^-24, far under the 2^-4 of the codes' rounding) and the
// division its reciprocal (1 ulp).  Both passes are bound by HBM: every value is
// read and written once.  Eight lanes hold one 128-channel block of g and the
// block of u that belongs to it.  32768 rows, inner = 2048 (MI355X): forward with
// checkpoint 84 us, backward with both outputs 124 us, 5.7 and 5.5 TB/s of the bytes
// they cannot do without (a 1 GiB copy: 5.05).
#include "expert_launch.h"
#include "quant16.h"

namespace moe_ep {

__device__ __forceinline__ float sigmoid(float g)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

template <bool CKPT>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluLaunch a)
{
    const int nb = a.inner / kQBlock;
    const int lane8 = threadIdx.x & 7;
    const int64_t u = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    const int r = (int)(u / nb), b = (int)(u % nb);
    const bool act = u < (int64_t)a.groups.rows * nb && row_in_group(a.groups, r);
    u32x4 d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        d[j] = u32x4{0u, 0u, 0u, 0u};
    const size_t row = (size_t)r * 2 * a.inner;
    const int c = b * kQBlock + lane8 * 16;
    if (act) {
        const uint16_t* p = a.h + row + c;
        d[0] = load16_hint<false>(p);
        d[1] = load16_hint<false>(p + 8);
        d[2] = load16_hint<false>(p + a.inner);
        d[3] = load16_hint<false>(p + a.inner + 8);
    }
    float g[16], up[16], v[16], scale;
    widen16(d[0], d[1], g);
    widen16(d[2], d[3], up);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        v[j] = g[j] * sigmoid(g[j]) * up[j];
    const u32x4 q = encode_block(v, scale);
    if (act) {
        store16_hint<false>(a.codes + (size_t)r * a.inner + c, q);
        if (lane8 == 0)
            a.scales[scale_at(r, b, nb, a.scale_ld)] = scale;
    }
    if (CKPT) {
        float sg, su;
        const u32x4 qg = encode_block(g, sg), qu = encode_block(up, su);
        if (act) {
            store16_hint<false>(a.ckpt + row + c, qg);
            store16_hint<false>(a.ckpt + row + a.inner + c, qu);
            if (lane8 == 0) {
                a.ckpt_scales[(size_t)r * 2 * nb + b] = sg;
                a.ckpt_scales[(size_t)r * 2 * nb + nb + b] = su;
            }
        }
    }
}

hipError_t launch_swiglu(const SwigluLaunch& L, hipStream_t stream)
{
    const int64_t units = (int64_t)L.groups.rows * (L.inner / kQBlock);
    if (units == 0)
        return hipSuccess;
    const dim3 grid((unsigned)((units + 31) / 32));
    debug_launch("swiglu", grid, dim3(256), 0);
    auto* kernel = L.ckpt ? swiglu_kernel<true> : swiglu_kernel<false>;
    kernel<<<grid, 256, 0, stream>>>(L);
    return hipGetLastError();
}

__device__ __forceinline__ void store_bf16x16(uint16_t* p, const float (&v)[16])
{
    u32x4 lo, hi;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        hi[j] = pack_bf16x2(v[8 + 2 * j], v[8 + 2 * j + 1]);
    }
    store16_hint<false>(p, lo);
    store16_hint<false>(p + 8, hi);
}

__global__ __launch_bounds__(256) void swiglu_backward_kernel(SwigluBackwardLaunch a)
{
    const int nb = a.inner / kQBlock;
    const int lane8 = threadIdx.x & 7;
    const int64_t u = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    const int r = (int)(u / nb), b = (int)(u % nb);
    const bool act = u < (int64_t)a.groups.rows * nb && row_in_group(a.groups, r);
    u32x4 d0 = u32x4{0u, 0u, 0u, 0u}, d1 = d0, qg = d0, qu = d0;
    float sg = 0.0f, su = 0.0f;
    const size_t row = (size_t)r * 2 * a.inner;
    const int c = b * kQBlock + lane8 * 16;
    if (act) {
        const uint16_t* p = a.da + (size_t)r * a.inner + c;
        d0 = load16_hint<false>(p);
        d1 = load16_hint<false>(p + 8);
        qg = load16_hint<false>(a.ckpt + row + c);
        qu = load16_hint<false>(a.ckpt + row + a.inner + c);
        sg = a.ckpt_scales[(size_t)r * 2 * nb + b];
        su = a.ckpt_scales[(size_t)r * 2 * nb + nb + b];
    }
    float da[16], g[16], up[16], dg[16], du[16];
    widen16(d0, d1, da);
    decode16(qg, sg, g);
    decode16(qu, su, up);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float s = sigmoid(g[j]);
        dg[j] = da[j] * up[j] * (s * (1.0f + g[j] * (1.0f - s)));
        du[j] = da[j] * (g[j] * s);
    }
    if (a.dh && act) {
        store_bf16x16(a.dh + row + c, dg);
        store_bf16x16(a.dh + row + a.inner + c, du);
    }
    if (a.codes) {
        float tg, tu;
        const u32x4 eg = encode_block(dg, tg), eu = encode_block(du, tu);
        if (act) {
            store16_hint<false>(a.codes + row + c, eg);
            store16_hint<false>(a.codes + row + a.inner + c, eu);
            if (lane8 == 0) {
                a.scales[scale_at(r, b, 2 * nb, a.scale_ld)] = tg;
                a.scales[scale_at(r, nb + b, 2 * nb, a.scale_ld)] = tu;
            }
        }
    }
}

hipError_t launch_swiglu_backward(const SwigluBackwardLaunch& L, hipStream_t stream)
{
    const int64_t units = (int64_t)L.groups.rows * (L.inner / kQBlock);
    if (units == 0)
        return hipSuccess;
    const dim3 grid((unsigned)((units + 31) / 32));
    debug_launch("swiglu_backward", grid, dim3(256), 0);
    swiglu_backward_kernel<<<grid, 256, 0, stream>>>(L);
    return hipGetLastError();
}

}  // namespace moe_ep
