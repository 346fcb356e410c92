// C entry points of the expert layer: argument checks and launches (nothing is
// allocated and nothing waits).
#include "api_check.h"
#include "expert_launch.h"

using moe_ep::aligned;
using moe_ep::fail;
using moe_ep::g_err;
using moe_ep::hip_fail;

namespace {

// 1 x 128 blocks a row launch covers: 32 a workgroup of 256, and fewer than 2^32 threads.
constexpr int64_t kMaxUnits = ((int64_t)1 << 29) - 32;

bool width_ok(int w) { return w >= 128 && w <= EP_MAX_HIDDEN && w % 128 == 0; }

int check_width(const char* name, int w)
{
    if (width_ok(w))
        return EP_OK;
    return fail(EP_EINVAL, "%s=%d must be a multiple of 128 in [128, %d]", name, w, EP_MAX_HIDDEN);
}

int check_groups(const int32_t* off, int G, int stride, int rows, bool optional = false)
{
    if (rows < 0 || rows > 0x7FFFFF00)
        return fail(EP_EINVAL, "num_rows=%d must be in [0, 2^31 - 256]", rows);
    if (optional && !off) {
        if (G != 0 || stride != 0)
            return fail(EP_EINVAL, "num_groups and group_stride must be 0 without group_offsets");
        return EP_OK;
    }
    if (G < 1 || G > EP_MAX_EXPERTS)
        return fail(EP_EINVAL, "num_groups=%d must be in [1, %d]", G, EP_MAX_EXPERTS);
    if (stride < 0)
        return fail(EP_EINVAL, "group_stride=%d must be >= 0", stride);
    if (!off || !aligned(off, 4))
        return fail(EP_EINVAL, "group_offsets must be a non-NULL 4-byte aligned device pointer");
    return EP_OK;
}

int check_ptr(const char* name, const void* p, size_t a)
{
    if (p && aligned(p, a))
        return EP_OK;
    return fail(EP_EINVAL, "%s must be a non-NULL %zu-byte aligned device pointer", name, a);
}

int check_scale_ld(int ld, int rows)
{
    if (ld == 0 || (ld >= rows && ld % 4 == 0))
        return EP_OK;
    return fail(EP_EINVAL, "scale_ld=%d must be 0, or >= num_rows=%d and a multiple of 4", ld, rows);
}

int check_units(int rows, int width)
{
    if ((int64_t)rows * (width / 128) <= kMaxUnits)
        return EP_OK;
    return fail(EP_EINVAL, "num_rows=%d x width=%d is more than one call covers (2^29 - 32 blocks of 128)", rows, width);
}

struct GateDims {
    int64_t ld;
    int T, E, K, score;
};

int check_gate(const void* logits, int bf16, const GateDims& d, int normalize)
{
    if (d.T < 0 || d.E < 1 || d.E > EP_MAX_EXPERTS || d.K < 1 || d.K > EP_MAX_TOPK || d.K > d.E ||
        (int64_t)d.T * d.K >= (int64_t)1 << 31)
        return fail(EP_EINVAL, "invalid dims T=%d E=%d K=%d (need T>=0, 1<=E<=%d, 1<=K<=min(E, %d), T*K<2^31)",
                    d.T, d.E, d.K, EP_MAX_EXPERTS, EP_MAX_TOPK);
    if (bf16 != 0 && bf16 != 1)
        return fail(EP_EINVAL, "logits_bf16 must be 0 or 1");
    if (normalize != 0 && normalize != 1)
        return fail(EP_EINVAL, "normalize must be 0 or 1");
    if (d.score != EP_GATE_SOFTMAX && d.score != EP_GATE_SIGMOID)
        return fail(EP_EINVAL, "score=%d must be EP_GATE_SOFTMAX or EP_GATE_SIGMOID", d.score);
    if (d.ld < d.E || d.ld > (int64_t)1 << 40)
        return fail(EP_EINVAL, "ld=%lld must be >= E=%d", (long long)d.ld, d.E);
    if (d.T > 0)
        return check_ptr("logits", logits, bf16 ? 2 : 4);
    return EP_OK;
}

}  // namespace

#define EP_TRY(call)          \
    do {                      \
        const int rc_ = call; \
        if (rc_)              \
            return rc_;       \
    } while (0)

extern "C" {

size_t ep_gate_workspace_bytes(int T, int E)
{
    if (T < 0 || E < 1 || E > EP_MAX_EXPERTS)
        return 0;
    return moe_ep::gate_workspace(T, E);
}

int ep_gate(const void* logits, int logits_bf16, int64_t ld, int T, int E, int K, int score,
            int normalize, float scale, float balance_coef, const uint8_t* token_mask,
            int64_t* topk_idx, float* topk_weights, int32_t* num_tokens_per_expert,
            int32_t* num_valid, float* loss, void* ws, size_t ws_bytes, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_gate(logits, logits_bf16, GateDims{ld, T, E, K, score}, normalize));
    if (T > 0) {
        EP_TRY(check_ptr("topk_idx", topk_idx, 8));
        EP_TRY(check_ptr("topk_weights", topk_weights, 4));
    }
    EP_TRY(check_ptr("num_tokens_per_expert", num_tokens_per_expert, 4));
    EP_TRY(check_ptr("num_valid", num_valid, 4));
    EP_TRY(check_ptr("loss", loss, 4));
    EP_TRY(check_ptr("workspace", ws, 256));
    if (ws_bytes < ep_gate_workspace_bytes(T, E))
        return fail(EP_EINVAL, "workspace too small: %zu bytes given, %zu needed", ws_bytes,
                    ep_gate_workspace_bytes(T, E));
    moe_ep::GateLaunch L;
    L.logits = logits;
    L.bf16 = logits_bf16;
    L.ld = ld;
    L.T = T;
    L.E = E;
    L.K = K;
    L.sigmoid = score == EP_GATE_SIGMOID;
    L.normalize = normalize;
    L.scale = scale;
    L.coef = balance_coef;
    L.token_mask = token_mask;
    L.topk_idx = topk_idx;
    L.topk_weights = topk_weights;
    L.counts = num_tokens_per_expert;
    L.num_valid = num_valid;
    L.loss = loss;
    L.part_p = nullptr;
    L.part_n = L.part_v = nullptr;
    const hipError_t e = moe_ep::launch_gate(L, ws, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "gate launch");
}

int ep_gate_backward(const void* logits, int logits_bf16, int64_t ld, int T, int E, int K, int score,
                     int normalize, float scale, float balance_coef, const uint8_t* token_mask,
                     const int64_t* topk_idx, const int32_t* num_tokens_per_expert,
                     const int32_t* num_valid, const float* grad_weights, const float* grad_loss,
                     void* grad_logits, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_gate(logits, logits_bf16, GateDims{ld, T, E, K, score}, normalize));
    EP_TRY(check_ptr("num_tokens_per_expert", num_tokens_per_expert, 4));
    EP_TRY(check_ptr("num_valid", num_valid, 4));
    if (grad_weights && !aligned(grad_weights, 4))
        return fail(EP_EINVAL, "grad_weights must be 4-byte aligned");
    if (grad_loss && !aligned(grad_loss, 4))
        return fail(EP_EINVAL, "grad_loss must be 4-byte aligned");
    if (T > 0) {
        EP_TRY(check_ptr("topk_idx", topk_idx, 8));
        EP_TRY(check_ptr("grad_logits", grad_logits, logits_bf16 ? 2 : 4));
    }
    moe_ep::GateBackwardLaunch L;
    L.logits = logits;
    L.bf16 = logits_bf16;
    L.ld = ld;
    L.T = T;
    L.E = E;
    L.K = K;
    L.sigmoid = score == EP_GATE_SIGMOID;
    L.normalize = normalize;
    L.scale = scale;
    L.coef = balance_coef;
    L.token_mask = token_mask;
    L.topk_idx = topk_idx;
    L.counts = num_tokens_per_expert;
    L.num_valid = num_valid;
    L.grad_weights = grad_weights;
    L.grad_loss = grad_loss;
    L.grad_logits = grad_logits;
    const hipError_t e = moe_ep::launch_gate_backward(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "gate backward launch");
}

int ep_quantize_rows(const void* x, int width, const int32_t* group_offsets, int num_groups,
                     int group_stride, int num_rows, int scale_ld, void* codes, float* scales,
                     hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_width("width", width));
    EP_TRY(check_groups(group_offsets, num_groups, group_stride, num_rows, true));
    EP_TRY(check_scale_ld(scale_ld, num_rows));
    EP_TRY(check_units(num_rows, width));
    if (num_rows > 0) {
        EP_TRY(check_ptr("x", x, 16));
        EP_TRY(check_ptr("codes", codes, 16));
        EP_TRY(check_ptr("scales", scales, 4));
    }
    const hipError_t e = moe_ep::launch_quantize_rows(
        x, width, moe_ep::Groups{group_offsets, num_groups, group_stride, num_rows}, scale_ld, codes,
        scales, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "row quantiser launch");
}

int ep_quantize_weights(const void* w, int w_f32, int num_groups, int n, int k, void* codes,
                        float* scales, void* codes_t, float* scales_t, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_width("n", n));
    EP_TRY(check_width("k", k));
    if (num_groups < 1 || num_groups > EP_MAX_EXPERTS)
        return fail(EP_EINVAL, "num_groups=%d must be in [1, %d]", num_groups, EP_MAX_EXPERTS);
    if (w_f32 != 0 && w_f32 != 1)
        return fail(EP_EINVAL, "w_f32 must be 0 or 1");
    EP_TRY(check_ptr("w", w, 16));
    EP_TRY(check_ptr("codes", codes, 16));
    EP_TRY(check_ptr("scales", scales, 4));
    if ((codes_t != nullptr) != (scales_t != nullptr))
        return fail(EP_EINVAL, "codes_t and scales_t must be given together");
    if (codes_t) {
        EP_TRY(check_ptr("codes_t", codes_t, 16));
        EP_TRY(check_ptr("scales_t", scales_t, 4));
    }
    const hipError_t e = moe_ep::launch_quantize_weights(w, w_f32, num_groups, n, k, codes, scales,
                                                         codes_t, scales_t, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "weight quantiser launch");
}

int ep_grouped_gemm_fp8(const void* x, const float* x_scales, int scale_ld, const void* w,
                        const float* w_scales, const int32_t* group_offsets, int num_groups,
                        int group_stride, int num_rows, int n, int k, int expected_rows, void* out,
                        hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_width("n", n));
    EP_TRY(check_width("k", k));
    EP_TRY(check_groups(group_offsets, num_groups, group_stride, num_rows));
    EP_TRY(check_scale_ld(scale_ld, num_rows));
    if (expected_rows < 0)
        return fail(EP_EINVAL, "expected_rows=%d must be >= 0", expected_rows);
    EP_TRY(check_ptr("w", w, 16));
    EP_TRY(check_ptr("w_scales", w_scales, 4));
    if (num_rows > 0) {
        EP_TRY(check_ptr("x", x, 16));
        EP_TRY(check_ptr("x_scales", x_scales, 4));
        EP_TRY(check_ptr("out", out, 16));
    }
    moe_ep::GemmLaunch L;
    L.x = static_cast<const uint8_t*>(x);
    L.x_scales = x_scales;
    L.x_scale_ld = scale_ld;
    L.w = static_cast<const uint8_t*>(w);
    L.w_scales = w_scales;
    L.groups = moe_ep::Groups{group_offsets, num_groups, group_stride, num_rows};
    L.N = n;
    L.K = k;
    L.expected_rows = expected_rows ? expected_rows : num_rows / num_groups;
    L.out = static_cast<uint16_t*>(out);
    const hipError_t e = moe_ep::launch_grouped_gemm(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "grouped product launch");
}

int ep_grouped_wgrad_fp8(const void* grad, const void* x, const float* x_scales, int scale_ld,
                         const int32_t* group_offsets, int num_groups, int group_stride,
                         int num_rows, int n, int k, void* out, int out_f32, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_width("n", n));
    EP_TRY(check_width("k", k));
    EP_TRY(check_groups(group_offsets, num_groups, group_stride, num_rows));
    EP_TRY(check_scale_ld(scale_ld, num_rows));
    if (out_f32 != 0 && out_f32 != 1)
        return fail(EP_EINVAL, "out_f32 must be 0 or 1");
    EP_TRY(check_ptr("out", out, 16));
    if (num_rows > 0) {
        EP_TRY(check_ptr("grad", grad, 16));
        EP_TRY(check_ptr("x", x, 16));
        EP_TRY(check_ptr("x_scales", x_scales, 4));
    }
    moe_ep::WgradLaunch L;
    L.dy = static_cast<const uint16_t*>(grad);
    L.x = static_cast<const uint8_t*>(x);
    L.x_scales = x_scales;
    L.x_scale_ld = scale_ld;
    L.groups = moe_ep::Groups{group_offsets, num_groups, group_stride, num_rows};
    L.N = n;
    L.K = k;
    L.dw = out;
    L.dw_f32 = out_f32;
    const hipError_t e = moe_ep::launch_grouped_wgrad(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "grouped weight gradient launch");
}

int ep_swiglu_fp8(const void* h, int inner, const int32_t* group_offsets, int num_groups,
                  int group_stride, int num_rows, int scale_ld, void* codes, float* scales,
                  void* ckpt, float* ckpt_scales, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_width("inner", inner));
    EP_TRY(check_groups(group_offsets, num_groups, group_stride, num_rows, true));
    EP_TRY(check_scale_ld(scale_ld, num_rows));
    EP_TRY(check_units(num_rows, inner));
    if ((ckpt != nullptr) != (ckpt_scales != nullptr))
        return fail(EP_EINVAL, "ckpt and ckpt_scales must be given together");
    if (num_rows > 0) {
        EP_TRY(check_ptr("h", h, 16));
        EP_TRY(check_ptr("codes", codes, 16));
        EP_TRY(check_ptr("scales", scales, 4));
        if (ckpt) {
            EP_TRY(check_ptr("ckpt", ckpt, 16));
            EP_TRY(check_ptr("ckpt_scales", ckpt_scales, 4));
        }
    }
    moe_ep::SwigluLaunch L;
    L.h = static_cast<const uint16_t*>(h);
    L.inner = inner;
    L.groups = moe_ep::Groups{group_offsets, num_groups, group_stride, num_rows};
    L.codes = static_cast<uint8_t*>(codes);
    L.scales = scales;
    L.scale_ld = scale_ld;
    L.ckpt = static_cast<uint8_t*>(ckpt);
    L.ckpt_scales = ckpt_scales;
    const hipError_t e = moe_ep::launch_swiglu(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "SwiGLU launch");
}

int ep_swiglu_fp8_backward(const void* grad_a, const void* ckpt, const float* ckpt_scales, int inner,
                           const int32_t* group_offsets, int num_groups, int group_stride,
                           int num_rows, int scale_ld, void* grad_h, void* codes, float* scales,
                           hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_width("inner", inner));
    EP_TRY(check_groups(group_offsets, num_groups, group_stride, num_rows, true));
    EP_TRY(check_scale_ld(scale_ld, num_rows));
    EP_TRY(check_units(num_rows, inner));
    if ((codes != nullptr) != (scales != nullptr))
        return fail(EP_EINVAL, "codes and scales must be given together");
    if (num_rows > 0) {
        EP_TRY(check_ptr("grad_a", grad_a, 16));
        EP_TRY(check_ptr("ckpt", ckpt, 16));
        EP_TRY(check_ptr("ckpt_scales", ckpt_scales, 4));
        if (!grad_h && !codes)
            return fail(EP_EINVAL, "neither grad_h nor codes is given: nothing to write");
        if (grad_h)
            EP_TRY(check_ptr("grad_h", grad_h, 16));
        if (codes) {
            EP_TRY(check_ptr("codes", codes, 16));
            EP_TRY(check_ptr("scales", scales, 4));
        }
    }
    moe_ep::SwigluBackwardLaunch L;
    L.da = static_cast<const uint16_t*>(grad_a);
    L.ckpt = static_cast<const uint8_t*>(ckpt);
    L.ckpt_scales = ckpt_scales;
    L.inner = inner;
    L.groups = moe_ep::Groups{group_offsets, num_groups, group_stride, num_rows};
    L.dh = static_cast<uint16_t*>(grad_h);
    L.codes = static_cast<uint8_t*>(codes);
    L.scales = scales;
    L.scale_ld = scale_ld;
    const hipError_t e = moe_ep::launch_swiglu_backward(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "SwiGLU backward launch");
}

}  // extern "C"
