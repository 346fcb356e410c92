// C entry points of the operators around the expert layer: argument checks and
// launches (nothing is allocated and nothing waits).
#include <math.h>

#include "block_launch.h"
#include "expert_check.h"

using namespace moe_ep;

namespace {

int check_flag(const char* name, int v)
{
    if (v == 0 || v == 1)
        return EP_OK;
    return fail(EP_EINVAL, "%s must be 0 or 1", name);
}

int check_norm(const ep_block_norm_t* a)
{
    if (!a)
        return fail(EP_EINVAL, "args must not be NULL");
    if (a->num_rows < 0 || a->num_rows > 0x7FFFFF00)
        return fail(EP_EINVAL, "num_rows=%d must be in [0, 2^31 - 256]", a->num_rows);
    if (a->width < 8 || a->width > EP_MAX_HIDDEN || a->width % 8)
        return fail(EP_EINVAL, "width=%d must be a multiple of 8 in [8, %d]", a->width, EP_MAX_HIDDEN);
    EP_TRY(check_flag("x_f32", a->x_f32));
    EP_TRY(check_flag("norm", a->norm));
    EP_TRY(check_flag("y_norm", a->y_norm));
    EP_TRY(check_flag("weights_f32", a->weights_f32));
    EP_TRY(check_flag("gate_f32", a->gate_f32));
    if (a->gate_kind < EP_GATE_NONE || a->gate_kind > EP_GATE_CHANNEL)
        return fail(EP_EINVAL, "gate_kind=%d must be EP_GATE_NONE, EP_GATE_TOKEN or EP_GATE_CHANNEL", a->gate_kind);
    if (!a->y && a->num_rows > 0 && (a->y_norm || a->y_weight || a->gate_kind != EP_GATE_NONE))
        return fail(EP_EINVAL, "y_norm, y_weight and gate need y");
    if (!a->y && a->num_rows > 0 && (!a->norm || a->residual_scale != 1.0f))
        return fail(EP_EINVAL, "without y, norm must be 1 and residual_scale 1");
    if (a->weight && !a->norm)
        return fail(EP_EINVAL, "weight needs norm");
    if ((a->gate != nullptr) != (a->gate_kind != EP_GATE_NONE) &&
        !(a->num_rows == 0 && a->gate_kind == EP_GATE_TOKEN))
        return fail(EP_EINVAL, "gate and gate_kind must be given together");
    if (!(a->eps >= 0x1p-100f && a->eps <= 0x1p100f))
        return fail(EP_EINVAL, "eps must be in [2^-100, 2^100]");
    if (!isfinite(a->residual_scale) || !isfinite(a->y_scale) || !isfinite(a->weight_offset))
        return fail(EP_EINVAL, "residual_scale, y_scale and weight_offset must be finite");
    const int64_t far = (int64_t)1 << 40;
    if (a->x_ld < a->width || a->x_ld > far || a->x_ld % 8)
        return fail(EP_EINVAL, "x_ld=%lld must be >= width=%d and a multiple of 8", (long long)a->x_ld, a->width);
    if (a->y && (a->y_ld < a->width || a->y_ld > far || a->y_ld % 8))
        return fail(EP_EINVAL, "y_ld=%lld must be >= width=%d and a multiple of 8", (long long)a->y_ld, a->width);
    if (a->num_rows > 0)
        EP_TRY(check_ptr("x", a->x, 16));
    if (!aligned(a->y, 16) || !aligned(a->weight, 16) || !aligned(a->y_weight, 16))
        return fail(EP_EINVAL, "y, weight and y_weight must be 16-byte aligned");
    if (!aligned(a->gate, a->gate_kind == EP_GATE_CHANNEL ? 16 : a->gate_f32 ? 4 : 2))
        return fail(EP_EINVAL, "gate must be aligned (a channel's to 16 bytes)");
    return EP_OK;
}

}  // namespace

extern "C" {

int ep_block_norm(const ep_block_norm_t* args, void* x_out, void* h, void* codes, float* scales,
                  hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_norm(args));
    if ((codes != nullptr) != (scales != nullptr))
        return fail(EP_EINVAL, "codes and scales must be given together");
    if (x_out && !args->y)
        return fail(EP_EINVAL, "x_out needs y: without it x' is x");
    if (x_out && x_out == args->x && args->x_ld != args->width)
        return fail(EP_EINVAL, "x_out may be x only where x is dense");
    if ((h || codes) && !args->norm)
        return fail(EP_EINVAL, "h and codes need norm");
    if (codes && args->width % 128)
        return fail(EP_EINVAL, "width=%d must be a multiple of 128 for codes", args->width);
    if (args->num_rows > 0 && !x_out && !h && !codes)
        return fail(EP_EINVAL, "no output is given: nothing to write");
    if (!aligned(x_out, 16) || !aligned(h, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return fail(EP_EINVAL, "x_out, h and codes must be 16-byte aligned, scales 4-byte");
    BlockNormLaunch L;
    L.in = *args;
    L.xo = x_out;
    L.h = static_cast<uint16_t*>(h);
    L.codes = static_cast<uint8_t*>(codes);
    L.scales = scales;
    const hipError_t e = launch_block_norm(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "block norm launch");
}

size_t ep_block_norm_workspace_bytes(int num_rows, int width)
{
    if (num_rows < 0 || num_rows > 0x7FFFFF00 || width < 8 || width > EP_MAX_HIDDEN || width % 8)
        return 0;
    return block_norm_workspace(num_rows, width);
}

int ep_block_norm_backward(const ep_block_norm_t* args, const void* grad_x, const void* grad_h,
                           void* out_x, void* out_y, void* out_weight, void* out_y_weight,
                           void* out_gate, void* ws, size_t ws_bytes, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_norm(args));
    if (grad_h && !args->norm)
        return fail(EP_EINVAL, "grad_h needs norm");
    if (out_y && !args->y)
        return fail(EP_EINVAL, "out_y needs y");
    if (out_weight && !args->weight)
        return fail(EP_EINVAL, "out_weight needs weight");
    if (out_y_weight && !args->y_weight)
        return fail(EP_EINVAL, "out_y_weight needs y_weight");
    if (out_gate && args->gate_kind == EP_GATE_NONE)
        return fail(EP_EINVAL, "out_gate needs a gate");
    const bool columns = out_weight || out_y_weight || (out_gate && args->gate_kind == EP_GATE_CHANNEL);
    if (args->num_rows > 0 && !out_x && !out_y && !out_gate && !columns)
        return fail(EP_EINVAL, "no output is given: nothing to write");
    if (!aligned(grad_x, 16) || !aligned(grad_h, 16) || !aligned(out_x, 16) || !aligned(out_y, 16))
        return fail(EP_EINVAL, "grad_x, grad_h, out_x and out_y must be 16-byte aligned");
    if (!aligned(out_weight, 4) || !aligned(out_y_weight, 4) || !aligned(out_gate, 4))
        return fail(EP_EINVAL, "out_weight, out_y_weight and out_gate must be 4-byte aligned");
    if (columns) {
        EP_TRY(check_ptr("workspace", ws, 256));
        const size_t need = ep_block_norm_workspace_bytes(args->num_rows, args->width);
        if (ws_bytes < need)
            return fail(EP_EINVAL, "workspace too small: %zu bytes given, %zu needed", ws_bytes, need);
    }
    BlockNormBackwardLaunch L;
    L.in = *args;
    L.gx = grad_x;
    L.gh = static_cast<const uint16_t*>(grad_h);
    L.dx = out_x;
    L.dy = static_cast<uint16_t*>(out_y);
    L.dw = out_weight;
    L.dyw = out_y_weight;
    L.dgate = out_gate;
    L.part = columns ? static_cast<float*>(ws) : nullptr;
    const hipError_t e = launch_block_norm_backward(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "block norm backward launch");
}

static int check_fp4(int w_f32, const char* flag, int num_groups, int n, int k)
{
    EP_TRY(check_width("n", n));
    EP_TRY(check_width("k", k));
    if (num_groups < 1 || num_groups > EP_MAX_EXPERTS)
        return fail(EP_EINVAL, "num_groups=%d must be in [1, %d]", num_groups, EP_MAX_EXPERTS);
    // a launch has fewer than 2^32 threads, of 16 weights each
    if ((int64_t)num_groups * n * k > (int64_t)1 << 35)
        return fail(EP_EINVAL, "%d groups of %d x %d weights are more than 2^35 in one call", num_groups, n, k);
    return check_flag(flag, w_f32);
}

int ep_quantize_weights_fp4(const void* w, int w_f32, int num_groups, int n, int k, void* codes,
                            void* scales, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_fp4(w_f32, "w_f32", num_groups, n, k));
    EP_TRY(check_ptr("w", w, 16));
    EP_TRY(check_ptr("codes", codes, 16));
    EP_TRY(check_ptr("scales", scales, 4));
    const hipError_t e = launch_quantize_fp4(w, w_f32, (int64_t)num_groups * n * (k / 32),
                                             static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "4-bit weight quantiser launch");
}

int ep_dequantize_weights_fp4(const void* codes, const void* scales, int num_groups, int n, int k,
                              void* out, int out_f32, hipStream_t stream)
{
    g_err.clear();
    EP_TRY(check_fp4(out_f32, "out_f32", num_groups, n, k));
    EP_TRY(check_ptr("codes", codes, 16));
    EP_TRY(check_ptr("scales", scales, 4));
    EP_TRY(check_ptr("out", out, 16));
    const hipError_t e = launch_dequantize_fp4(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                                               (int64_t)num_groups * n * (k / 32), out, out_f32, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "4-bit weight dequantiser launch");
}

int ep_grouped_gemm_fp4(const void* x, const float* x_scales, int scale_ld, const void* w,
                        const void* w_scales, const int32_t* group_offsets, int num_groups,
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
    GemmFp4Launch L;
    L.x = static_cast<const uint8_t*>(x);
    L.x_scales = x_scales;
    L.x_scale_ld = scale_ld;
    L.w = static_cast<const uint8_t*>(w);
    L.w_scales = static_cast<const uint8_t*>(w_scales);
    L.groups = Groups{group_offsets, num_groups, group_stride, num_rows};
    L.N = n;
    L.K = k;
    L.expected_rows = expected_rows ? expected_rows : num_rows / num_groups;
    L.out = static_cast<uint16_t*>(out);
    const hipError_t e = launch_grouped_gemm_fp4(L, stream);
    return e == hipSuccess ? EP_OK : hip_fail(e, "grouped 4-bit product launch");
}

}  // extern "C"
