// Host-side launchers of the expert-layer kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "groups.h"

namespace moe_ep {

void debug_launch(const char* kernel, dim3 grid, dim3 block, size_t lds);

hipError_t launch_quantize_rows(const void* x, int H, const Groups& g, int scale_ld, void* codes,
                                float* scales, hipStream_t stream);
hipError_t launch_quantize_weights(const void* w, bool w_f32, int G, int N, int K, void* codes,
                                   float* scales, void* codes_t, float* scales_t, hipStream_t stream);

struct GemmLaunch {
    const uint8_t* x;         // [rows][K]
    const float* x_scales;    // ld 0: [rows][K/128], else [K/128][ld]
    int x_scale_ld;
    const uint8_t* w;         // [G][N][K]
    const float* w_scales;    // [G][N/128][K/128]
    Groups groups;
    int N, K;
    int expected_rows;        // typical rows of a group (chooses the tile)
    uint16_t* out;            // [rows][N]
};
hipError_t launch_grouped_gemm(const GemmLaunch& L, hipStream_t stream);

struct WgradLaunch {
    const uint16_t* dy;       // [rows][N]
    const uint8_t* x;         // [rows][K]
    const float* x_scales;
    int x_scale_ld;
    Groups groups;
    int N, K;
    void* dw;                 // [G][N][K]
    bool dw_f32;
};
hipError_t launch_grouped_wgrad(const WgradLaunch& L, hipStream_t stream);

struct SwigluLaunch {
    const uint16_t* h;        // [rows][2*inner]
    int inner;
    Groups groups;
    uint8_t* codes;           // [rows][inner]
    float* scales;
    int scale_ld;
    uint8_t* ckpt;            // [rows][2*inner] or NULL
    float* ckpt_scales;       // [rows][2*inner/128]
};
hipError_t launch_swiglu(const SwigluLaunch& L, hipStream_t stream);

struct SwigluBackwardLaunch {
    const uint16_t* da;       // [rows][inner]
    const uint8_t* ckpt;
    const float* ckpt_scales;
    int inner;
    Groups groups;
    uint16_t* dh;             // [rows][2*inner] or NULL
    uint8_t* codes;           // [rows][2*inner] or NULL
    float* scales;
    int scale_ld;
};
hipError_t launch_swiglu_backward(const SwigluBackwardLaunch& L, hipStream_t stream);

struct GateLaunch {
    const void* logits;
    bool bf16;
    int64_t ld;               // elements between rows
    int T, E, K;
    bool sigmoid, normalize;
    float scale, coef;
    const uint8_t* token_mask;
    int64_t* topk_idx;
    float* topk_weights;
    int32_t* counts;          // [E]
    int32_t* num_valid;       // [1]
    float* loss;              // [1]
    float* part_p;            // workgroups' sums, in the workspace (set by launch_gate)
    int32_t* part_n;
    int32_t* part_v;
};
size_t gate_workspace(int T, int E);
hipError_t launch_gate(GateLaunch L, void* ws, hipStream_t stream);

struct GateBackwardLaunch {
    const void* logits;
    bool bf16;
    int64_t ld;
    int T, E, K;
    bool sigmoid, normalize;
    float scale, coef;
    const uint8_t* token_mask;
    const int64_t* topk_idx;
    const int32_t* counts;
    const int32_t* num_valid;
    const float* grad_weights;   // [T][K] or NULL
    const float* grad_loss;      // [1] or NULL
    void* grad_logits;           // [T][E], dense, the logits' type
};
hipError_t launch_gate_backward(const GateBackwardLaunch& L, hipStream_t stream);

}  // namespace moe_ep
