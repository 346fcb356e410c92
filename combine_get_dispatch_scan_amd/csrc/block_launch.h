// Host-side launchers of the operators around the expert layer (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "groups.h"
#include "moe_ep.h"

namespace moe_ep {

void debug_launch(const char* kernel, dim3 grid, dim3 block, size_t lds);

struct BlockNormLaunch {
    ep_block_norm_t in;
    void* xo;                 // [rows][width], x's type, or NULL
    uint16_t* h;              // or NULL
    uint8_t* codes;           // or NULL
    float* scales;            // [rows][width/128]
};
hipError_t launch_block_norm(const BlockNormLaunch& L, hipStream_t stream);

struct BlockNormBackwardLaunch {
    ep_block_norm_t in;
    const void* gx;           // or NULL
    const uint16_t* gh;       // or NULL
    void* dx;                 // or NULL
    uint16_t* dy;             // or NULL
    void* dw;                 // or NULL
    void* dyw;                // or NULL
    void* dgate;              // or NULL
    float* part;              // workgroups' column sums, [blocks][2][width], or NULL
};
size_t block_norm_workspace(int rows, int width);
hipError_t launch_block_norm_backward(const BlockNormBackwardLaunch& L, hipStream_t stream);

hipError_t launch_quantize_fp4(const void* w, bool w_f32, int64_t groups32, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream);
hipError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t groups32, void* out,
                                 bool out_f32, hipStream_t stream);

struct GemmFp4Launch {
    const uint8_t* x;         // [rows][K] E4M3FN
    const float* x_scales;    // ld 0: [rows][K/128], else [K/128][ld]
    int x_scale_ld;
    const uint8_t* w;         // [G][N][K/2] E2M1
    const uint8_t* w_scales;  // [G][N][K/32] E8M0
    Groups groups;
    int N, K;
    int expected_rows;        // typical rows of a group (chooses the tile)
    uint16_t* out;            // [rows][N]
};
hipError_t launch_grouped_gemm_fp4(const GemmFp4Launch& L, hipStream_t stream);

}  // namespace moe_ep
