// layer_launch.hpp -- host-side launchers of the operators around the chunked
// scan: the short causal convolution and the per-channel scan.  Arguments are
// already validated by the C ABI layer (api_layer.hpp); these only enqueue.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// ---- short causal convolution (kernels_conv.hip) -------------------------------
struct ConvShape {
    int64_t Bz, L, C;
    int W;                 // taps, 2..4
    int64_t xb, xr;        // elements between x's batches and steps
    int64_t piece[3];      // widths of the pieces of y / dy (unused: 0)
    bool bf16, silu;
};
// Steps one wavefront walks; a workgroup is kConvWaves wavefronts consecutive
// in time (shapes.cpp).
constexpr int kConvWaves = 4;
int64_t conv_rows(const ConvShape& s, bool bwd);
int64_t conv_time_blocks(const ConvShape& s, int64_t rows);   // workgroups along a sequence, at least 1
// The backward's parts of dweight and dbias: [Bz * time blocks][W + 1][C]
int64_t conv_bwd_parts(const ConvShape& s);
hipError_t launch_conv_fwd(const ConvShape& s, const void* x, const float* weight, const float* bias,
                           const void* win0, const int32_t* lens, void* const* y, void* win1, hipStream_t st);
hipError_t launch_conv_bwd(const ConvShape& s, const void* x, const float* weight, const float* bias,
                           const void* win0, const int32_t* lens, const void* const* dy, const void* dwin1,
                           void* dx, float* dweight, float* dbias, void* dwin0, float* parts, hipStream_t st);
hipError_t launch_conv_step(const ConvShape& s, void* window, const void* x, const float* weight,
                            const float* bias, void* const* y, hipStream_t st);

}  // namespace ssd
