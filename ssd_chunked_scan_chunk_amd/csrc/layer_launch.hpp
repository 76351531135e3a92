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
int conv_vec(const ConvShape& s);   // channels of a thread: 4, or 1 where a piece has fewer
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

// ---- per-channel scan (kernels_channel.hip) --------------------------------------
struct ChanShape {
    int64_t Bz, L, D, N, G;
    int64_t ub, ur, db, dr, zb, zr, Bb, Br, Cb, Cr;   // batch and step strides in elements
    bool bf16, softplus;
};
struct ChanIn {
    const void *u, *delta, *B, *C, *gate;
    const float *A, *skip, *dbias, *h0;
    const int32_t* lens;
};
// How the forward is laid over the GPU (shapes.cpp): channels of a workgroup (64
// or 32), and segments of `seg` steps the sequence is cut into; whole > 0: one
// segment, that many workgroups of 64 channels, the rest of 32.
struct ChanPlan {
    int cw;
    int64_t seg, nseg, whole;
};
ChanPlan chan_fwd_plan(const ChanShape& s);
int64_t chan_tiles(const ChanShape& s, int cw);   // workgroups over the channels of one batch
size_t chan_fwd_bytes(const ChanShape& s, const ChanPlan& p);
hipError_t launch_chan_fwd(const ChanShape& s, const ChanPlan& p, const ChanIn& in, void* y, float* hfin,
                           float* ws, hipStream_t st);
// The backward's instance (channels of a workgroup, 64 or 32, and states of a thread, by
// the number of states; the launcher takes these, which the regions are laid out for),
// segments, batches of eight steps per segment, and the workspace's regions: states
// of the batches and their sums of dt, states, adjoints and sums of dt of the
// segments, the workgroups' sums of dB and dC, the segments' of dA, dskip, dbias.
struct ChanBwdPlan {
    int cw, nr;
    int64_t seg, nseg, nb;
    size_t off[10];          // off[9]: bytes in all
};
struct ChanGrads {
    void *du, *ddelta, *dgate, *dB, *dC;
    float *dA, *dskip, *ddbias, *dh0;
};
ChanBwdPlan chan_bwd_plan(const ChanShape& s);
hipError_t launch_chan_bwd(const ChanShape& s, const ChanBwdPlan& p, const ChanIn& in, const void* dy,
                           const float* dh, const ChanGrads& o, void* ws, hipStream_t st);
hipError_t launch_chan_step(const ChanShape& s, float* state, const ChanIn& in, void* y, hipStream_t st);

}  // namespace ssd
