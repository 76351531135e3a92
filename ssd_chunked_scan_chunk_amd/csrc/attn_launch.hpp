// attn_launch.hpp -- host-side launchers of linear attention with a decay per head
// and of the norm over groups of channels.  Arguments are already validated by
// the C ABI layer (api_attn.hpp); these only enqueue.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// The most workgroups of a launch: 512 threads each, 2^32 items at most.
constexpr int64_t kAttnGroups = ((int64_t)1 << 23) - 1;

// ---- linear attention (kernels_attn*.hip) ----------------------------------------
struct AttnShape {
    int64_t Bz, L, H, K;                 // K: heads of k and v
    int64_t Dk, Dv;
    int64_t qb, qr, kb, kr, vb, vr;      // batch and step strides in elements
    bool bf16;
    float scale;
};
// One walk over the sequences, in time or against it: with rows a, c of `cd`
// elements and rows x of `xd`
//     S[t] = gamma S[t-1] + scale_w x[t] c[t]^T,   y[t] = S[t] a[t],
// the part of y from inside a chunk times scale_p, the rest times scale_in.  The
// forward and each of the gradients is one such walk.
struct AttnPass {
    const void *a, *c, *x;
    void* y;                             // dense [Bz][L][H][xd]; fp32 if y_f32
    int64_t ab, cb, xb;                  // batch strides in elements
    uint32_t ar, cr, xr;                 // step strides in elements
    int ag, cg, xg;                      // heads that share a head of a, c, x
    int cd, xd;
    const float *first;                  // states [Bz][H][Dv][Dk] (or NULL)
    float* last;
    int sc, sx;                          // element (c, x) of a state is at c * sc + x * sx
    float scale_p, scale_in, scale_w;
    int rev, y_f32;
    int exact;                           // bf16: states to 25 bits, as they are results, not to 17 (y is
                                         // rounded to 8; the same whether `last` is asked for).  A
                                         // backward of 4 x 2048 x 40 heads of 128 x 128 with it for
                                         // dq and dk too: 245 us, else 238; the error of each against
                                         // 64 bits is the same, its rounding's
};
// The first `whole` (batch, head) pairs are walked in one piece, the others in nseg segments
// of `steps` steps (whole chunks of every walk's).  The workspace: the states at the
// segments' ends [pairs - whole][nseg - 1][Dv][Dk], forward and backward, and the heads'
// gradients of shared keys and values (shapes.cpp).
struct AttnPlan {
    int64_t whole, steps, nseg;
    size_t states, adjoint, dk, dv, bytes;   // offsets; bytes in all
};
AttnPlan attn_plan(const AttnShape& s, bool bwd);
// columns of a workgroup, and workgroups across `xd` columns
inline int attn_columns(int64_t xd) { return xd > 64 ? 128 : 64; }
inline int64_t attn_slices(int64_t xd) { return (xd + attn_columns(xd) - 1) / attn_columns(xd); }
// contracted elements the kernels hold for `cd`
inline int attn_width(int64_t cd) { return cd > 128 ? 256 : cd > 64 ? 128 : 64; }
// steps of a chunk
inline int attn_chunk(bool bf16, int64_t cd, int64_t xd) {
    return bf16 && attn_width(cd) == 128 && attn_columns(xd) == 128 ? 64 : 32;
}

// n walks (at most two, to slots[0] and [1]): the states at the ends of all segments but the last,
// each from nothing (the first from p.first); then joined there
hipError_t launch_attn_states(const AttnShape& s, const AttnPlan& pl, const AttnPass* p, float* const* slots, int n,
                              const float* log_decay, const int32_t* lens, hipStream_t st);
// n walks (at most three); those of the same sizes side by side share a launch
hipError_t launch_attn_walks(const AttnShape& s, const AttnPlan& pl, const AttnPass* p, float* const* slots, int n,
                             const float* log_decay, const int32_t* lens, hipStream_t st);
// sums over each key and value head's heads: [Bz][L][H][..] fp32 -> dk, dv [Bz][L][K][..]
hipError_t launch_attn_share(const AttnShape& s, const float* dk_heads, const float* dv_heads, void* dk, void* dv,
                             hipStream_t st);
hipError_t launch_attn_step(const AttnShape& s, float* state, const void* q, const void* k, const void* v,
                            const float* log_decay, void* y, hipStream_t st);

// ---- group norm (kernels_norm.hip) --------------------------------------------------
struct NormShape {
    int64_t Bz, L, C, G;
    int64_t xb, xr, zb, zr;              // batch and row strides of x and the gate in elements
    float eps;
    bool bf16, center, silu, gate_first;
};
struct NormIn {
    const void *x, *gate;
    const float *weight, *bias;
    const int32_t* lens;
};
// How rows lie over the GPU (shapes.cpp): channels of a thread's piece (16 bytes of them, or
// 1 where a group is smaller), pieces of a thread, lanes of a group (block: the whole
// workgroup), groups and rows of a workgroup, workgroups across a row and down the rows.
struct NormLayout {
    int vec, pieces, lanes, gw, rw, threads;
    bool block;
    int64_t across, down;
};
constexpr int64_t kNormMost = 16384;          // channels of a group
NormLayout norm_layout(const NormShape& s, bool bwd);
int64_t norm_bwd_parts(const NormShape& s);   // rows of the partial sums of dweight and dbias
hipError_t launch_norm_fwd(const NormShape& s, const NormIn& in, void* y, hipStream_t st);
hipError_t launch_norm_bwd(const NormShape& s, const NormIn& in, const void* dy, void* dx, void* dgate, float* dweight,
                           float* dbias, float* parts, hipStream_t st);

}  // namespace ssd
