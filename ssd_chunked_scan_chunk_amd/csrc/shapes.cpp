// shapes.cpp -- host-side description of the compiled kernel set: which
// shapes each kernel family takes and how the forward MFMA kernel groups
// heads into workgroups.  Host code only (no kernels), so the C ABI's
// planning can also be built and checked without a GPU toolchain.
#include "layer_launch.hpp"
#include "ssd_launch.hpp"

namespace ssd {

bool mfma_supported(int64_t Q, int64_t P, int64_t N) {
    return (Q == 64 || Q == 128 || Q == 256) && (P == 32 || P == 64) && (N == 64 || N == 128);
}

int64_t mfma_heads_per_workgroup(int64_t P, int64_t N) {
    (void)N;
    return kMfmaStateWaves / (P / 32);
}

// The fused pass's units per workgroup: 4, 5 or 6 for headdim 64; 4 or 5
// for headdim 32 (six single-unit heads would need more LDS for their
// per-head stage-1 results than a CU has).
bool fwd_units_supported(int64_t P, int sw) {
    return sw == 4 || sw == 5 || (sw == 6 && P == 64);
}

bool valu_fwd_supported(const FwdShape& s) {
    return s.Q >= 1 && s.Q <= 256 && s.P * s.N <= 16384;
}

bool bwd_da_supported(int64_t Q, int64_t P, int64_t N) {
    return (Q == 64 || Q == 128 || Q == 256) && (P == 32 || P == 64) && (N == 64 || N == 128);
}

// bytes of the da kernel's C B^T tiles: every (batch, chunk, group) holds the
// T(T+1)/2 lower-triangle 32x32 fp32 tiles of its chunk, T = chunk / 32
int64_t cb_tiles_bytes(const FwdShape& s) {
    const int64_t nI = s.Q / 32;
    return s.Bz * s.nc * s.G * (nI * (nI + 1) / 2) * 1024 * 4;
}

int64_t conv_rows(const ConvShape& s, bool bwd) {
    (void)s;
    (void)bwd;
    return 32;
}
int64_t conv_time_blocks(const ConvShape& s, int64_t rows) {
    const int64_t n = (s.L + kConvWaves * rows - 1) / (kConvWaves * rows);
    return n > 0 ? n : 1;
}
int64_t conv_bwd_parts(const ConvShape& s) { return s.Bz * conv_time_blocks(s, conv_rows(s, true)); }

int64_t chan_tiles(const ChanShape& s, int R) {
    const int64_t per = s.D / s.G, w = 16 * R;
    return s.G * ((per + w - 1) / w);
}
ChanPlan chan_fwd_plan(const ChanShape& s) {
    return ChanPlan{1, s.L > 0 ? s.L : 1, 1};
}
// the segments' end states (slot s becomes the state entering segment s) and
// their sums of dt
size_t chan_fwd_bytes(const ChanShape& s, const ChanPlan& p) {
    if (p.nseg <= 1) return 0;
    return (size_t)s.Bz * p.nseg * s.D * (s.N + 1) * sizeof(float);
}

}  // namespace ssd
