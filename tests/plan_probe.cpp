// plan_probe.cpp -- the launch plans of the operators around the chunked scan
// (csrc/shapes.cpp) for the tests, built for the host alone.
#include "layer_launch.hpp"

extern "C" {

// channels of a workgroup, steps of a segment, segments, whole workgroups
void probe_chan_fwd(int64_t Bz, int64_t L, int64_t D, int64_t N, int64_t G, int64_t* out) {
    ssd::ChanShape s = {};
    s.Bz = Bz; s.L = L; s.D = D; s.N = N; s.G = G;
    const ssd::ChanPlan p = ssd::chan_fwd_plan(s);
    out[0] = p.cw; out[1] = p.seg; out[2] = p.nseg; out[3] = p.whole;
}

// channels of a workgroup, steps of a segment, segments
void probe_chan_bwd(int64_t Bz, int64_t L, int64_t D, int64_t N, int64_t G, int64_t* out) {
    ssd::ChanShape s = {};
    s.Bz = Bz; s.L = L; s.D = D; s.N = N; s.G = G;
    const ssd::ChanBwdPlan p = ssd::chan_bwd_plan(s);
    out[0] = p.cw; out[1] = p.seg; out[2] = p.nseg;
}

// channels of a workgroup, states of a thread, and the bytes that the batches' states,
// the segments' states, their adjoints and the sums of dB and dC have in the workspace
void probe_chan_bwd_regions(int64_t Bz, int64_t L, int64_t D, int64_t N, int64_t G, int64_t* out) {
    ssd::ChanShape s = {};
    s.Bz = Bz; s.L = L; s.D = D; s.N = N; s.G = G;
    const ssd::ChanBwdPlan p = ssd::chan_bwd_plan(s);
    const int region[] = {0, 2, 3, 5};
    out[0] = p.cw; out[1] = p.nr;
    for (int i = 0; i < 4; ++i) out[2 + i] = (int64_t)(p.off[region[i] + 1] - p.off[region[i]]);
}

// channels of a thread, steps of a walk forward and backward
void probe_conv(int64_t Bz, int64_t L, int64_t p0, int64_t p1, int64_t p2, int64_t* out) {
    ssd::ConvShape s = {};
    s.Bz = Bz; s.L = L; s.C = p0 + p1 + p2;
    s.piece[0] = p0; s.piece[1] = p1; s.piece[2] = p2;
    out[0] = ssd::conv_vec(s); out[1] = ssd::conv_rows(s, false); out[2] = ssd::conv_rows(s, true);
}

}  // extern "C"
