// attn_plan_probe.cpp -- the plans of linear attention and the layouts of the group norm
// (csrc/shapes.cpp) for the tests, built for the host alone.
#include "attn_launch.hpp"

extern "C" {

// whole pairs, steps of a segment, segments, bytes of the workspace
void probe_attn(int64_t Bz, int64_t L, int64_t H, int64_t K, int64_t Dk, int64_t Dv, int64_t bf16, int64_t bwd,
                int64_t* out) {
    ssd::AttnShape s = {};
    s.Bz = Bz; s.L = L; s.H = H; s.K = K; s.Dk = Dk; s.Dv = Dv; s.bf16 = bf16 != 0;
    const ssd::AttnPlan p = ssd::attn_plan(s, bwd != 0);
    out[0] = p.whole; out[1] = p.steps; out[2] = p.nseg; out[3] = (int64_t)p.bytes;
}

// channels of a piece, pieces of a thread, lanes of a group, groups and rows of a workgroup, threads, whether
// a workgroup holds one group, workgroups across a row and down the rows, parts
void probe_norm(int64_t Bz, int64_t L, int64_t C, int64_t G, int64_t bf16, int64_t bwd, int64_t* out) {
    ssd::NormShape s = {};
    s.Bz = Bz; s.L = L; s.C = C; s.G = G; s.bf16 = bf16 != 0;
    const ssd::NormLayout l = ssd::norm_layout(s, bwd != 0);
    out[0] = l.vec; out[1] = l.pieces; out[2] = l.lanes; out[3] = l.gw; out[4] = l.rw; out[5] = l.threads;
    out[6] = l.block; out[7] = l.across; out[8] = l.down; out[9] = ssd::norm_bwd_parts(s);
}

}  // extern "C"
