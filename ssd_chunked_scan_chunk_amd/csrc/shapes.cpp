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

int conv_vec(const ConvShape& s) {
    for (const int64_t w : s.piece)
        if (w > 0 && w < 4) return 1;
    return 4;
}
// The longest walk that leaves enough wavefronts: short walks read their filters
// and the rows ahead of them more often (the backward also redoes W-1 steps and
// writes more parts of dweight), long ones are too few to hide latency.  On MI355X,
// bf16, four channels per thread: forward 8 x 4096 x 5376 at 4, 16 and 64 steps 223,
// 139 and 145 us, 1 x 1024 x 1792 at 4, 16 and 64 5.1, 6.3 and 15 us (the kernel);
// backward 4 x 2048 x 5376 at 4, 16 and 64 134, 73 and 63 us, 4 x 2048 x 1792 at 8, 32
// and 64 37, 30 and 42 us.
int64_t conv_rows(const ConvShape& s, bool bwd) {
    const int64_t wide = 64 * conv_vec(s), across = s.Bz * ((s.C + wide - 1) / wide);
    int64_t rows = bwd ? 64 : 16;
    while (rows > 4 && across * ((s.L + rows - 1) / rows) < (bwd ? 1700 : 1024)) rows /= 2;
    return rows;
}
int64_t conv_time_blocks(const ConvShape& s, int64_t rows) {
    const int64_t n = (s.L + kConvWaves * rows - 1) / (kConvWaves * rows);
    return n > 0 ? n : 1;
}
int64_t conv_bwd_parts(const ConvShape& s) { return s.Bz * conv_time_blocks(s, conv_rows(s, true)); }

int64_t chan_tiles(const ChanShape& s, int cw) { return s.G * ((s.D / s.G + cw - 1) / cw); }
// Nanoseconds a CU takes for one step of the r workgroups it holds: the latency
// of a step while few run, the rate of vector issue once they fill it.  Fitted on
// MI355X to forwards of 1 x 1536 to 8 x 5120 channels and 8, 16, 32 and 64 states at
// four wavefronts per SIMD (a step of one workgroup, 16 states: 118 ns at 64 channels,
// 88 ns at 32; filled: 65 and 38 ns per workgroup; most shapes within 15%).  At the five
// that up to 16 states run now, a filled step takes 60 and 31 ns; the plans still come
// within 4% of the best that was tried (1 x 32768 x 1536 x 16: 337 us, 328 in 96 segments).
static double chan_step_ns(int cw, int64_t N, int64_t r) {
    const double lat = cw == 64 ? 62 + 3.6 * N : 64 + 1.75 * N, rate = cw == 64 ? 21.7 + 2.7 * N : 16 + 1.41 * N;
    const double few = lat + 0.6 * (double)(r - 1) * rate, many = (double)r * rate;
    return few > many ? few : many;
}
// The cheapest of a few segment counts at 64 and at 32 channels per workgroup.
// Segments pay a second pass (0.72 of the steps' time), the scan over them (one
// read and one write of their states) and two launches: 2 x 2048 x 5120 x 16 takes
// 265 us in one segment, 149 us in 16; 8 x 2048 x 5120 x 16, whose channels fill the
// GPU, 414 us in one (64 channels wide throughout) and 524 us in 16.
ChanPlan chan_fwd_plan(const ChanShape& s) {
    const int64_t all = s.L > 0 ? s.L : 1;
    ChanPlan best{64, all, 1, 0};
    double least = 1e300;
    constexpr int kCounts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 192, 256};
    for (const int cw : {64, 32}) {
        for (const int want : kCounts) {
            const int64_t seg = ((s.L + want - 1) / want + 7) / 8 * 8;
            if (want > 1 && seg < 16) break;
            const int64_t nseg = s.L > 0 ? (s.L + seg - 1) / seg : 1;
            const int64_t r = (s.Bz * chan_tiles(s, cw) * nseg + 255) / 256;
            const double steps = (double)(nseg > 1 ? seg : s.L) * chan_step_ns(cw, s.N, r) * 1e-3;
            double us = steps;
            if (nseg > 1)
                us = 1.05 * (1.72 * steps + 10 + 0.05 * (double)nseg + 1e-6 * (double)(nseg * s.Bz * s.D * s.N));
            if (us < least) {
                least = us;
                best = ChanPlan{cw, nseg > 1 ? seg : all, nseg, 0};
            }
        }
    }
    // up to half a 64-wide workgroup per CU left over: as halves they add half a
    // workgroup's time to every CU, not a whole one's to some (8 x 2048 x 5120 x 16, 640
    // workgroups: 340 us against 414, and 385 if all are 32 channels wide)
    const int64_t flats = s.Bz * chan_tiles(s, 64), full = flats / 256, rest = flats % 256;
    if (full > 0 && rest > 0 && rest <= 128) {
        const double w = chan_step_ns(64, s.N, full), n = 16 + 1.41 * (double)s.N;
        const double us = (double)s.L * (w + 0.8 * n) * 1e-3;
        if (us < least) best = ChanPlan{64, all, 1, full * 256};
    }
    return best;
}
// the segments' end states (slot s becomes the state entering segment s) and
// their sums of dt
size_t chan_fwd_bytes(const ChanShape& s, const ChanPlan& p) {
    if (p.nseg <= 1) return 0;
    return (size_t)s.Bz * p.nseg * s.D * (s.N + 1) * sizeof(float);
}

// Segments of the backward: three to eleven workgroups per CU in all, as evenly as
// they come (the CU with one more sets the time), the fewer the better as each
// costs some twelve steps' time of its own, and none shorter than 16 steps.  4 x
// 2048 x 5120 x 16 (320 workgroups per segment) takes 1077 us in one segment, 657 in
// four, 678 in five, 650 in eight, 713 in 32; 1 x 2048 x 1536 x 16 (24) 805 us in one,
// 92 in 16, 74 in 32, 77 in 43.  64 channels to a workgroup measured 15% faster than
// 32 wherever a lane's states of a batch fit the registers (dstate up to 16).
ChanBwdPlan chan_bwd_plan(const ChanShape& s) {
    ChanBwdPlan p;
    p.cw = s.N <= 16 ? 64 : 32;
    const int64_t tiles = chan_tiles(s, p.cw), pieces = 256 / p.cw;
    const int64_t np = s.N <= 8 ? 8 : s.N <= 16 ? 16 : s.N <= 32 ? 32 : 64, nr = np / pieces;
    p.nr = (int)nr;
    const int64_t groups = s.Bz * tiles > 0 ? s.Bz * tiles : 1, most = s.L > 16 ? (s.L + 15) / 16 : 1;
    int64_t want = groups >= 768 ? 1 : (768 + groups - 1) / groups;
    if (want > most) want = most;
    double least = 1e300;
    p.seg = 16;
    for (int64_t k = want; k == want || (k <= most && groups * k <= 2816); k += 1 + k / 16) {
        const int64_t seg = ((s.L + k - 1) / k + 7) / 8 * 8, w = groups * k;
        const double uneven = (double)((w + 255) / 256 * 256) / (double)w;
        const double cost = uneven * (1.0 + 12.0 / (double)(seg > 0 ? seg : 8)) * (1.0 + 64.0 / (double)w);
        if (cost < least) {
            least = cost;
            p.seg = seg > 16 ? seg : 16;
        }
    }
    p.nseg = s.L > 0 ? (s.L + p.seg - 1) / p.seg : 1;
    p.nb = p.seg / 8;
    const int64_t rows = s.Bz * p.nseg;
    const bool several = p.nseg > 1;
    const int64_t floats[9] = {rows * p.nb * tiles * 256 * nr, several ? rows * p.nb * tiles * p.cw : 0,
                               several ? rows * tiles * 256 * nr : 0, several ? rows * tiles * 256 * nr : 0,
                               several ? rows * tiles * p.cw : 0, s.Bz * s.L * tiles * 2 * np, rows * s.D * s.N,
                               rows * s.D, rows * s.D};
    size_t o = 0;
    for (int i = 0; i < 9; ++i) {
        p.off[i] = o;
        o += ((size_t)floats[i] * 4 + 255) / 256 * 256;
    }
    p.off[9] = s.Bz > 0 ? o : 0;
    return p;
}

}  // namespace ssd
