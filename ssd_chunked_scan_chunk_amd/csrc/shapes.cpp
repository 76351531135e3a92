// shapes.cpp -- host-side description of the compiled kernel set: which
// shapes each kernel family takes and how the forward MFMA kernel groups
// heads into workgroups.  Host code only (no kernels), so the C ABI's
// planning can also be built and checked without a GPU toolchain.
#include "attn_launch.hpp"
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

// Segments of the linear attention's walks.  A walk of an instance takes `few` us for 64 steps
// where its workgroups have the GPU nearly to themselves, `few` + `more` where `slots` of them
// fill it, and `ends` where it only makes the segments' end states.  Fitted on MI355X to
// the forward and the backward of 1 x 32768 to 8 x 2048 steps and 1 to 64 heads of all widths
// (bf16, 128 x 128: 8 x 2048 x 32 heads 139 us, 1 x 32768 x 12 in 16, 21 and 40 segments 173, 160
// and 183 us, its backward in 7 and 21 390 and 404 us; fp32: 2 x 2048 x 40 whole 261, in 3 and
// 6 segments 161 and 190 us, 3 x 517 x 6 in 1, 5 and 9 62, 34 and 26 us; the chosen number is
// within 10% of the best of those tried).  What a last round that does not fill the GPU would
// hold may be cut into segments while the rest stays whole: 8 x 2048 x 40 heads 223 us whole,
// 203 us with 64 pairs in four.
AttnPlan attn_plan(const AttnShape& s, bool bwd) {
    struct Rate { double few, more, ends; int64_t slots; };
    const int kd = attn_width(s.Dk > s.Dv && bwd ? s.Dk : bwd ? s.Dv : s.Dk);
    const bool narrow = attn_columns(bwd && s.Dk > s.Dv ? s.Dk : s.Dv) == 64;
    const Rate bf16 = kd == 256             ? Rate{5.0, 2.6, 3.0, 256}
                      : kd == 128 && !narrow ? Rate{3.0, 1.2, 1.6, 256}
                      : kd == 64 && narrow   ? Rate{2.5, 2.8, 1.5, 768}
                                             : Rate{3.0, 3.0, 1.8, 512};
    const Rate f32 = kd == 256             ? Rate{narrow ? 19.0 : 16.5, 2.0, 9.0, 256}
                     : kd == 128 && !narrow ? Rate{7.6, 2.4, 4.0, 256}
                     : kd == 128            ? Rate{8.2, 1.2, 4.0, 256}
                     : narrow               ? Rate{5.3, 3.0, 2.7, 512}
                                            : Rate{5.5, 1.3, 2.7, 256};
    const Rate& t = s.bf16 ? bf16 : f32;
    AttnPlan p = {};
    const int64_t chunks = (s.L + 63) / 64, pairs = s.Bz * s.H, walks = bwd ? 3 : 1;
    const int64_t slices = attn_slices(s.Dk) > attn_slices(s.Dv) && bwd ? attn_slices(s.Dk) : attn_slices(s.Dv);
    const int64_t per = slices * walks;                       // workgroups of a whole pair
    auto time = [&](int64_t groups, int64_t steps64, double few, double more) {
        const int64_t rounds = groups / t.slots, left = groups % t.slots;
        return (double)steps64 * ((double)rounds * (few + more) +
                                  (left ? few + more * (double)left / (double)t.slots : 0.0));
    };
    double least = 1e300;
    int64_t each = chunks > 0 ? chunks : 1;
    // every length e of a segment once: 2 sqrt(chunks) of them
    for (int64_t n = 1, next; n <= 512 && pairs > 0 && n <= chunks; n = next) {
        const int64_t e = (chunks + n - 1) / n, segs = (chunks + e - 1) / e;
        next = e > 1 ? (chunks + e - 2) / (e - 1) : chunks + 1;
        for (int64_t whole : {(int64_t)0, pairs * per / t.slots * t.slots / per}) {
            const int64_t cut = pairs - whole;
            // the walks' workgroups, and the join's: 256 threads for 256 numbers of a state
            if (segs > 1 && (cut > kAttnGroups / (segs * per) || cut > kAttnGroups / 256)) continue;
            double us = time(whole * per, chunks, t.few, t.more) + time(cut * segs * per, e, t.few, t.more);
            if (segs > 1 && cut > 0)
                us += time(cut * (segs - 1) * slices * (bwd ? 2 : 1), e, t.ends, 0.2 * t.ends) + 11 + 0.15 * (double)segs +
                      (double)(cut * (segs - 1) * s.Dk * s.Dv * (bwd ? 2 : 1)) * 8 / 4.5e6;
            if (us < least * (n > 1 ? 0.97 : 1.0)) {
                least = us;
                each = e;
                p.whole = segs > 1 ? whole : 0;
            }
        }
    }
    p.steps = 64 * each;
    p.nseg = chunks > 0 ? (chunks + each - 1) / each : 1;
    if (p.nseg == 1) p.whole = pairs;
    const size_t state = (size_t)((pairs - p.whole) * (p.nseg - 1) * s.Dk * s.Dv) * sizeof(float);
    const size_t rows = bwd && s.K != s.H ? (size_t)(s.Bz * s.L * s.H) * sizeof(float) : 0;
    auto take = [&](size_t n) {
        const size_t at = p.bytes;
        p.bytes += (n + 255) / 256 * 256;
        return at;
    };
    p.states = take(state);
    p.adjoint = take(bwd ? state : 0);
    p.dk = take(rows * s.Dk);
    p.dv = take(rows * s.Dv);
    return p;
}

// A group's channels over lanes of a wavefront if 64 pieces hold them, else over a
// workgroup of up to 16 wavefronts.  Rows are walked by as many workgroups as fill the
// GPU, the same columns in every one (the backward leaves one part of dweight and dbias
// for each).
NormLayout norm_layout(const NormShape& s, bool bwd) {
    NormLayout l = {};
    const int64_t m = s.C / s.G, full = s.bf16 ? 8 : 4, rows = s.Bz * s.L;
    l.vec = (int)(m < full ? 1 : full);
    const int64_t pieces = (m + l.vec - 1) / l.vec;
    l.pieces = 1;
    l.rw = 1;
    if (pieces <= 64) {
        l.lanes = 1;
        while (l.lanes < pieces) l.lanes *= 2;
        const int64_t waves = (s.G * l.lanes + 63) / 64;
        l.across = (waves + 7) / 8;
        const int64_t each = (waves + l.across - 1) / l.across;
        l.gw = (int)(each * 64 / l.lanes);
        if (l.gw > s.G) l.gw = (int)s.G;
        if (l.across == 1 && s.G * l.lanes <= 128) l.rw = (int)(256 / (s.G * l.lanes));
        l.threads = (int)((l.gw * l.rw * l.lanes + 63) / 64 * 64);
        l.across = (s.G + l.gw - 1) / l.gw;
    } else {
        l.block = true;
        l.lanes = 64;
        while ((pieces + 64 * l.pieces - 1) / (64 * l.pieces) > 16) l.pieces *= 2;   // 4 at most, as m is at most kNormMost
        l.threads = (int)((pieces + 64 * l.pieces - 1) / (64 * l.pieces) * 64);
        l.gw = 1;
        l.across = s.G;
    }
    const int64_t want = (256 * 2048 / l.threads + l.across - 1) / l.across, most = (rows + l.rw - 1) / l.rw;
    const int64_t cap = bwd ? 512 : 32768;
    l.down = want < most ? want : most;
    if (l.down > cap) l.down = cap;
    if (l.down < 1) l.down = 1;
    return l;
}
int64_t norm_bwd_parts(const NormShape& s) {
    return norm_layout(s, true).down;
}

}  // namespace ssd
