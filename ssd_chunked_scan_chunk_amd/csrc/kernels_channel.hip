// kernels_channel.hip -- the scan with one decay per channel and state on
// gfx950: forward and single-token step.
//
//     dt = softplus(delta + bias),  h[n] = e^{dt A[n]} h[n] + dt u B[n],
//     y = (sum_n h[n] C[n] + skip u) silu(gate)
// for every (batch, channel), n < N states.  Every (step, channel, state) costs
// two multiplications, an exponential and two fused multiply-adds, none of which
// the matrix units can take (no operand is shared between channels): 24 cycles of
// a SIMD for 64 of them, so the forward is bound by vector issue and the kernel
// is laid out to spend little beside those.
//
// A workgroup owns 64 consecutive channels of a group (32 where that balances the
// GPU better), a lane one of them and a quarter (an eighth) of its states, in
// registers.  Steps are taken in batches of eight: dt and dt u are formed once,
// spread over the workgroup, and passed through LDS with the batch's B and C (the
// same for all channels: broadcast reads), the parts of every step's y are summed
// through LDS, and one barrier per batch orders all of it; inputs are in flight
// two batches ahead.  The recurrence itself runs sequentially, which needs the
// fewest operations; the sequence is cut into segments only where the channels
// alone leave the GPU idle (a first pass then finds each segment's end state from
// zero and its sum of dt, a scan over segments the states entering them; the
// decay over a segment is e^{A sum dt}).
#include <type_traits>

#include "chan_util.hpp"

namespace ssd {

namespace {

template <int V> using Int = std::integral_constant<int, V>;

constexpr int TB = 8;   // steps of a batch

template <int NR, int CW, bool FULL> struct FwdLds {
    static constexpr int kParts = 256 / CW;
    float2 dt[2][TB][CW];                                    // dt, dt u
    float bc[2][TB * kParts * NR * (FULL ? 2 : 1)];          // [B, C][step][state]
    float y[FULL ? 2 : 1][FULL ? TB : 1][kParts][CW];
};

// The scan of the CW channels from cg0 on of group g, in segment `seg` of batch b.
// CW: channels of a workgroup (64, or 32 with half the states in each half of a
// wavefront); NR: states of a lane, 256 / CW parts of a channel's states.
// FULL: outputs from the states entering each segment; otherwise each segment's
// end state from zero (S) and its sum of dt.
template <typename T, int NR, int CW, bool FULL>
__device__ __forceinline__ void chan_fwd(const ChanArgs& a, FwdLds<NR, CW, FULL>& lds, int g, int cg0, int64_t b,
                                         int64_t seg)
{
    constexpr int ES = sizeof(T), NPART = 256 / CW, NP = NPART * NR;
    constexpr int TP = TB * CW / 256;               // (step, channel) pairs of a thread
    constexpr int NBC = TB * NP * (FULL ? 2 : 1);   // elements of B and C in a batch
    constexpr int NE = (NBC + 255) / 256;           // of these, passed on by a thread
    constexpr bool EXACT = ES == 4;
    const int tid = threadIdx.x, c = tid & (CW - 1), part = tid / CW, n0 = part * NR;
    const int cg = cg0 + c;
    const bool live = cg < a.per;
    // threads past the group repeat its last channel and store nothing
    const int cl = live ? cg : a.per - 1;
    uint32_t col = (uint32_t)cl * ES;
    const int64_t gch = (int64_t)g * a.per, ch = gch + cl;
    const int64_t ts = seg * a.seg, t1 = ts + a.seg < a.L ? ts + a.seg : a.L;
    const int64_t len = chan_length(a.in.lens, b, a.L);
    const int te = (int)(len < ts ? 0 : (len < t1 ? len : t1) - ts);   // steps to compute from ts on
    const bool gated = a.in.gate != nullptr;

    float A2[NR], h[NR] = {}, sdt = 0.f;
    const float bias = a.in.dbias ? a.in.dbias[ch] : 0.f, skip = a.in.skip ? a.in.skip[ch] : 0.f;
    const float* h0 = !FULL ? nullptr
                      : seg > 0 ? a.S + ((b * a.nseg + seg) * a.D + ch) * a.N
                      : a.in.h0 ? a.in.h0 + (b * a.D + ch) * a.N : nullptr;
    // rows of the batch being fetched, and of the one being written
    RowIn up = row_in(a.in.u, (b * a.ub + gch) * ES + ts * a.ur);
    RowIn dp = row_in(a.in.delta, (b * a.db + gch) * ES + ts * a.dr);
    RowIn zp = row_in(gated ? a.in.gate : a.in.u, (b * a.zb + gch) * ES + ts * a.zr);
    RowIn Bp = row_in(a.in.B, (b * a.Bb + (int64_t)g * a.N) * ES + ts * a.Br);
    RowIn Cp = row_in(a.in.C, (b * a.Cb + (int64_t)g * a.N) * ES + ts * a.Cr);
    const uint32_t yr = (uint32_t)a.D * ES;
    RowOut yp = row_out(a.y, ((b * a.L + ts) * a.D + gch) * ES);

    // This thread's pairs of a batch are the steps part + k NPART of channel c, its
    // elements of B and C those at e 256 + tid; offsets in the batch's rows.  Steps
    // past `last` repeat that one.
    const int wave64 = __builtin_amdgcn_readfirstlane(tid >> 6) * 64;
    auto in_C = [&](int e) { return FULL && e * 256 + wave64 >= TB * NP; };   // else in B
    uint32_t ou[TP], od[TP], oz[TP], oy[TP], obc[NE];
    auto offsets = [&](int last) {
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int s = part + k * NPART;
            const uint32_t r = s < last ? s : last;
            ou[k] = r * a.ur + col;
            od[k] = r * a.dr + col;
            oz[k] = r * a.zr + col;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int i = e * 256 + tid, s = i / NP & (TB - 1), n = i & (NP - 1);
            const uint32_t r = s < last ? s : last;
            obc[e] = r * (in_C(e) ? a.Cr : a.Br) + (uint32_t)(n < a.N ? n : a.N - 1) * ES;
        }
    };
    // Two batches in flight: the one at t, or past the end the last one again.
    T ru[2][TP], rd[2][TP], rz[2][TP], rbc[2][NE];
    auto fetch = [&](auto slot, int t) {
        constexpr int P = decltype(slot)::value;
        const int last = te - 1 - t;
        if ((FULL || last >= 0) && last < TB - 1) offsets(last);
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            ru[P][k] = load_at<T>(up, ou[k]);
            rd[P][k] = load_at<T>(dp, od[k]);
            if (FULL) rz[P][k] = load_at<T>(zp, oz[k]);
        }
#pragma unroll
        for (int e = 0; e < NE; ++e)
            rbc[P][e] = load_at<T>(in_C(e) ? Cp : Bp, obc[e]);
        if (FULL || last >= TB) {
            up += TB * (uint64_t)a.ur;
            dp += TB * (uint64_t)a.dr;
            zp += TB * (uint64_t)a.zr;
            Bp += TB * (uint64_t)a.Br;
            Cp += TB * (uint64_t)a.Cr;
        }
    };
    float u[2][TP], z[2][TP];
    auto prepare = [&](int t, auto slot) {
        constexpr int P = decltype(slot)::value;
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int s = part + k * NPART;
            const bool on = t + s < te;   // a step past the end changes nothing, whatever it repeats
            const float x = as_f32(rd[P][k]) + bias, sp = softplus_of<EXACT>(x);
            float dt = a.softplus ? sp : x;
            dt = on ? dt : 0.f;
            u[P][k] = on ? as_f32(ru[P][k]) : 0.f;
            z[P][k] = as_f32(rz[P][k]);
            sdt += dt;
            lds.dt[P][s][c] = make_float2(dt, dt * u[P][k]);
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int i = e * 256 + tid;
            const bool in = (i & (NP - 1)) < a.N && t + (i / NP & (TB - 1)) < te;
            if (NBC % 256 == 0 || i < NBC) lds.bc[P][i] = in ? as_f32(rbc[P][e]) : 0.f;
        }
    };
    // The batch at t, whose values lie in slot P; the inputs of the one after the
    // next are fetched into that slot, those of the next prepared.
    auto batch = [&](int t, auto slot) {
        constexpr int P = decltype(slot)::value;
        // Without outputs to write, reading the last batch again past the end is faster:
        // beside reads that may not take place the compiler waits for both batches (147
        // against 139 us in 1 x 32768 x 1536 x 16).  With them it is slower (358 against 369
        // us in 8 x 2048 x 5120 x 16).
        if (!FULL || t + 2 * TB < te) fetch(slot, t + 2 * TB);
        if (t == 0 || !FULL) lds_barrier();   // otherwise the one below has ordered slot P
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            const float2 d = lds.dt[P][k][c];
            const float* bc = lds.bc[P] + k * NP + n0;
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float e = fast_exp2(d.x * A2[i]);
                h[i] = fmaf(e, h[i], d.y * bc[i]);
                if (FULL) y = i == 0 ? h[i] * bc[TB * NP + i] : fmaf(h[i], bc[TB * NP + i], y);
            }
            if (FULL) lds.y[P][k][part][c] = y;
        }
        if (t + TB < te) prepare(t + TB, Int<P ^ 1>());
        if constexpr (FULL) {
            lds_barrier();
#pragma unroll
            for (int k = 0; k < TP; ++k) {
                const int s = part + k * NPART;
                float y = 0.f;
#pragma unroll
                for (int q = 0; q < NPART; q += 2) y += lds.y[P][s][q][c] + lds.y[P][s][q + 1][c];
                y = fmaf(skip, u[P][k], y);
                const float sz = z[P][k] * sigmoid_of(z[P][k]);
                y *= gated ? sz : 1.f;
                if (live && t + s < te) store_at(yp, oy[k], y, T());
            }
        }
        yp += TB * (uint64_t)yr;
    };
#pragma unroll
    for (int k = 0; k < TP; ++k) oy[k] = (part + k * NPART) * yr + col;
    if (te > 0) {
        offsets(TB - 1);
        fetch(Int<0>(), 0);
        if (!FULL || TB < te) fetch(Int<1>(), TB);
    }
    load_values<NR>(a.in.A + ch * a.N, n0, a.N, A2);   // states past N: A = B = C = 0
    if (h0) load_values<NR>(h0, n0, a.N, h);
    if (te > 0) {
        prepare(0, Int<0>());
#pragma unroll
        for (int i = 0; i < NR; ++i) A2[i] = log2_rate(A2[i]);
        for (int t = 0; t < te; t += 2 * TB) {
            batch(t, Int<0>());
            if (t + TB < te) batch(t + TB, Int<1>());
        }
    }

    if constexpr (FULL) {
        const RowOut yz = row_out(a.y, ((b * a.L + ts) * a.D + gch) * ES);
        for (int64_t s = te + part; s < t1 - ts; s += NPART)
            if (live) store_at(yz + s * (uint64_t)yr, col, 0.f, T());
    }
    float* out = FULL ? (seg == a.nseg - 1 ? a.hfin : nullptr) : a.S;
    if (out) {
        const int64_t row = FULL ? b : b * a.nseg + seg + 1;   // slot s + 1: what enters the next segment
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (live && n0 + i < a.N) out[(row * a.D + ch) * a.N + n0 + i] = h[i];
        if constexpr (!FULL) {   // each thread summed its own share of the steps
            __syncthreads();
            float* sum = &lds.dt[0][0][0].x;
            sum[tid] = sdt;
            __syncthreads();
            sdt = 0.f;
#pragma unroll
            for (int q = 0; q < NPART; ++q) sdt += sum[q * CW + c];
            if (live && part == 0) a.sumdt[row * a.D + ch] = sdt;
        }
    }
}

// Five wavefronts per SIMD need two registers fewer than the compiler takes with up to
// four states in a lane (16 x 1024 x 5120 x 16, five workgroups per CU: 337 us at four,
// 321 at five; six would spill, 696 us).
template <typename T, int NR, int CW, bool FULL>
__global__ __launch_bounds__(256, NR <= 4 ? 5 : FULL ? 4 : 2) void k_chan_fwd(ChanArgs a)
{
    __shared__ __align__(16) FwdLds<NR, CW, FULL> lds;
    const int g = blockIdx.x / a.tpg;
    chan_fwd<T, NR, CW, FULL>(a, lds, g, (blockIdx.x - g * a.tpg) * CW, blockIdx.z, blockIdx.y);
}

// One segment, the first `whole` workgroups 64 channels wide, the others the halves
// of the remaining 64-wide tiles: where the channels come to a few workgroups per CU
// and up to half a one more, the halves even out what the CUs get.
template <typename T, int NR>
__global__ __launch_bounds__(256, 4) void k_chan_fwd_mixed(ChanArgs a, int whole, int tiles)
{
    __shared__ __align__(16) union { FwdLds<NR, 64, true> w; FwdLds<NR / 2, 32, true> n; } lds;
    const int past = (int)blockIdx.x - whole, flat = past < 0 ? blockIdx.x : whole + past / 2;
    const int b = flat / tiles, tile = flat - b * tiles, g = tile / a.tpg, cg0 = (tile - g * a.tpg) * 64;
    if (past < 0) {
        chan_fwd<T, NR, 64, true>(a, lds.w, g, cg0, b, 0);
    } else {
        const int half = cg0 + (past & 1) * 32;
        if (half < a.per) chan_fwd<T, NR / 2, 32, true>(a, lds.n, g, half, b, 0);
    }
}

// S[seg + 1] <- e^{A sum dt} S[seg] + S[seg + 1], S[0] the initial state: slot
// s ends up holding the state that enters segment s.  One thread per (batch,
// channel, state); slots 1 .. nseg - 1.
__global__ __launch_bounds__(256) void k_chan_pass(ChanArgs a, int64_t items)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items) return;
    const int64_t DN = a.D * a.N, b = i / DN, dn = i - b * DN, ch = dn / a.N;
    const float A2 = log2_rate(a.in.A[dn]);
    float h = a.in.h0 ? a.in.h0[i] : 0.f;
    float* S = a.S + b * a.nseg * DN + dn;
    const float* sd = a.sumdt + b * a.nseg * a.D + ch;
    constexpr int U = 8;   // segments in flight
    for (int64_t s = 1; s < a.nseg; s += U) {
        float v[U], d[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s + k < a.nseg) { v[k] = S[(s + k) * DN]; d[k] = sd[(s + k) * a.D]; }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s + k < a.nseg) {
                h = fmaf(fast_exp2(A2 * d[k]), h, v[k]);
                S[(s + k) * DN] = h;
            }
    }
}

// Single token: LPC lanes per channel, four states each.  The states are read and
// written once, 128 bytes a channel at 16 of them: bound by HBM (256 x 5120 x 16: 37 us,
// 4.8 TB/s, above a large copy's median rate).
template <typename T, int LPC>
__global__ __launch_bounds__(256) void k_chan_step(ChanArgs a, float* __restrict__ state, int64_t items)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t bc = i / LPC;          // (batch, channel)
    const int n0 = (int)(i % LPC) * 4;
    const bool on = i < items;
    const int64_t b = on ? bc / a.D : 0, ch = on ? bc - b * a.D : 0;
    const int g = (int)(ch / a.per);
    const T* Bp = (const T*)a.in.B + b * a.Bb + (int64_t)g * a.N + n0;
    const T* Cp = (const T*)a.in.C + b * a.Cb + (int64_t)g * a.N + n0;
    const float* Ap = a.in.A + ch * a.N + n0;
    float* hp = state + (b * a.D + ch) * a.N + n0;
    float h[4], A[4], Bv[4], Cv[4];
    const bool quad = on && n0 + 4 <= a.N;
    if (quad) {
        const f32x4_any hv = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(hp));
        load_quad(Ap, A);
        load_quad(Bp, Bv);
        load_quad(Cp, Cv);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = hv[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool in = on && n0 + k < a.N;
            h[k] = in ? hp[k] : 0.f;
            A[k] = in ? Ap[k] : 0.f;
            Bv[k] = in ? as_f32(Bp[k]) : 0.f;
            Cv[k] = in ? as_f32(Cp[k]) : 0.f;
        }
    }
    const float u = on ? as_f32(((const T*)a.in.u)[b * a.ub + ch]) : 0.f;
    float dt = on ? as_f32(((const T*)a.in.delta)[b * a.db + ch]) : 0.f;
    if (on && a.in.dbias) dt += a.in.dbias[ch];
    const float z = on && a.in.gate ? as_f32(((const T*)a.in.gate)[b * a.zb + ch]) : 0.f;
    const float skip = on && a.in.skip ? a.in.skip[ch] : 0.f;
    if (a.softplus) dt = softplus_of<sizeof(T) == 4>(dt);
    const float du = dt * u;
    float y = 0.f, A2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] = A[k] * kLog2e;
    // what log2_rate is for; of all tokens it would cost 2.6% (256 x 5120 x 16)
    if (dt == 0.f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) A2[k] = log2_rate(A[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(fast_exp2(dt * A2[k]), h[k], du * Bv[k]);
        y = fmaf(h[k], Cv[k], y);
    }
    if (quad) {
        const f32x4_any hv = {h[0], h[1], h[2], h[3]};
        __builtin_nontemporal_store(hv, reinterpret_cast<f32x4_any*>(hp));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (on && n0 + k < a.N) hp[k] = h[k];
    }
#pragma unroll
    for (int off = LPC / 2; off >= 1; off >>= 1) y += __shfl_xor(y, off, 64);
    y = fmaf(skip, u, y);
    if (a.in.gate) y *= z * sigmoid_of(z);
    if (on && n0 == 0) Elem<T>::store((T*)a.y + b * a.D + ch, y);
}

template <typename T, int NR, int CW> hipError_t run_fwd(const ChanArgs& a, const ChanShape& s, hipStream_t st) {
    const dim3 blk(256), grid((unsigned)chan_tiles(s, CW), (unsigned)a.nseg, (unsigned)s.Bz);
    if (a.nseg > 1) {
        // the last segment's end state enters nothing
        hipLaunchKernelGGL((k_chan_fwd<T, NR, CW, false>), dim3(grid.x, grid.y - 1, grid.z), blk, 0, st, a);
        const int64_t items = s.Bz * s.D * s.N;
        hipLaunchKernelGGL(k_chan_pass, dim3((unsigned)((items + 255) / 256)), blk, 0, st, a, items);
    }
    hipLaunchKernelGGL((k_chan_fwd<T, NR, CW, true>), grid, blk, 0, st, a);
    return hipGetLastError();
}
template <typename T, int NR>
hipError_t run_fwd_mixed(const ChanArgs& a, const ChanShape& s, int64_t whole, hipStream_t st) {
    const int64_t tiles = chan_tiles(s, 64), flats = s.Bz * tiles;
    hipLaunchKernelGGL((k_chan_fwd_mixed<T, NR>), dim3((unsigned)(whole + 2 * (flats - whole))), dim3(256), 0, st, a,
                       (int)whole, (int)tiles);
    return hipGetLastError();
}
template <typename T> hipError_t run_fwd_t(const ChanArgs& a, const ChanShape& s, const ChanPlan& p, hipStream_t st) {
    if (p.whole > 0) {
        if (s.N <= 8) return run_fwd_mixed<T, 2>(a, s, p.whole, st);
        if (s.N <= 16) return run_fwd_mixed<T, 4>(a, s, p.whole, st);
        if (s.N <= 32) return run_fwd_mixed<T, 8>(a, s, p.whole, st);
        return run_fwd_mixed<T, 16>(a, s, p.whole, st);
    }
    if (p.cw == 32) {
        if (s.N <= 8) return run_fwd<T, 1, 32>(a, s, st);
        if (s.N <= 16) return run_fwd<T, 2, 32>(a, s, st);
        if (s.N <= 32) return run_fwd<T, 4, 32>(a, s, st);
        return run_fwd<T, 8, 32>(a, s, st);
    }
    if (s.N <= 8) return run_fwd<T, 2, 64>(a, s, st);
    if (s.N <= 16) return run_fwd<T, 4, 64>(a, s, st);
    if (s.N <= 32) return run_fwd<T, 8, 64>(a, s, st);
    return run_fwd<T, 16, 64>(a, s, st);
}

template <typename T> hipError_t run_step(const ChanArgs& a, const ChanShape& s, float* state, hipStream_t st) {
    const int lpc = s.N <= 4 ? 1 : s.N <= 8 ? 2 : s.N <= 16 ? 4 : s.N <= 32 ? 8 : 16;
    const int64_t items = s.Bz * s.D * lpc;
    const dim3 grid((unsigned)((items + 255) / 256)), blk(256);
    if (lpc == 1) hipLaunchKernelGGL((k_chan_step<T, 1>), grid, blk, 0, st, a, state, items);
    else if (lpc == 2) hipLaunchKernelGGL((k_chan_step<T, 2>), grid, blk, 0, st, a, state, items);
    else if (lpc == 4) hipLaunchKernelGGL((k_chan_step<T, 4>), grid, blk, 0, st, a, state, items);
    else if (lpc == 8) hipLaunchKernelGGL((k_chan_step<T, 8>), grid, blk, 0, st, a, state, items);
    else hipLaunchKernelGGL((k_chan_step<T, 16>), grid, blk, 0, st, a, state, items);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_chan_fwd(const ChanShape& s, const ChanPlan& p, const ChanIn& in, void* y, float* hfin,
                           float* ws, hipStream_t st)
{
    ChanArgs a = chan_args(s, in);
    a.seg = p.seg; a.nseg = p.nseg;
    a.tpg = (int)(chan_tiles(s, p.cw) / s.G);
    a.y = y; a.hfin = hfin;
    a.S = ws;
    a.sumdt = ws ? ws + s.Bz * p.nseg * s.D * s.N : nullptr;
    return s.bf16 ? run_fwd_t<u16>(a, s, p, st) : run_fwd_t<float>(a, s, p, st);
}

hipError_t launch_chan_step(const ChanShape& s, float* state, const ChanIn& in, void* y, hipStream_t st)
{
    ChanArgs a = chan_args(s, in);
    a.y = y;
    return s.bf16 ? run_step<u16>(a, s, state, st) : run_step<float>(a, s, state, st);
}

}  // namespace ssd
