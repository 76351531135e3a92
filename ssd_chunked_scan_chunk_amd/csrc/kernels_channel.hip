// kernels_channel.hip -- the scan with one decay per channel and state on
// gfx950: forward and single-token step.
//
//     dt = softplus(delta + bias),  h[n] = e^{dt A[n]} h[n] + dt u B[n],
//     y = (sum_n h[n] C[n] + skip u) silu(gate)
// for every (batch, channel), n < N states.  Every (step, channel, state) costs
// a multiplication, an exponential, another multiplication and two fused
// multiply-adds, none of which the matrix units can take (no operand is shared
// between channels), so the forward is bound by vector issue, not by HBM: it is
// written to spend as little as possible beside those.  The layout is described
// in chan_util.hpp.  The recurrence itself runs sequentially in registers, which
// needs the fewest operations; the sequence is cut into segments only where the
// channels alone leave the GPU idle (a first pass then finds each segment's end
// state from zero and its sum of dt, a scan over segments the states entering
// them; the decay over a segment is e^{A sum dt}).
#include "chan_util.hpp"

namespace ssd {

namespace {

// FULL: outputs from the states entering each segment; otherwise each segment's
// end state from zero (S) and its sums of dt.
template <typename T, int R, int NR, bool FULL>
__global__ __launch_bounds__(256) void k_chan_fwd(ChanArgs a)
{
    constexpr int S = 4 / R, TB = 4 * S, NP = 4 * NR;
    constexpr int NB = (TB * NP + 63) / 64;
    __shared__ float4 s_dt[4][64], s_du[4][64];
    __shared__ float s_B[4][TB * NP], s_C[4][FULL ? TB * NP : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x * 4 + wave;
    if (tile >= a.tiles) return;   // wavefronts share nothing
    const int g = tile / a.tpg, cg = (tile - g * a.tpg) * 16 * R + c * R;   // channel within the group
    const int live = a.per - cg < 0 ? 0 : a.per - cg > R ? R : a.per - cg;
    const int64_t ch = (int64_t)g * a.per + cg, b = blockIdx.z, seg = blockIdx.y;
    const bool wide = a.wide;
    const int64_t ts = seg * a.seg, t1 = ts + a.seg < a.L ? ts + a.seg : a.L;
    const int64_t n = chan_length(a.in.lens, b, a.L), te = n < t1 ? n : t1;

    float A2[R][NR], h[R][NR], bias[R], skip[R], sdt[R] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        bias[r] = a.in.dbias && r < live ? a.in.dbias[ch + r] : 0.f;
        skip[r] = a.in.skip && r < live ? a.in.skip[ch + r] : 0.f;
        const float* h0 = !FULL ? nullptr
                          : seg > 0 ? a.S + ((b * a.nseg + seg) * a.D + ch + r) * a.N
                          : a.in.h0 ? a.in.h0 + (b * a.D + ch + r) * a.N : nullptr;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int k = q * NR + i;
            const bool in = r < live && k < a.N;
            A2[r][i] = in ? a.in.A[(ch + r) * a.N + k] * kLog2e : 0.f;
            h[r][i] = in && h0 ? h0[k] : 0.f;
        }
    }
    const T* up = (const T*)a.in.u + b * a.ub + ch;
    const T* dp = (const T*)a.in.delta + b * a.db + ch;
    const T* zp = a.in.gate ? (const T*)a.in.gate + b * a.zb + ch : nullptr;
    const T* Bp = (const T*)a.in.B + b * a.Bb + (int64_t)g * a.N;
    const T* Cp = (const T*)a.in.C + b * a.Cb + (int64_t)g * a.N;
    T* yp = (T*)a.y + b * a.L * a.D + ch;

    Elems<T, R> ru[S], rd[S], rz[S];
    T rB[NB], rC[NB];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const int64_t s = t + q * S + k;
            const int lv = s < te ? live : 0;
            ru[k] = load_elems<T, R>(up + s * a.ur, lv, wide);
            rd[k] = load_elems<T, R>(dp + s * a.dr, lv, wide);
            if (FULL && zp) rz[k] = load_elems<T, R>(zp + s * a.zr, lv, wide);
        }
#pragma unroll
        for (int e = 0; e < NB; ++e) {
            const int idx = e * 64 + lane, k = idx & (NP - 1);
            const int64_t s = t + idx / NP;
            const bool in = k < a.N && s < te && idx < TB * NP;
            rB[e] = in ? Bp[s * a.Br + k] : T(0);
            if (FULL) rC[e] = in ? Cp[s * a.Cr + k] : T(0);
        }
    };

    fetch(ts);
    for (int64_t t = ts; t < te; t += TB) {
        // this row's unit: dt and dt u, once per (step, channel)
        float u[S][R], gz[S][R], d4[4], w4[4];
#pragma unroll
        for (int k = 0; k < S; ++k)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float x = as_f32(rd[k].v[r]) + bias[r];
                float dt = a.softplus ? softplus_of(x) : x;
                dt = t + q * S + k < te ? dt : 0.f;   // a step past the end changes nothing
                u[k][r] = as_f32(ru[k].v[r]);
                d4[k * R + r] = dt;
                w4[k * R + r] = dt * u[k][r];
                sdt[r] += dt;
                if (FULL && zp) {
                    const float z = as_f32(rz[k].v[r]);
                    gz[k][r] = z * sigmoid_of(z);
                }
            }
        wave_lds_fence();
        s_dt[wave][q * 16 + c] = make_float4(d4[0], d4[1], d4[2], d4[3]);
        s_du[wave][q * 16 + c] = make_float4(w4[0], w4[1], w4[2], w4[3]);
#pragma unroll
        for (int e = 0; e < NB; ++e)
            if (TB * NP >= 64 || lane < TB * NP) {
                s_B[wave][e * 64 + lane] = as_f32(rB[e]);
                if (FULL) s_C[wave][e * 64 + lane] = as_f32(rC[e]);
            }
        wave_lds_fence();
        if (t + TB < te) fetch(t + TB);

        float v[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 dv = s_dt[wave][j * 16 + c], wv = s_du[wave][j * 16 + c];
            const float dd[4] = {dv.x, dv.y, dv.z, dv.w}, ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int k = 0; k < S; ++k) {
                float Bv[NR], Cv[NR];
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    Bv[i] = s_B[wave][(j * S + k) * NP + q * NR + i];
                    if (FULL) Cv[i] = s_C[wave][(j * S + k) * NP + q * NR + i];
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        const float e = fast_exp2(dd[k * R + r] * A2[r][i]);
                        h[r][i] = fmaf(e, h[r][i], ww[k * R + r] * Bv[i]);
                        if (FULL) s = fmaf(h[r][i], Cv[i], s);
                    }
                    v[j][k * R + r] = s;
                }
            }
        }
        if constexpr (FULL) {
#pragma unroll
            for (int k = 0; k < S; ++k) {
                float o[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int m = k * R + r;
                    o[r] = fmaf(skip[r], u[k][r], sum_to_rows(v[0][m], v[1][m], v[2][m], v[3][m]));
                    if (zp) o[r] *= gz[k][r];
                }
                const int64_t s = t + q * S + k;
                if (s < te) store_elems<T, R>(yp + s * a.D, o, live, wide);
            }
        }
    }

    if constexpr (FULL) {
        const float zero[R] = {};
        for (int64_t s = (te > ts ? te : ts) + q; s < t1; s += 4) store_elems<T, R>(yp + s * a.D, zero, live, wide);
    }
    float* out = FULL ? (seg == a.nseg - 1 ? a.hfin : nullptr) : a.S;
    if (out) {
        const int64_t row = FULL ? b : b * a.nseg + seg + 1;   // slot s + 1: what enters the next segment
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (r < live && q * NR + i < a.N) out[(row * a.D + ch + r) * a.N + q * NR + i] = h[r][i];
            if (!FULL) {
                const float sum = sum_rows(sdt[r]);
                if (r < live && q == 0) a.sumdt[row * a.D + ch + r] = sum;
            }
        }
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
    const float A2 = a.in.A[dn] * kLog2e;
    float h = a.in.h0 ? a.in.h0[i] : 0.f;
    float* S = a.S + b * a.nseg * DN + dn;
    const float* sd = a.sumdt + b * a.nseg * a.D + ch;
    for (int64_t s = 1; s < a.nseg; ++s) {
        h = fmaf(fast_exp2(A2 * sd[s * a.D]), h, S[s * DN]);
        S[s * DN] = h;
    }
}

// Single token: LPC lanes per channel, four states each.
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
    const bool quad = on && a.wide && n0 < a.N;   // N a multiple of 4, 16-byte rows
    if (quad) {
        const f32x4 hv = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(hp));
        const float4 av = *reinterpret_cast<const float4*>(Ap);
        const Elems<T, 4> bv = load_elems<T, 4>(Bp, 4, true), cv = load_elems<T, 4>(Cp, 4, true);
        A[0] = av.x; A[1] = av.y; A[2] = av.z; A[3] = av.w;
#pragma unroll
        for (int k = 0; k < 4; ++k) { h[k] = hv[k]; Bv[k] = as_f32(bv.v[k]); Cv[k] = as_f32(cv.v[k]); }
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
    if (a.softplus) dt = softplus_of(dt);
    const float du = dt * u;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(fast_exp2(dt * (A[k] * kLog2e)), h[k], du * Bv[k]);
        y = fmaf(h[k], Cv[k], y);
    }
    if (quad) {
        const f32x4 hv = {h[0], h[1], h[2], h[3]};
        __builtin_nontemporal_store(hv, reinterpret_cast<f32x4*>(hp));
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

ChanArgs args_of(const ChanShape& s, const ChanIn& in, int R) {
    ChanArgs a = {};
    a.in = in;
    a.L = s.L; a.D = s.D; a.N = (int)s.N;
    a.ub = s.ub; a.ur = s.ur; a.db = s.db; a.dr = s.dr; a.zb = s.zb; a.zr = s.zr;
    a.Bb = s.Bb; a.Br = s.Br; a.Cb = s.Cb; a.Cr = s.Cr;
    a.per = (int)(s.D / s.G);
    a.tiles = (int)chan_tiles(s, R);
    a.tpg = (int)(a.tiles / s.G);
    a.softplus = s.softplus;
    return a;
}

bool on16(const void* p, int64_t es, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (es * n) == 0; }

template <typename T, int R, int NR> hipError_t run_fwd(const ChanArgs& a, const ChanShape& s, hipStream_t st) {
    const dim3 blk(256), grid((unsigned)((a.tiles + 3) / 4), (unsigned)a.nseg, (unsigned)s.Bz);
    if (a.nseg > 1) {
        // the last segment's end state enters nothing
        hipLaunchKernelGGL((k_chan_fwd<T, R, NR, false>), dim3(grid.x, grid.y - 1, grid.z), blk, 0, st, a);
        const int64_t items = s.Bz * s.D * s.N;
        hipLaunchKernelGGL(k_chan_pass, dim3((unsigned)((items + 255) / 256)), blk, 0, st, a, items);
    }
    hipLaunchKernelGGL((k_chan_fwd<T, R, NR, true>), grid, blk, 0, st, a);
    return hipGetLastError();
}
template <typename T, int R> hipError_t run_fwd_n(const ChanArgs& a, const ChanShape& s, hipStream_t st) {
    if (s.N <= 4) return run_fwd<T, R, 1>(a, s, st);
    if (s.N <= 8) return run_fwd<T, R, 2>(a, s, st);
    if (s.N <= 16) return run_fwd<T, R, 4>(a, s, st);
    if (s.N <= 32) return run_fwd<T, R, 8>(a, s, st);
    return run_fwd<T, R, 16>(a, s, st);
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
    ChanArgs a = args_of(s, in, p.R);
    a.seg = p.seg; a.nseg = p.nseg;
    a.y = y; a.hfin = hfin;
    a.S = ws;
    a.sumdt = ws ? ws + s.Bz * p.nseg * s.D * s.N : nullptr;
    const int64_t es = s.bf16 ? 2 : 4;
    a.wide = a.per % 4 == 0 && on16(in.u, es, 4) && on16(in.delta, es, 4) && on16(in.gate, es, 4) && on16(y, es, 4) &&
             (s.ub | s.ur | s.db | s.dr) % 4 == 0 && (!in.gate || (s.zb | s.zr) % 4 == 0);
    if (s.bf16) return p.R == 4 ? run_fwd_n<u16, 4>(a, s, st) : run_fwd_n<u16, 1>(a, s, st);
    return p.R == 4 ? run_fwd_n<float, 4>(a, s, st) : run_fwd_n<float, 1>(a, s, st);
}

hipError_t launch_chan_step(const ChanShape& s, float* state, const ChanIn& in, void* y, hipStream_t st)
{
    ChanArgs a = args_of(s, in, 1);
    a.y = y;
    const int64_t es = s.bf16 ? 2 : 4;
    a.wide = s.N % 4 == 0 && on16(state, 4, 4) && on16(in.A, 4, 4) && on16(in.B, es, 4) && on16(in.C, es, 4) &&
             (s.Bb | s.Cb) % 4 == 0;
    return s.bf16 ? run_step<u16>(a, s, state, st) : run_step<float>(a, s, state, st);
}

}  // namespace ssd
