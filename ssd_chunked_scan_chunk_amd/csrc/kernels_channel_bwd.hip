// kernels_channel_bwd.hip -- gradients of the scan with one decay per channel
// and state (kernels_channel.hip) on gfx950.
//
// With e = e^{dt A}, d = dy silu(gate) and the adjoint g[t] of h[t],
//     g[t] = d[t] C[t] + e[t+1] g[t+1],       m[t] = e[t] g[t] h[t-1],
//     dB = sum_c g dt u,  dC = sum_c h d,  dA = sum_t m dt,
//     du = dt sum_n g B + skip d,  d(dt) = u sum_n g B + sum_n m A,
//     dgate = dy (sum_n h C + skip u) silu'(gate),
// and ddelta = d(dt) softplus'(delta + bias).  The states are not kept by the
// forward: a first pass writes them at every eighth step (a quarter of the
// inputs' own bytes per state), and the main pass walks the batches of eight steps
// backwards, runs each forward again with its states and decays in registers and
// then takes the eight steps in reverse, the adjoint staying in registers
// throughout.  About 31 vector instructions per (step, channel, state), nine of them in
// the first pass, against some 45 bytes per (step, channel) in and out: the main pass is
// bound by vector issue (4 x 2048 x 5120 x 16: 450 us, its vector units active 95% of the
// time), the first by that and HBM at once (178 us, always active; the states it
// writes are half of its 726 MB, 4.1 TB/s).
//
// The layout is the forward's: a workgroup owns CW channels of a group, a thread
// NR of a channel's states; dt, dt u and d are formed once per (step, channel) and
// the sums over states finished through LDS.  The sums over channels of dB and
// dC take the CW lanes of a wavefront together, halving the number of values a
// lane holds with the number of lanes that hold parts of one; each workgroup
// writes its sums, and a last kernel adds the workgroups' in a fixed order.
// Few channels: the sequence is cut into segments, whose end states and adjoints
// from zero the first pass also finds (the adjoint in forward order, weighted by
// the decay since the segment's start).
#include <type_traits>

#include "chan_util.hpp"

namespace ssd {

namespace {

template <int V> using Int = std::integral_constant<int, V>;

constexpr int TB = 8;   // steps of a batch
constexpr int RB = 2;   // of these, taken in reverse together

struct BwdArgs {
    ChanArgs f;
    const void* dy;
    const float* dh;              // dfinal_state
    void *du, *ddelta, *dgate;
    float* dh0;                   // dinitial_state
    // workspace: states at the start of every batch [b][batch][tile][thread][NR]
    // and, with several segments, the sums of dt before them [b][batch][tile][CW]
    float *ck, *cdt;
    // per segment [b][seg][tile][thread][NR]: state and adjoint from zero, if linked
    // then those that enter it; its sum of dt [b][seg][tile][CW]
    float *hs, *gs, *sumdt;
    float* pbc;                   // [b][t][tile][B, C][NP]: sums over a workgroup's channels
    float *pA, *pskip, *pbias;    // [b][seg][channel]([state])
    int tiles, nb;                // workgroups along the channels, batches of a segment
    bool linked;                  // k_chan_link runs
};

// Up to this many segments every workgroup joins them by itself, above it a kernel of
// its own does it once (whole calls in us, joined by the workgroups and by the kernel: 4 x
// 2048 x 5120 x 16, eight segments, 646 and 647; 3 x 301 x 770 x 12, 19, 37.5 and 38.1;
// 1 x 2048 x 1536 x 16, 32, 70 and 72; 1 x 4096 x 256 x 16, 256, 113 and 80).
constexpr int kJoinMost = 24;

// A wavefront's reduction of NV values over W neighbouring lanes (64 or 32): lane l
// is left with values index(l) .. of sum over the lanes.  Each level pairs lanes,
// which hand over one half of their values each.  Levels in the order of their cost
// per pair of values: 8 and 4 lanes apart two instructions (an addition with the
// partner by DPP for the one value in all lanes, for the other in those that keep it),
// 32 and 16 apart an exchange, which takes two issue slots, and an addition, then
// 2 and 1 apart, inside the quads that masks do not divide, two selections and an
// addition.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
// d + (d of the partner) in the lanes whose bit D is clear, s + (s of the partner) in
// the others.  A DPP operand may not be read within two slots of its write, which the
// compiler sees to around its own instructions only, hence the s_nop on both sides.
#define SSD_ADD_8(d, s)                                                      \
    "v_add_f32_dpp " d ", " d ", " d " row_ror:8 row_mask:0xf bank_mask:0x3\n\t" \
    "v_add_f32_dpp " d ", " s ", " s " row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
#define SSD_ADD_4(d, s)                                                            \
    "v_add_f32_dpp " d ", " d ", " d " row_half_mirror row_mask:0xf bank_mask:0x5\n\t" \
    "v_add_f32_dpp " d ", " s ", " s " row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
#define SSD_ADD_PAIRS(ADD)                                                                               \
    if constexpr (K % 4 == 0) {                                                                          \
        _Pragma("unroll") for (int j = 0; j < K; j += 4)                                                 \
            asm("s_nop 1\n\t" ADD("%0", "%4") ADD("%1", "%5") ADD("%2", "%6") ADD("%3", "%7") "s_nop 1"  \
                : "+&v"(d[j]), "+&v"(d[j + 1]), "+&v"(d[j + 2]), "+&v"(d[j + 3])                          \
                : "v"(s[j]), "v"(s[j + 1]), "v"(s[j + 2]), "v"(s[j + 3]));                               \
    } else {                                                                                             \
        _Pragma("unroll") for (int j = 0; j < K; ++j)                                                    \
            asm("s_nop 1\n\t" ADD("%0", "%1") "s_nop 1" : "+&v"(d[j]) : "v"(s[j]));                      \
    }
template <int D, int K> __device__ __forceinline__ void add_partners(float* d, const float* s) {
    if constexpr (D == 8) {
        SSD_ADD_PAIRS(SSD_ADD_8)
    } else {
        SSD_ADD_PAIRS(SSD_ADD_4)
    }
}
#undef SSD_ADD_PAIRS
#undef SSD_ADD_4
#undef SSD_ADD_8

template <int NV, int W> struct LaneSum {
    static constexpr int kLeft = NV > W ? NV / W : 1;
    static constexpr int after(int D) { return D == 8 ? 4 : D == 4 ? W / 2 : D == 32 ? 16 : D == 16 ? 2 : D / 2; }
    // first value of lane l; lanes that share one (NV < W) hold the same sum
    __device__ static int index(int l) {
        int at = 0, m = NV;
#pragma unroll
        for (int d = 8; d >= 1; d = after(d))
            if (m > 1) {
                m /= 2;
                if (l & d) at += m;
            }
        return at;
    }
    template <int D> __device__ static float exchanged(float a, float b) {
        const unsigned x = __float_as_uint(a), y = __float_as_uint(b);
        const auto r = D == 32 ? __builtin_amdgcn_permlane32_swap(x, y, false, false)
                               : __builtin_amdgcn_permlane16_swap(x, y, false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    template <int D, int M> __device__ static void level(float (&v)[NV], int l) {
        if constexpr (D >= 1) {
            constexpr int K = M > 1 ? M / 2 : 1;
            if constexpr (M > 1 && (D == 8 || D == 4)) {
                add_partners<D, K>(v, v + K);
            } else {
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const float a = v[j], b = v[M > 1 ? j + K : j];
                    if constexpr (D >= 16) {
                        v[j] = exchanged<D>(a, b);
                    } else if constexpr (M > 1) {
                        const float keep = (l & D) ? b : a, give = (l & D) ? a : b;
                        v[j] = keep + across<D>(give);
                    } else {
                        v[j] = a + across<D>(a);
                    }
                }
            }
            level<after(D), K>(v, l);
        }
    }
    // the partner's value: row rotation by 8, mirror of 8, quad exchanges (each
    // pairs a lane with one of the other half of its group)
    template <int D> __device__ static float across(float v) {
        if constexpr (D == 8) return dpp<0x128>(v);
        else if constexpr (D == 4) return dpp<0x141>(v);
        else if constexpr (D == 2) return dpp<0x4E>(v);
        else return dpp<0xB1>(v);
    }
    __device__ static void run(float (&v)[NV], int l) { level<8, NV>(v, l); }
};

// a lane's NR consecutive floats
template <int NR> __device__ __forceinline__ void load_states(RowIn row, uint32_t& off, float (&v)[NR]) {
    typedef float vec __attribute__((ext_vector_type(NR < 4 ? NR : 4)));
#pragma unroll
    for (int i = 0; i < NR; i += 4) {
        const vec q = load_at<vec>(row + i * 4, off);
#pragma unroll
        for (int k = 0; k < 4 && k < NR; ++k) v[i + k] = q[k];
    }
}
template <int NR> __device__ __forceinline__ void store_states(RowOut row, uint32_t off, const float (&v)[NR]) {
    typedef float vec __attribute__((ext_vector_type(NR < 4 ? NR : 4)));
#pragma unroll
    for (int i = 0; i < NR; i += 4) {
        vec q;
#pragma unroll
        for (int k = 0; k < 4 && k < NR; ++k) q[k] = v[i + k];
        *reinterpret_cast<__attribute__((address_space(1))) vec*>(row + off + i * 4) = q;
    }
}

// The states at the start of every batch.  SEGS: from zero, with the segment's
// adjoint, state and sum of dt; otherwise from the initial state.
// Up to four states in a lane fit five wavefronts per SIMD, a few registers short of
// what the compiler would take (4 x 2048 x 5120 x 16: the whole call 653 us at four, 647
// at five).
template <typename T, int NR, int CW, bool SEGS>
__global__ __launch_bounds__(256, NR <= 4 ? 5 : 2) void k_chan_states(BwdArgs a)
{
    constexpr int ES = sizeof(T), NPART = 256 / CW, NP = NPART * NR;
    constexpr int TP = TB * CW / 256;
    constexpr int NBC = TB * NP * (SEGS ? 2 : 1), NE = (NBC + 255) / 256;
    constexpr bool EXACT = ES == 4;
    const ChanArgs& f = a.f;
    __shared__ float2 s_dt[2][TB][CW];
    __shared__ float s_d[SEGS ? 2 : 1][SEGS ? TB : 1][CW];
    __shared__ __align__(16) float s_bc[2][NBC];   // [B, C][step][state]
    const int tid = threadIdx.x, c = tid & (CW - 1), part = tid / CW, n0 = part * NR;
    const int wave64 = __builtin_amdgcn_readfirstlane(tid >> 6) * 64;
    const int tile = blockIdx.x, g = tile / f.tpg, cg = (tile - g * f.tpg) * CW + c;
    const int cl = cg < f.per ? cg : f.per - 1;   // threads past the group repeat its last channel
    const uint32_t col = (uint32_t)cl * ES;
    const int64_t gch = (int64_t)g * f.per, ch = gch + cl, b = blockIdx.z, seg = blockIdx.y;
    const int64_t ts = seg * f.seg, t1 = ts + f.seg < f.L ? ts + f.seg : f.L;
    const int64_t len = chan_length(f.in.lens, b, f.L);
    const int te = (int)(len < ts ? 0 : (len < t1 ? len : t1) - ts);
    const bool gated = f.in.gate != nullptr;

    float A2[NR], h[NR] = {}, G[NR] = {}, P[NR], sum = 0.f;
    const float bias = f.in.dbias ? f.in.dbias[ch] : 0.f;
    RowIn up = row_in(f.in.u, (b * f.ub + gch) * ES + ts * f.ur);
    RowIn dp = row_in(f.in.delta, (b * f.db + gch) * ES + ts * f.dr);
    RowIn zp = row_in(gated ? f.in.gate : f.in.u, (b * f.zb + gch) * ES + ts * f.zr);
    RowIn Bp = row_in(f.in.B, (b * f.Bb + (int64_t)g * f.N) * ES + ts * f.Br);
    RowIn Cp = row_in(f.in.C, (b * f.Cb + (int64_t)g * f.N) * ES + ts * f.Cr);
    const uint32_t yr = (uint32_t)f.D * ES;
    RowIn gp = row_in(a.dy, ((b * f.L + ts) * f.D + gch) * ES);

    auto in_C = [&](int e) { return e * 256 + wave64 >= TB * NP; };   // else in B
    uint32_t ou[TP], od[TP], oz[TP], og[TP], obc[NE];
    auto offsets = [&](int last) {
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int s = part + k * NPART;
            const uint32_t r = s < last ? s : last;
            ou[k] = r * f.ur + col;
            od[k] = r * f.dr + col;
            oz[k] = r * f.zr + col;
            og[k] = r * yr + col;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int i = e * 256 + tid, s = i / NP & (TB - 1), n = i & (NP - 1);
            const uint32_t r = s < last ? s : last;
            obc[e] = r * (SEGS && in_C(e) ? f.Cr : f.Br) + (uint32_t)(n < f.N ? n : f.N - 1) * ES;
        }
    };
    T ru[2][TP], rd[2][TP], rz[2][TP], rg[2][TP], rbc[2][NE];
    auto fetch = [&](auto slot, int last) {
        constexpr int Q = decltype(slot)::value;
        if (last < TB - 1) offsets(last);
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            ru[Q][k] = load_at<T>(up, ou[k]);
            rd[Q][k] = load_at<T>(dp, od[k]);
            if (SEGS) {
                rz[Q][k] = load_at<T>(zp, oz[k]);
                rg[Q][k] = load_at<T>(gp, og[k]);
            }
        }
#pragma unroll
        for (int e = 0; e < NE; ++e)
            rbc[Q][e] = load_at<T>(SEGS && in_C(e) ? Cp : Bp, obc[e]);
        up += TB * (uint64_t)f.ur;
        dp += TB * (uint64_t)f.dr;
        zp += TB * (uint64_t)f.zr;
        gp += TB * (uint64_t)yr;
        Bp += TB * (uint64_t)f.Br;
        Cp += TB * (uint64_t)f.Cr;
    };
    auto prepare = [&](int t, auto slot) {
        constexpr int Q = decltype(slot)::value;
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int s = part + k * NPART;
            const bool on = t + s < te;
            const float x = as_f32(rd[Q][k]) + bias, sp = softplus_of<EXACT>(x);
            float dt = f.softplus ? sp : x;
            dt = on ? dt : 0.f;
            s_dt[Q][s][c] = make_float2(dt, on ? dt * as_f32(ru[Q][k]) : 0.f);
            if (SEGS) {
                const float z = as_f32(rz[Q][k]), sz = z * sigmoid_of(z);
                const float d = as_f32(rg[Q][k]) * (gated ? sz : 1.f);
                s_d[Q][s][c] = on ? d : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int i = e * 256 + tid;
            const bool in = (i & (NP - 1)) < f.N && t + (i / NP & (TB - 1)) < te;
            if (NBC % 256 == 0 || i < NBC) s_bc[Q][i] = in ? as_f32(rbc[Q][e]) : 0.f;
        }
    };
    int64_t at = (b * f.nseg + seg) * a.nb * a.tiles + tile;   // (batch, tile)
    auto batch = [&](int t, auto slot) {
        constexpr int Q = decltype(slot)::value;
        if (t + 2 * TB < te) fetch(slot, te - 1 - t - 2 * TB);
        store_states<NR>(row_out(a.ck, at * 256 * NR * 4), tid * NR * 4, h);
        if (SEGS && part == 0) a.cdt[at * CW + c] = sum;
        at += a.tiles;
        lds_barrier();
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            const float2 d = s_dt[Q][k][c];
            const float* bc = s_bc[Q] + k * NP + n0;
            if (SEGS) sum += d.x;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float e = fast_exp2(d.x * A2[i]);
                h[i] = fmaf(e, h[i], d.y * bc[i]);
                if constexpr (SEGS) {
                    P[i] *= e;
                    G[i] = fmaf(P[i], s_d[Q][k][c] * bc[TB * NP + i], G[i]);
                }
            }
        }
        if (t + TB < te) prepare(t + TB, Int<Q ^ 1>());
    };
    if (te > 0) {
        offsets(TB - 1);
        fetch(Int<0>(), te - 1);
        if (TB < te) fetch(Int<1>(), te - 1 - TB);
        load_values<NR>(f.in.A + ch * f.N, n0, f.N, A2);
        if (!SEGS && f.in.h0) load_values<NR>(f.in.h0 + (b * f.D + ch) * f.N, n0, f.N, h);
        prepare(0, Int<0>());
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            A2[i] = log2_rate(A2[i]);
            P[i] = 1.f;
        }
        for (int t = 0; t < te; t += 2 * TB) {
            batch(t, Int<0>());
            if (t + TB < te) batch(t + TB, Int<1>());
        }
    }
    if constexpr (SEGS) {
        const int64_t s = (b * f.nseg + seg) * a.tiles + tile;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            a.hs[(s * 256 + tid) * NR + i] = h[i];
            a.gs[(s * 256 + tid) * NR + i] = G[i];
        }
        if (part == 0) a.sumdt[s * CW + c] = sum;
    }
}

// h through `count` segments: their end states from zero S (a thread's NR) and sums of
// dt sd, at steps of ss and ds
template <int NR>
__device__ __forceinline__ void join_segments(const float* S, int64_t ss, const float* sd, int64_t ds, int count,
                                              const float (&A2)[NR], float (&h)[NR]) {
    constexpr int U = NR <= 4 ? 8 : 4;   // in flight
    for (int s = 0; s < count; s += U) {
        float v[U][NR], d[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t q = s + k < count ? s + k : count - 1;
            load_values<NR>(S + q * ss, 0, NR, v[k]);
            d[k] = sd[q * ds];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s + k < count) {
#pragma unroll
                for (int i = 0; i < NR; ++i) h[i] = fmaf(fast_exp2(A2[i] * d[k]), h[i], v[k][i]);
            }
    }
}

// Segments joined: hs[seg] becomes the state that enters it, gs[seg] the adjoint
// that enters it from behind.  One thread per (batch, tile, thread, state).
template <int NR, int CW>
__global__ __launch_bounds__(256) void k_chan_link(BwdArgs a, int64_t items)
{
    const ChanArgs& f = a.f;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items) return;
    const int64_t per_b = (int64_t)a.tiles * 256 * NR, b = i / per_b, k = i - b * per_b;
    const int tile = (int)(k / (256 * NR)), rest = (int)(k - (int64_t)tile * 256 * NR), tid = rest / NR;
    const int c = tid & (CW - 1), n = tid / CW * NR + rest % NR;
    const int g = tile / f.tpg, cg = (tile - g * f.tpg) * CW + c;
    const int64_t ch = (int64_t)g * f.per + (cg < f.per ? cg : f.per - 1), at = (b * f.D + ch) * f.N + n;
    const bool in = n < f.N;
    const int last = in ? 0 : n - f.N + 1;   // states past N read the last one's values
    const float A = f.in.A[ch * f.N + n - last];
    float h = f.in.h0 ? f.in.h0[at - last] : 0.f, gr = a.dh ? a.dh[at - last] : 0.f;
    const float A2 = in ? log2_rate(A) : 0.f;
    h = in ? h : 0.f;
    gr = in ? gr : 0.f;
    float* S = a.hs + b * f.nseg * per_b + k;
    float* G = a.gs + b * f.nseg * per_b + k;
    const int64_t per_s = (int64_t)a.tiles * CW;
    const float* sd = a.sumdt + b * f.nseg * per_s + (int64_t)tile * CW + c;
    constexpr int U = 8;   // segments in flight
    for (int64_t s = 0; s < f.nseg; s += U) {
        float v[U], w[U], d[U], x[U];
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (s + q < f.nseg) {
                const int64_t r = f.nseg - 1 - s - q;
                v[q] = S[(s + q) * per_b]; d[q] = sd[(s + q) * per_s];
                w[q] = G[r * per_b]; x[q] = sd[r * per_s];
            }
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (s + q < f.nseg) {
                S[(s + q) * per_b] = h;
                h = fmaf(fast_exp2(A2 * d[q]), h, v[q]);
                G[(f.nseg - 1 - s - q) * per_b] = gr;
                gr = fmaf(fast_exp2(A2 * x[q]), gr, w[q]);
            }
    }
}

template <typename T, int NR, int CW, bool SEGS>
__global__ __launch_bounds__(256, NR <= 4 ? 3 : 2) void k_chan_bwd(BwdArgs a)
{
    constexpr int ES = sizeof(T), NPART = 256 / CW, NP = NPART * NR;
    constexpr int TP = TB * CW / 256, NBC = TB * NP * 2, NE = (NBC + 255) / 256;
    constexpr bool EXACT = ES == 4;
    const ChanArgs& f = a.f;
    __shared__ float2 s_dt[TB][CW];
    __shared__ float s_d[TB][CW];
    __shared__ __align__(16) float s_bc[NBC];          // [B, C][step][state]
    __shared__ float s_part[3][TB][NPART][CW];         // parts of h C, g B and m A
    const int tid = threadIdx.x, c = tid & (CW - 1), part = tid / CW, n0 = part * NR, lane = tid & 63;
    const int wave64 = __builtin_amdgcn_readfirstlane(tid >> 6) * 64;
    const int tile = blockIdx.x, g = tile / f.tpg, cg = (tile - g * f.tpg) * CW + c;
    const bool live = cg < f.per;
    // threads past the group repeat its last channel, store nothing and add nothing
    // to sums over channels
    const int cl = live ? cg : f.per - 1;
    const uint32_t col = (uint32_t)cl * ES;
    const int64_t gch = (int64_t)g * f.per, ch = gch + cl, b = blockIdx.z, seg = blockIdx.y;
    const int64_t ts = seg * f.seg, t1 = ts + f.seg < f.L ? ts + f.seg : f.L;
    const int64_t len = chan_length(f.in.lens, b, f.L);
    const int te = (int)(len < ts ? 0 : (len < t1 ? len : t1) - ts);
    const bool gated = f.in.gate != nullptr;
    const int nb = (te + TB - 1) / TB;                 // batches of this segment
    // A last batch of fewer steps holds them at its end, behind `idle` ones of dt = 0: what
    // these multiply by 0 for dA is the first step's own e g h, where past the end it would
    // be the state after the last step, which may be infinite and is no part of dA.
    const int idle = nb * TB - te;

    float A2[NR], dA[NR] = {}, carry[NR] = {}, hin[NR] = {};
    const float bias = f.in.dbias ? f.in.dbias[ch] : 0.f, skip = f.in.skip ? f.in.skip[ch] : 0.f;
    const int64_t sat = (((b * f.nseg + seg) * a.tiles + tile) * 256 + tid) * NR;
    const RowIn up = row_in(f.in.u, (b * f.ub + gch) * ES + ts * f.ur);
    const RowIn dp = row_in(f.in.delta, (b * f.db + gch) * ES + ts * f.dr);
    const RowIn zp = row_in(gated ? f.in.gate : f.in.u, (b * f.zb + gch) * ES + ts * f.zr);
    const RowIn Bp = row_in(f.in.B, (b * f.Bb + (int64_t)g * f.N) * ES + ts * f.Br);
    const RowIn Cp = row_in(f.in.C, (b * f.Cb + (int64_t)g * f.N) * ES + ts * f.Cr);
    const uint32_t yr = (uint32_t)f.D * ES;
    const int64_t dense = ((b * f.L + ts) * f.D + gch) * ES;
    const RowIn gp = row_in(a.dy, dense);
    const RowOut dup = row_out(a.du, dense), ddp = row_out(a.ddelta, dense), dzp = row_out(a.dgate, dense);

    // The share of batch j of this thread, as in the forward: the steps part + k
    // NPART of channel c, elements e 256 + tid of B and C.  Idle steps, the first `ahead`
    // (of the last batch of a segment only), repeat the first one's row.
    auto in_C = [&](int e) { return e * 256 + wave64 >= TB * NP; };   // else in B
    uint32_t ou[TP], od[TP], oz[TP], oy[TP], obc[NE], ock = tid * NR * 4, ocdt = c * 4;
    auto offsets = [&](int ahead) {
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int s = part + k * NPART;
            const uint32_t r = s > ahead ? s - ahead : 0;
            ou[k] = r * f.ur + col;
            od[k] = r * f.dr + col;
            oz[k] = r * f.zr + col;
            oy[k] = r * yr + col;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int i = e * 256 + tid, s = i / NP & (TB - 1), n = i & (NP - 1);
            const uint32_t r = s > ahead ? s - ahead : 0;
            obc[e] = r * (in_C(e) ? f.Cr : f.Br) + (uint32_t)(n < f.N ? n : f.N - 1) * ES;
        }
    };
    T ru[TP], rd[TP], rz[TP], rg[TP], rbc[NE];
    float rck[NR], rcdt = 0.f;
    auto fetch = [&](int j) {
        const uint64_t t = (uint64_t)j * TB;
        const RowIn ut = up + t * f.ur, dt = dp + t * f.dr, zt = zp + t * f.zr, gt = gp + t * yr;
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            ru[k] = load_at<T>(ut, ou[k]);
            rd[k] = load_at<T>(dt, od[k]);
            rz[k] = load_at<T>(zt, oz[k]);
            rg[k] = load_at<T>(gt, oy[k]);
        }
#pragma unroll
        for (int e = 0; e < NE; ++e)
            rbc[e] = load_at<T>((in_C(e) ? Cp : Bp) + t * (in_C(e) ? f.Cr : f.Br), obc[e]);
        const int64_t at = ((b * f.nseg + seg) * a.nb + j) * a.tiles + tile;
        load_states<NR>(row_in(a.ck, at * 256 * NR * 4), ock, rck);
        if (SEGS) rcdt = load_at<float>(row_in(a.cdt, at * CW * 4), ocdt);
    };
    // of a pair: u, dt, d, softplus' and dy silu'(gate)
    float u[TP], dtv[TP], d[TP], sx[TP], dz[TP], h[NR], sskip = 0.f, sbias = 0.f;
    auto prepare = [&](int ahead) {
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int s = part + k * NPART;
            const bool on = live && s >= ahead;        // neither an idle step nor a channel past
            const float x = as_f32(rd[k]) + bias;      // the group may add to anything
            const float e = exp_neg_abs<EXACT>(x), r = __builtin_amdgcn_rcpf(1.f + e);
            const float sp = fmaxf(x, 0.f) + log1p_unit(e);
            dtv[k] = on ? (f.softplus ? sp : x) : 0.f;
            sx[k] = f.softplus ? (x >= 0.f ? r : e * r) : 1.f;
            u[k] = as_f32(ru[k]);
            const float z = as_f32(rz[k]), sg = sigmoid_of(z), dy = as_f32(rg[k]);
            dz[k] = dy * (sg * fmaf(z, 1.f - sg, 1.f));
            d[k] = on ? dy * (gated ? z * sg : 1.f) : 0.f;
            s_dt[s][c] = make_float2(dtv[k], on ? dtv[k] * u[k] : 0.f);
            s_d[s][c] = d[k];
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int i = e * 256 + tid;
            const bool in = (i & (NP - 1)) < f.N && (i / NP & (TB - 1)) >= ahead;
            if (NBC % 256 == 0 || i < NBC) s_bc[i] = in ? as_f32(rbc[e]) : 0.f;
        }
        // the state entering the batch
#pragma unroll
        for (int i = 0; i < NR; ++i)
            h[i] = SEGS ? fmaf(fast_exp2(A2[i] * rcdt), hin[i], rck[i]) : rck[i];
    };

    if (nb > 0) {
        offsets(idle);
        fetch(nb - 1);
    }
    load_values<NR>(f.in.A + ch * f.N, n0, f.N, A2);
    if (SEGS && a.linked) {
        load_values<NR>(a.gs + sat, 0, NR, carry);
        load_values<NR>(a.hs + sat, 0, NR, hin);
    } else {
        if (a.dh) load_values<NR>(a.dh + (b * f.D + ch) * f.N, n0, f.N, carry);
        if (SEGS && f.in.h0) load_values<NR>(f.in.h0 + (b * f.D + ch) * f.N, n0, f.N, hin);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) A2[i] = log2_rate(A2[i]);
    if (SEGS && !a.linked) {   // states from the segments before, adjoints from those behind
        const int64_t ss = (int64_t)a.tiles * 256 * NR, ds = (int64_t)a.tiles * CW, nth = f.nseg - 1;
        const int64_t first = b * f.nseg * ss + ((int64_t)tile * 256 + tid) * NR;
        const int64_t dfirst = b * f.nseg * ds + (int64_t)tile * CW + c;
        join_segments<NR>(a.hs + first, ss, a.sumdt + dfirst, ds, (int)seg, A2, hin);
        join_segments<NR>(a.gs + first + nth * ss, -ss, a.sumdt + dfirst + nth * ds, -ds, (int)(nth - seg), A2, carry);
    }
    if (nb > 0) prepare(idle);
    offsets(0);   // of all other batches, and of the outputs
    using Sum = LaneSum<RB * 2 * NR, CW>;
    // the values this lane is left with, vi .. : state (part's n0 +) i of B or C at step k
    const int vi = Sum::index(lane);
    int vk[Sum::kLeft];                // the step of each in its RB
    uint32_t ov[TB / RB][Sum::kLeft];
#pragma unroll
    for (int e = 0; e < Sum::kLeft; ++e) {
        const int m = vi + e, k = m / (2 * NR), which = m / NR & 1, i = m % NR;
        vk[e] = k;
#pragma unroll
        for (int r = 0; r < TB / RB; ++r) ov[r][e] = (uint32_t)((((r * RB + k) * a.tiles * 2 + which) * NP + n0 + i) * 4);
    }
    // what was loaded so far has arrived before the loop counts its own loads
#pragma unroll
    for (int i = 0; i < NR; ++i) asm volatile("" : "+v"(carry[i]), "+v"(hin[i]));
    for (int j = nb - 1, ahead = idle; j >= 0; --j, ahead = 0) {
        const int row0 = j * TB - ahead;   // of the batch's first step, idle or not
        if (j > 0) fetch(j - 1);
        lds_barrier();
        // forward: states and decays of the batch
        float H[TB][NR], E[TB][NR], hfirst[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) hfirst[i] = h[i];
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            const float2 dt = s_dt[k][c];
            const float* bc = s_bc + k * NP + n0;
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                E[k][i] = fast_exp2(dt.x * A2[i]);
                h[i] = fmaf(E[k][i], h[i], dt.y * bc[i]);
                H[k][i] = h[i];
                y = i == 0 ? h[i] * bc[TB * NP + i] : fmaf(h[i], bc[TB * NP + i], y);
            }
            s_part[0][k][part][c] = y;
        }
        // Reverse, RB steps at a time, whose terms of dB and dC are summed over the
        // channels before the next.  The batch's values are read from LDS again (the
        // empty asm keeps the compiler from holding them): kept, they would cost a
        // third of the registers and with them a wavefront per SIMD (876 against
        // 532 us for 4 x 2048 x 5120 x 16 in four segments when both were built).
        const RowOut pbc = row_out(a.pbc, (((b * f.L + ts + row0) * a.tiles + tile) * 2 * NP) * 4);
#pragma unroll
        for (int k0 = TB - RB; k0 >= 0; k0 -= RB) {
            asm volatile("" ::: "memory");
            float v[RB * 2 * NR];
#pragma unroll
            for (int m = RB - 1; m >= 0; --m) {
                const int k = k0 + m;
                const float2 dt = s_dt[k][c];
                const float dk = s_d[k][c];
                const float* bc = s_bc + k * NP + n0;
                float fed = 0.f, ma = 0.f;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const float gr = fmaf(dk, bc[TB * NP + i], carry[i]);
                    fed = i == 0 ? gr * bc[i] : fmaf(gr, bc[i], fed);
                    v[(m * 2) * NR + i] = gr * dt.y;
                    v[(m * 2 + 1) * NR + i] = H[k][i] * dk;
                    carry[i] = gr * E[k][i];
                    const float mh = carry[i] * (k > 0 ? H[k > 0 ? k - 1 : 0][i] : hfirst[i]);
                    dA[i] = fmaf(mh, dt.x, dA[i]);
                    ma = i == 0 ? mh * A2[i] : fmaf(mh, A2[i], ma);
                }
                s_part[1][k][part][c] = fed;
                s_part[2][k][part][c] = ma;
            }
            Sum::run(v, lane);
#pragma unroll
            for (int e = 0; e < Sum::kLeft; ++e) {
                asm volatile("" : "+v"(v[e]));   // the last addition stays ahead of the branch, in one instruction
                // lanes that share a value store it more than once, the same bits
                if (k0 + vk[e] >= ahead) store_at(pbc, ov[k0 / RB][e], v[e], 0.f);
            }
        }
        lds_barrier();
        // this thread's pairs of the batch
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int s = part + k * NPART;
            float y = 0.f, fed = 0.f, ma = 0.f;
#pragma unroll
            for (int q = 0; q < NPART; ++q) {
                y += s_part[0][s][q][c];
                fed += s_part[1][s][q][c];
                ma += s_part[2][s][q][c];
            }
            // A2 = A log2(e)
            const float dd = fmaf(fed, u[k], ma * 0.69314718f) * sx[k];
            if (live && s >= ahead) {
                sskip = fmaf(d[k], u[k], sskip);
                sbias += dd;
                store_at(dup + (int64_t)row0 * yr, oy[k], fmaf(fed, dtv[k], skip * d[k]), T());
                store_at(ddp + (int64_t)row0 * yr, oy[k], dd, T());
                if (gated) store_at(dzp + (int64_t)row0 * yr, oy[k], dz[k] * fmaf(skip, u[k], y), T());
            }
        }
        if (j > 0) prepare(0);
    }

    // the channel once more: kept over the loop, whose registers are full, it is spilled
    int c1 = c;
    asm volatile("" : "+v"(c1));
    const int cl1 = (tile - g * f.tpg) * CW + c1;   // of live threads
    const int64_t row = b * f.nseg + seg, ch1 = gch + cl1;
    uint32_t col1 = (uint32_t)cl1 * ES;
    for (int64_t s = te + part; s < t1 - ts; s += NPART)
        if (live) {
            store_at(dup + s * (uint64_t)yr, col1, 0.f, T());
            store_at(ddp + s * (uint64_t)yr, col1, 0.f, T());
            if (gated) store_at(dzp + s * (uint64_t)yr, col1, 0.f, T());
        }
#pragma unroll
    for (int i = 0; i < NR; ++i)
        if (live && n0 + i < f.N) {
            a.pA[(row * f.D + ch1) * f.N + n0 + i] = dA[i];
            if (a.dh0 && seg == 0) a.dh0[(b * f.D + ch1) * f.N + n0 + i] = carry[i];
        }
    __syncthreads();
    float* sum = &s_part[0][0][0][0];
    sum[tid] = sskip;
    sum[256 + tid] = sbias;
    __syncthreads();
    if (live && part == 0) {
        sskip = sbias = 0.f;
#pragma unroll
        for (int q = 0; q < NPART; ++q) {
            sskip += sum[q * CW + c];
            sbias += sum[256 + q * CW + c];
        }
        if (a.pskip) a.pskip[row * f.D + ch1] = sskip;
        if (a.pbias) a.pbias[row * f.D + ch1] = sbias;
    }
}

// The sums over workgroups, in a fixed order.  The first `bc_blocks` workgroups:
// dB and dC, one thread per (batch, step, group, B or C, state), zeros past a
// sequence's end.  The others: dA, dskip and dbias over the segments of all
// batches, one thread per column.
__device__ __forceinline__ float sum_strided(const float* p, int64_t n, int64_t stride) {
    float s = 0.f;
    int64_t r = 0;
    constexpr int U = 8;   // loads in flight
    for (; r + U <= n; r += U) {
        float v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) v[k] = p[(r + k) * stride];
        s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; r < n; ++r) s += p[r * stride];
    return s;
}
template <typename T>
__global__ __launch_bounds__(256) void k_chan_sums(BwdArgs a, int NP, unsigned bc_blocks, int64_t rows,
                                                   int64_t segs, ChanGrads o)
{
    const ChanArgs& f = a.f;
    if (blockIdx.x < bc_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        const int G = a.tiles / f.tpg, n = (int)(i & (2 * NP - 1)), k = n & (NP - 1);   // [B, C][state]
        const int64_t r = i / (2 * NP), g = r % G, bt = r / G, b = bt / f.L, t = bt - b * f.L;
        if (bt >= rows || k >= f.N) return;
        const float s = t < chan_length(f.in.lens, b, f.L)
                            ? sum_strided(a.pbc + (bt * a.tiles + g * f.tpg) * 2 * NP + n, f.tpg, 2 * NP) : 0.f;
        Elem<T>::store((T*)(n < NP ? o.dB : o.dC) + r * f.N + k, s);
        return;
    }
    int64_t i = (int64_t)(blockIdx.x - bc_blocks) * 256 + threadIdx.x;
    const int64_t nA = f.D * f.N;
    const float* p = a.pA;
    float* out = o.dA;
    int64_t n = nA;
    if (i >= nA) {
        i -= nA;
        n = f.D;
        p = i < f.D ? a.pskip : a.pbias;
        out = i < f.D ? o.dskip : o.ddbias;
        if (i >= f.D) i -= f.D;
        if (i >= f.D) return;
    }
    if (out) out[i] = sum_strided(p + i, segs, n);
}

template <typename T, int NR, int CW>
hipError_t run_bwd(const BwdArgs& a, const ChanShape& s, const ChanGrads& o, hipStream_t st) {
    constexpr int NP = 256 / CW * NR;
    const dim3 blk(256), grid((unsigned)a.tiles, (unsigned)a.f.nseg, (unsigned)s.Bz);
    if (s.L > 0) {
        if (a.f.nseg > 1) {
            hipLaunchKernelGGL((k_chan_states<T, NR, CW, true>), grid, blk, 0, st, a);
            if (a.linked) {
                const int64_t items = s.Bz * a.tiles * 256 * NR;
                hipLaunchKernelGGL((k_chan_link<NR, CW>), dim3((unsigned)((items + 255) / 256)), blk, 0, st, a, items);
            }
        } else {
            hipLaunchKernelGGL((k_chan_states<T, NR, CW, false>), grid, blk, 0, st, a);
        }
    }
    if (a.f.nseg > 1) hipLaunchKernelGGL((k_chan_bwd<T, NR, CW, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_chan_bwd<T, NR, CW, false>), grid, blk, 0, st, a);
    const unsigned bc_blocks = (unsigned)((s.Bz * s.L * s.G * 2 * NP + 255) / 256);
    const unsigned columns = (unsigned)((s.D * (s.N + 2) + 255) / 256);
    hipLaunchKernelGGL(k_chan_sums<T>, dim3(bc_blocks + columns), blk, 0, st, a, NP, bc_blocks, s.Bz * s.L,
                       s.Bz * a.f.nseg, o);
    return hipGetLastError();
}
// The plan's instance alone fits the regions of its workspace.
template <typename T>
hipError_t run_bwd_t(const BwdArgs& a, const ChanShape& s, const ChanBwdPlan& p, const ChanGrads& o, hipStream_t st) {
    if (256 / p.cw * p.nr < s.N) return hipErrorInvalidConfiguration;
    if (p.cw == 64 && p.nr == 2) return run_bwd<T, 2, 64>(a, s, o, st);
    if (p.cw == 64 && p.nr == 4) return run_bwd<T, 4, 64>(a, s, o, st);
    if (p.cw == 32 && p.nr == 4) return run_bwd<T, 4, 32>(a, s, o, st);
    if (p.cw == 32 && p.nr == 8) return run_bwd<T, 8, 32>(a, s, o, st);
    return hipErrorInvalidConfiguration;
}

}  // namespace

hipError_t launch_chan_bwd(const ChanShape& s, const ChanBwdPlan& p, const ChanIn& in, const void* dy,
                           const float* dh, const ChanGrads& o, void* ws, hipStream_t st)
{
    BwdArgs a = {};
    a.f = chan_args(s, in);
    a.f.seg = p.seg; a.f.nseg = p.nseg;
    a.linked = p.nseg > kJoinMost;
    a.tiles = (int)chan_tiles(s, p.cw);
    a.f.tpg = (int)(a.tiles / s.G);
    a.nb = (int)p.nb;
    a.dy = dy; a.dh = dh;
    a.du = o.du; a.ddelta = o.ddelta; a.dgate = o.dgate; a.dh0 = o.dh0;
    auto at = [&](int i) { return reinterpret_cast<float*>(static_cast<char*>(ws) + p.off[i]); };
    a.ck = at(0); a.cdt = at(1); a.hs = at(2); a.gs = at(3); a.sumdt = at(4); a.pbc = at(5); a.pA = at(6);
    a.pskip = o.dskip ? at(7) : nullptr;
    a.pbias = o.ddbias ? at(8) : nullptr;
    return s.bf16 ? run_bwd_t<u16>(a, s, p, o, st) : run_bwd_t<float>(a, s, p, o, st);
}

}  // namespace ssd
