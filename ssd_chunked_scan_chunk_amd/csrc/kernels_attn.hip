// kernels_attn.hip -- linear attention with a decay per head, bf16: one walk over the
// sequences in chunks of 64 steps (AttnPass in attn_launch.hpp has the recurrence).
//
// With gamma the head's decay and S the state before the chunk,
//     y_i = sum_{j<=i} gamma^(i-j) (a_i . c_j) x_j + gamma^(i+1) S a_i
//     S'  = gamma^64 S + sum_j gamma^(63-j) x_j c_j^T
// on v_mfma_f32_32x32x16_bf16.  A workgroup owns a (batch, head), 32 columns x per
// wavefront and a segment of the chunks; its state stays in accumulators.
//
// Precision.  The rows are bf16 and their products exact, but three factors are made
// here and have to be rounded to multiply on: the decayed scores and the state in
// the product with a are split into a high and a low bf16 part (17 bits), so that
// y's error is the rounding of y itself; the decayed x, whose errors stay in the
// states (an fp32 output), into three parts (25 bits).  One part each would put y
// 1.7 roundings off in place of one and the states at 2e-3 in place of 1e-7.
#include "attn_util.hpp"

namespace ssd {
namespace {

constexpr int kC = kAttnChunkBf16;

template <int PR> __device__ __forceinline__ int tile_bits(int r) { return swzbits<(PR > 16 ? 16 : PR)>(r); }
template <int PR> __device__ __forceinline__ int tile_at(int row, int col) {
    return row * (PR * 8) + ((((col >> 3) ^ tile_bits<PR>(row)) << 3) | (col & 7));
}

// A tile of 64 rows on its way from memory to LDS: PR pieces of 16 bytes a row, the
// workgroup's threads side by side.
template <int PR, int NTH> struct Stage {
    static constexpr int N = kC * PR / NTH, RS = NTH / PR;   // pieces of a thread, rows between them
    Piece<u16> piece;
    int row0, lds;
    u32x4 v[N];
    __device__ __forceinline__ Stage(int tid, int col0, int d) : piece(col0 + tid % PR * 8, d) {
        row0 = tid / PR;
        lds = tile_at<PR>(row0, tid % PR * 8);
    }
    // rows r0 .. 63 of the tile; `base` is row 0 (63 against time) and `rs` elements lie
    // between rows.  Rows before r0 are read as r0 and dropped by put().
    __device__ __forceinline__ void get(const u16* base, uint32_t rs, int rev, int r0, int d) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            int r = row0 + k * RS;
            r = r < r0 ? r0 : r;
            v[k] = piece.load(base + (uint32_t)(rev ? kC - 1 - r : r) * rs, d);
        }
    }
    __device__ __forceinline__ void put(u16* tile, int r0, bool whole) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            u32x4 w = v[k];
            if (!whole) {
                w = piece.shifted(w);
                if (row0 + k * RS < r0) w = u32x4{0, 0, 0, 0};
            }
            static_assert(RS % 16 == 0 || 16 % RS == 0, "the swizzle repeats every 16 rows");
            if constexpr (RS % 16 == 0) *reinterpret_cast<u32x4*>(tile + lds + k * RS * PR * 8) = w;
            else *reinterpret_cast<u32x4*>(tile + tile_at<PR>(row0 + k * RS, (threadIdx.x % PR) * 8)) = w;
        }
    }
};

// v (eight bf16) times w, as a sum of three bf16 parts
__device__ __forceinline__ void split3(const bf16x8& v, const float (&w)[8], bf16x8 (&o)[3]) {
    const u32x4 u = as_u32x4(v);
    u32x4 part[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo = w[2 * e] * __uint_as_float(u[e] << 16), hi = w[2 * e + 1] * __uint_as_float(u[e] & 0xffff0000u);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            part[p][e] = pack2(lo, hi);
            lo -= __uint_as_float(part[p][e] << 16);
            hi -= __uint_as_float(part[p][e] & 0xffff0000u);
        }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) o[p] = as_bf16x8(part[p]);
}

// KD: contracted elements held (64, 128 or 256); NW wavefronts.  FULL: y and the last
// state; else the states at the segments' ends.
template <int KD, int NW, bool FULL>
__global__ __launch_bounds__(64 * NW, KD > 128 ? 1 : 2) void k_attn(const AttnArgs A) {
    constexpr int NTH = 64 * NW, NT = KD / 32, CPR = KD / 8, XW = 32 * NW, XPR = XW / 8;
    __shared__ __attribute__((aligned(16))) u16 sA[FULL ? kC * KD : 8];
    __shared__ __attribute__((aligned(16))) u16 sK[kC * KD];
    __shared__ __attribute__((aligned(16))) u16 sX[kC * XW];
    __shared__ __attribute__((aligned(16))) u16 sP[FULL ? 3 : 1][FULL ? 2 * 32 * 32 : 8];   // scores, [i][j], high, low

    AttnPlace w;
    if (!attn_place(A, XW, &w)) return;
    const AttnPass& P = A.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, hi = lane >> 5;
    const int rev = P.rev;
    const int64_t chunks = (w.len + kC - 1) / kC;
    const int64_t c0 = w.seg * A.cps, c1 = c0 + A.cps < chunks ? c0 + A.cps : chunks;
    if (!FULL && c0 + A.cps >= chunks) return;   // no segment follows: its end is not asked for
    const Decay g = log2_decay(A.log_decay[w.h]);

    // Lane l32 of wavefront w holds column x = x0 + 32 w + 16 (l32 / 16) + ..., the column
    // quads of each 16 in the order 0, 2, 1, 3: register r of a 32x32 product's rows is
    // then row 16 (r / 8) + 8 hi + r % 8, eight consecutive columns (or contracted
    // elements) to a half, one 16-byte piece.
    const int quad = (l32 >> 2) & 3;
    const int sigma = (l32 & 16) + 4 * (quad == 1 ? 2 : quad == 2 ? 1 : quad) + (l32 & 3);
    const int xc = w.x0 + 32 * wave + sigma;
    const bool mine = xc < P.xd;

    // ---- the state: register r of S[nt] is element c = 32 nt + 16 (r / 8) + 8 hi + r % 8 ----
    f32x16 S[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) S[nt] = zero16();
    const int64_t SE = (int64_t)P.cd * P.xd;
    auto element = [&](int nt, int r) { return 32 * nt + 16 * (r >> 3) + 8 * hi + (r & 7); };
    const float* from = w.seg == 0 ? (P.first ? P.first + w.state * SE : nullptr)
                      : FULL ? A.slots + (w.state * (A.nseg - 1) + w.seg - 1) * SE : nullptr;
    if (from && (w.seg == 0 || c0 < chunks)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int c = element(nt, r);
                if (mine && c < P.cd) S[nt][r] = from[c * P.sc + xc * P.sx];
            }
    }
    auto save = [&](float* to, float f) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int c = element(nt, r);
                if (mine && c < P.cd) to[c * P.sc + xc * P.sx] = f * S[nt][r];
            }
    };

    const u16* Ab = FULL ? static_cast<const u16*>(P.a) + w.b * P.ab + (w.h / P.ag) * P.cd : nullptr;
    const u16* Cb = static_cast<const u16*>(P.c) + w.b * P.cb + (w.h / P.cg) * P.cd;
    const u16* Xb = static_cast<const u16*>(P.x) + w.b * P.xb + (w.h / P.xg) * P.xd;
    const bool wide = P.cd == KD, xwide = w.x0 + XW <= P.xd;

    Stage<CPR, NTH> ga(tid, 0, P.cd), gc(tid, 0, P.cd);
    Stage<XPR, NTH> gx(tid, w.x0, P.xd);
    // A partial chunk's steps are the last rows of its tile (rows before are zero), so
    // that what follows it by 63 - j steps does so there too.
    auto first_row = [&](int64_t c) { return c == chunks - 1 ? (int)(chunks * kC - w.len) : 0; };
    auto get = [&](int64_t c) {
        const int r0 = first_row(c);
        const int64_t t0 = c * kC - r0, m0 = rev ? w.len - kC - t0 : t0;   // memory row of tile row 0, or 63 against time
        if constexpr (FULL) ga.get(Ab + m0 * (int64_t)P.ar, P.ar, rev, r0, P.cd);
        gc.get(Cb + m0 * (int64_t)P.cr, P.cr, rev, r0, P.cd);
        gx.get(Xb + m0 * (int64_t)P.xr, P.xr, rev, r0, P.xd);
    };

    // scores: wavefronts 0 .. 2 (0 and 1 of two) form tiles (I, J) = (0,0), (1,1), (1,0) of
    // 32 x 32; register r is row j = 8 (r / 4) + 4 hi + r % 4, the lane column i
    auto scores = [&](int t) {
        const int I = t > 0 ? 1 : 0, J = t == 1 ? 1 : 0;
        f32x16 s = zero16();
#pragma unroll
        for (int k = 0; k < KD / 16; ++k) {
            const int col = 16 * k + 8 * hi;
            const bf16x8 cf = as_bf16x8(*reinterpret_cast<const u32x4*>(&sK[tile_at<CPR>(32 * J + l32, col)]));
            const bf16x8 af = as_bf16x8(*reinterpret_cast<const u32x4*>(&sA[tile_at<CPR>(32 * I + l32, col)]));
            s = mfma32(cf, af, s);
        }
        u16* row = &sP[t][l32 * 32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int back = 32 * (I - J) + l32 - (8 * q + 4 * hi + e);
                // steps ahead are replaced, not multiplied by 0
                v[e] = back >= 0 ? s[4 * q + e] * (P.scale_p * decay_pow(g, back)) : 0.f;
            }
            const uint32_t h01 = pack2(v[0], v[1]), h23 = pack2(v[2], v[3]);
            const uint32_t l01 = pack2(v[0] - __uint_as_float(h01 << 16), v[1] - __uint_as_float(h01 & 0xffff0000u));
            const uint32_t l23 = pack2(v[2] - __uint_as_float(h23 << 16), v[3] - __uint_as_float(h23 & 0xffff0000u));
            const int off = 8 * (q ^ ((l32 >> 2) & 3)) + 4 * hi;
            *reinterpret_cast<uint2*>(row + off) = make_uint2(h01, h23);
            *reinterpret_cast<uint2*>(row + 32 * 32 + off) = make_uint2(l01, l23);
        }
    };

    // transposing reads: rows 8 hi + 4 s + trow, four columns from tcol of the sigma order
    const int trow = (lane & 15) >> 2, tq = lane & 3;
    const int tcol = 16 * ((lane >> 4) & 1) + 4 * (tq == 1 ? 2 : tq == 2 ? 1 : tq);
    float g8[8];                       // gamma^(7 - e), with the state's scale
#pragma unroll
    for (int e = 0; e < 8; ++e) g8[e] = P.scale_w * decay_pow(g, 7 - e);

    if (c0 < c1) get(c0);
    for (int64_t c = c0; c < c1; ++c) {
        const int r0 = first_row(c), lead = rev && c == 0 ? 0 : 1;   // against time the given state is the last step's own
        sync_lds();                    // the tiles' readers are done
        const bool whole = wide && r0 == 0;
        if constexpr (FULL) ga.put(sA, r0, whole);
        gc.put(sK, r0, whole);
        gx.put(sX, r0, xwide && r0 == 0);
        if (c + 1 < c1) get(c + 1);
        sync_lds();

        bf16x8 xf[4];                  // x^T: lane = column, k = step 16 s + 8 hi + 0 .. 7
#pragma unroll
        for (int s = 0; s < 4; ++s)
            xf[s] = join8(lds_tr4(&sX[tile_at<XPR>(16 * s + 8 * hi + trow, 32 * wave + tcol)]),
                          lds_tr4(&sX[tile_at<XPR>(16 * s + 8 * hi + 4 + trow, 32 * wave + tcol)]));

        if constexpr (FULL) {
            if constexpr (NW == 4) {
                if (wave < 3) scores(wave);
            } else {
                scores(wave);
                if (wave == 0) scores(2);
            }
            // ---- from the state: y^T, rows the columns x, lane = step i of half I ----
            f32x16 Y[2] = {zero16(), zero16()};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8 sh = acc_half(S[nt], h), sl = acc_half_lo(S[nt], h, sh);
                    const int col = 32 * nt + 16 * h + 8 * hi;
#pragma unroll
                    for (int I = 0; I < 2; ++I) {
                        const bf16x8 af =
                            as_bf16x8(*reinterpret_cast<const u32x4*>(&sA[tile_at<CPR>(32 * I + l32, col)]));
                        Y[I] = mfma32(sh, af, Y[I]);
                        Y[I] = mfma32(sl, af, Y[I]);
                    }
                }
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                const int n = 32 * I + l32 - r0 + lead;
                const float f = P.scale_in * decay_pow(g, n > 0 ? n : 0);
#pragma unroll
                for (int r = 0; r < 16; ++r) Y[I][r] *= f;
            }
            sync_lds();                // the scores are there
            // ---- from inside the chunk ----
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                const int I = t > 0 ? 1 : 0, J = t == 1 ? 1 : 0;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const u16* row = &sP[t][l32 * 32 + 8 * ((2 * s + hi) ^ ((l32 >> 2) & 3))];
                    Y[I] = mfma32(xf[2 * J + s], as_bf16x8(*reinterpret_cast<const u32x4*>(row)), Y[I]);
                    Y[I] = mfma32(xf[2 * J + s], as_bf16x8(*reinterpret_cast<const u32x4*>(row + 32 * 32)), Y[I]);
                }
            }
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                const int i = 32 * I + l32;
                const int64_t t = c * kC - r0 + i, m = rev ? w.len - 1 - t : t;
                if (i < r0) continue;
                const int64_t at = ((w.b * A.L + m) * A.H + w.h) * P.xd;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = w.x0 + 32 * wave + 16 * h + 8 * hi;
                    if (P.y_f32) {
                        float* y = static_cast<float*>(P.y) + at + x;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (x + e < P.xd) y[e] = Y[I][8 * h + e];
                    } else {
                        u16* y = static_cast<u16*>(P.y) + at + x;
                        const u32x4 v = as_u32x4(acc_half(Y[I], h));
                        if (x + 8 <= P.xd) *reinterpret_cast<u32x4_any*>(y) = v;
                        else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (x + e < P.xd) y[e] = (u16)(v[e / 2] >> (16 * (e & 1)));
                        }
                    }
                }
            }
        }

        // ---- the state after the chunk ----
        const float through = decay_pow(g, kC - 1 - r0 + lead);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] *= through;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const float f = decay_pow(g, kC - 8 - (16 * s + 8 * hi));
            float wt[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) wt[e] = f * g8[e];
            bf16x8 xs[3];
            split3(xf[s], wt, xs);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const bf16x8 cf = join8(lds_tr4(&sK[tile_at<CPR>(16 * s + 8 * hi + trow, 32 * nt + tcol)]),
                                        lds_tr4(&sK[tile_at<CPR>(16 * s + 8 * hi + 4 + trow, 32 * nt + tcol)]));
#pragma unroll
                for (int p = 0; p < 3; ++p) S[nt] = mfma32(cf, xs[p], S[nt]);
            }
        }
    }

    if constexpr (FULL) {
        if (P.last && (chunks > 0 ? c0 < chunks && c1 == chunks : w.seg == 0))
            save(P.last + w.state * SE, rev && chunks > 0 ? decay_pow(g, 1) : 1.f);
        // rows behind the sequence's end
        const int64_t e0 = c0 * kC > w.len ? c0 * kC : w.len;
        const int64_t e1 = w.seg + 1 == A.nseg || (c0 + A.cps) * kC > A.L ? A.L : (c0 + A.cps) * kC;
        for (int64_t t = e0 + tid / XW; t < e1; t += NTH / XW) {
            const int x = w.x0 + tid % XW;
            const int64_t at = ((w.b * A.L + t) * A.H + w.h) * P.xd + x;
            if (x < P.xd) {
                if (P.y_f32) static_cast<float*>(P.y)[at] = 0.f;
                else static_cast<u16*>(P.y)[at] = 0;
            }
        }
    } else {
        save(A.slots + (w.state * (A.nseg - 1) + w.seg) * SE, 1.f);
    }
}

template <bool FULL, int KD>
hipError_t launch(const AttnArgs& A, int waves, unsigned grid, hipStream_t st) {
    if (waves == 4) k_attn<KD, 4, FULL><<<grid, 256, 0, st>>>(A);
    else k_attn<KD, 2, FULL><<<grid, 128, 0, st>>>(A);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bf16(const AttnArgs& A, bool full, hipStream_t st) {
    const unsigned grid = (unsigned)((A.items + kXcds - 1) / kXcds * kXcds);
    const int waves = attn_waves(A.p.xd);
    switch (attn_width(A.p.cd)) {
        case 64: return full ? launch<true, 64>(A, waves, grid, st) : launch<false, 64>(A, waves, grid, st);
        case 128: return full ? launch<true, 128>(A, waves, grid, st) : launch<false, 128>(A, waves, grid, st);
        default: return full ? launch<true, 256>(A, waves, grid, st) : launch<false, 256>(A, waves, grid, st);
    }
}

}  // namespace ssd
