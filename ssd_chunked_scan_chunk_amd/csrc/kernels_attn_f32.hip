// kernels_attn_f32.hip -- linear attention with a decay per head, fp32: the walk of
// kernels_attn.hip in chunks of 32 steps on the fp32 matrix instructions
// (v_mfma_f32_32x32x2_f32 and, for the scores, 16x16x4), which round as fused
// multiply-adds do.
#include "attn_util.hpp"

namespace ssd {
namespace {

constexpr int kC = 32, kPad = 4;   // rows padded by 16 bytes: row reads of 16 bytes fall on different banks

template <int W, int NTH> struct StageF {
    static constexpr int PR = W / 4, N = kC * PR / NTH, RS = NTH / PR;
    Piece<float> piece;
    int row0, lds;
    u32x4 v[N];
    __device__ __forceinline__ StageF(int tid, int col0, int d) : piece(col0 + tid % PR * 4, d) {
        row0 = tid / PR;
        lds = row0 * (W + kPad) + tid % PR * 4;
    }
    __device__ __forceinline__ void get(const float* base, uint32_t rs, int rev, int r0, int d) {
        const bool shortrow = d < 4;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            int r = row0 + k * RS;
            r = r < r0 ? r0 : r;
            const float* row = base + (uint32_t)(rev ? kC - 1 - r : r) * rs;
            if (!shortrow) v[k] = load16(row + piece.at);
            else v[k] = piece.load_short(row, d);
        }
    }
    __device__ __forceinline__ void put(float* tile, int r0, bool whole) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            u32x4 w = v[k];
            if (!whole) {
                w = piece.shifted(w);
                if (row0 + k * RS < r0) w = u32x4{0, 0, 0, 0};
            }
            *reinterpret_cast<u32x4*>(tile + lds + k * RS * (W + kPad)) = w;
        }
    }
};

__device__ __forceinline__ f32x16 mfma2(float a, float b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

template <int KD, int NW, bool FULL>
__global__ __launch_bounds__(64 * NW, KD > 128 ? 1 : 2) void k_attn_f32(const AttnArgs A) {
    constexpr int NTH = 64 * NW, NT = KD / 32, KR = KD + kPad, XW = 32 * NW, XR = XW + kPad, PR = kC + kPad;
    __shared__ __attribute__((aligned(16))) float sA[FULL ? kC * KR : 4];
    __shared__ __attribute__((aligned(16))) float sK[kC * KR];
    __shared__ __attribute__((aligned(16))) float sX[kC * XR];
    __shared__ __attribute__((aligned(16))) float sP[FULL ? kC * PR : 4];     // scores, [i][j]

    AttnPlace w;
    if (!attn_place(A, XW, &w)) return;
    const AttnPass& P = A.p[w.walk];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, hi = lane >> 5;
    const int rev = P.rev;
    const int chunks = (w.len + kC - 1) / kC;
    const int c0 = w.seg * w.cps, c1 = c0 + w.cps < chunks ? c0 + w.cps : chunks;
    if (!FULL && c0 + w.cps >= chunks) return;   // no segment follows: its end is not asked for
    const Decay g = log2_decay(A.log_decay[w.h]);

    // columns and state rows in the order of kernels_attn.hip: a lane's registers 8h .. 8h+7
    // are eight consecutive ones
    const int quad = (l32 >> 2) & 3;
    const int sigma = (l32 & 16) + 4 * (quad == 1 ? 2 : quad == 2 ? 1 : quad) + (l32 & 3);
    const int xl = 32 * wave + sigma, xc = w.x0 + xl;
    const bool mine = xc < P.xd;

    f32x16 S[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) S[nt] = zero16();
    const int64_t SE = (int64_t)P.cd * P.xd;
    auto element = [&](int nt, int r) { return 32 * nt + 16 * (r >> 3) + 8 * hi + (r & 7); };
    const float* from = w.seg == 0 ? (P.first ? P.first + w.state * SE : nullptr)
                      : FULL ? A.slots[w.walk] + (w.slot + w.seg - 1) * SE : nullptr;
    if (from && (w.seg == 0 || c0 < chunks)) {
        // read at a clamped place and dropped: a condition around each read would have it
        // wait for its own value
        const float* col = from + (int64_t)(mine ? xc : 0) * P.sx;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int c = element(nt, r);
                S[nt][r] = col[(c < P.cd ? c : 0) * P.sc];
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) S[nt][r] = mine && element(nt, r) < P.cd ? S[nt][r] : 0.f;
        }
    }
    auto save = [&](float* to, float f) {
        float* col = to + (int64_t)xc * P.sx;
        int cd = P.cd;
        asm volatile("" : "+s"(cd));   // or the comparisons above stay in 128 scalar registers till here
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (mine && element(nt, r) < cd) col[element(nt, r) * P.sc] = f * S[nt][r];
    };

    const float* Ab = FULL ? static_cast<const float*>(P.a) + w.b * P.ab + (w.h / P.ag) * P.cd : nullptr;
    const float* Cb = static_cast<const float*>(P.c) + w.b * P.cb + (w.h / P.cg) * P.cd;
    const float* Xb = static_cast<const float*>(P.x) + w.b * P.xb + (w.h / P.xg) * P.xd;
    const bool wide = P.cd == KD, xwide = w.x0 + XW <= P.xd;

    StageF<KD, NTH> ga(tid, 0, P.cd), gc(tid, 0, P.cd);
    StageF<XW, NTH> gx(tid, w.x0, P.xd);
    auto first_row = [&](int c) { return c == chunks - 1 ? chunks * kC - w.len : 0; };
    auto get = [&](int c) {
        const int r0 = first_row(c);
        const int64_t t0 = c * kC - r0, m0 = rev ? w.len - kC - t0 : t0;
        if constexpr (FULL) ga.get(Ab + m0 * (int64_t)P.ar, P.ar, rev, r0, P.cd);
        gc.get(Cb + m0 * (int64_t)P.cr, P.cr, rev, r0, P.cd);
        gx.get(Xb + m0 * (int64_t)P.xr, P.xr, rev, r0, P.xd);
    };

    // scores: 16 x 16 tiles (I, J) = (t / 2, t % 2); register r is row j = 4 (lane / 16) + r,
    // the lane column i = lane % 16
    const int l16 = lane & 15, g4 = lane >> 4;
    auto scores = [&](int t) {
        const int I = t >> 1, J = t & 1;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        if (I >= J) {
#pragma unroll
            for (int k = 0; k < KD / 16; ++k) {
                const f32x4 cf = *reinterpret_cast<const f32x4*>(&sK[(16 * J + l16) * KR + 16 * k + 4 * g4]);
                const f32x4 af = *reinterpret_cast<const f32x4*>(&sA[(16 * I + l16) * KR + 16 * k + 4 * g4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_16x16x4f32(cf[e], af[e], s, 0, 0, 0);
            }
        }
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int back = 16 * (I - J) + l16 - (4 * g4 + e);
            v[e] = back >= 0 ? s[e] * (P.scale_p * decay_pow(g, back)) : 0.f;   // steps ahead are replaced
        }
        *reinterpret_cast<f32x4*>(&sP[(16 * I + l16) * PR + 16 * J + 4 * g4]) = v;
    };

    // step s of a product over the chunk's rows takes row j = 8 (s / 4) + 4 hi + s % 4
    float wt[16];
#pragma unroll
    for (int s = 0; s < 16; ++s) wt[s] = P.scale_w * decay_pow(g, kC - 1 - (8 * (s >> 2) + 4 * hi + (s & 3)));

    if (c0 < c1) get(c0);
    for (int c = c0; c < c1; ++c) {
        const int r0 = first_row(c), lead = rev && c == 0 ? 0 : 1;
        sync_lds();
        const bool whole = wide && r0 == 0;
        if constexpr (FULL) ga.put(sA, r0, whole);
        gc.put(sK, r0, whole);
        gx.put(sX, r0, xwide && r0 == 0);
        if (c + 1 < c1) get(c + 1);
        sync_lds();

        float xv[16];
#pragma unroll
        for (int s = 0; s < 16; ++s) xv[s] = sX[(8 * (s >> 2) + 4 * hi + (s & 3)) * XR + xl];

        if constexpr (FULL) {
#pragma unroll
            for (int t = 0; t < 4; t += NW) scores(t + wave);
            f32x16 Y = zero16();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 af = *reinterpret_cast<const f32x4*>(&sA[l32 * KR + element(nt, 4 * q)]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) Y = mfma2(S[nt][4 * q + e], af[e], Y);
                }
            const int n = l32 - r0 + lead;
            const float f = P.scale_in * decay_pow(g, n > 0 ? n : 0);
#pragma unroll
            for (int r = 0; r < 16; ++r) Y[r] *= f;
            sync_lds();                // the scores are there
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 pf = *reinterpret_cast<const f32x4*>(&sP[l32 * PR + 8 * q + 4 * hi]);
#pragma unroll
                for (int e = 0; e < 4; ++e) Y = mfma2(xv[4 * q + e], pf[e], Y);
            }
            if (l32 >= r0) {
                const int64_t t = c * kC - r0 + l32, m = rev ? w.len - 1 - t : t;
                float* y = static_cast<float*>(P.y) + ((w.b * A.L + m) * A.H + w.h) * P.xd;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = w.x0 + 32 * wave + 16 * h + 8 * hi;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (x + 4 * q + 4 <= P.xd) {
                            u32x4 v;
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(Y[8 * h + 4 * q + e]);
                            *reinterpret_cast<u32x4_any4*>(y + x + 4 * q) = v;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (x + 4 * q + e < P.xd) y[x + 4 * q + e] = Y[8 * h + 4 * q + e];
                        }
                    }
                }
            }
        }

        const float through = decay_pow(g, kC - 1 - r0 + lead);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] *= through;
#pragma unroll
        for (int s = 0; s < 16; ++s) {
            const float x = xv[s] * wt[s];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                S[nt] = mfma2(sK[(8 * (s >> 2) + 4 * hi + (s & 3)) * KR + 32 * nt + sigma], x, S[nt]);
        }
    }

    if constexpr (FULL) {
        if (P.last && (chunks > 0 ? c0 < chunks && c1 == chunks : w.seg == 0))
            save(P.last + w.state * SE, rev && chunks > 0 ? decay_pow(g, 1) : 1.f);
        const int64_t e0 = c0 * kC > w.len ? c0 * kC : w.len;
        const int64_t e1 = w.seg + 1 == w.nseg ? A.L : (c0 + w.cps) * kC;
        for (int64_t t = e0 + tid / XW; t < e1; t += NTH / XW) {
            const int x = w.x0 + tid % XW;
            if (x < P.xd) static_cast<float*>(P.y)[((w.b * A.L + t) * A.H + w.h) * P.xd + x] = 0.f;
        }
    } else {
        save(A.slots[w.walk] + (w.slot + w.seg) * SE, 1.f);
    }
}

template <bool FULL, int KD>
hipError_t launch(const AttnArgs& A, unsigned grid, hipStream_t st) {
    if (attn_columns(A.p[0].xd) == 128) k_attn_f32<KD, 4, FULL><<<grid, 256, 0, st>>>(A);
    else k_attn_f32<KD, 2, FULL><<<grid, 128, 0, st>>>(A);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_f32(const AttnArgs& A, bool full, hipStream_t st) {
    const unsigned grid = attn_grid(A);
    switch (attn_width(A.p[0].cd)) {
        case 64: return full ? launch<true, 64>(A, grid, st) : launch<false, 64>(A, grid, st);
        case 128: return full ? launch<true, 128>(A, grid, st) : launch<false, 128>(A, grid, st);
        default: return full ? launch<true, 256>(A, grid, st) : launch<false, 256>(A, grid, st);
    }
}

}  // namespace ssd
