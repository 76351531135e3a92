// kernels_attn_f32.hip -- linear attention with a decay per head, fp32: the walk of
// attn_walk.hpp in chunks of 32 steps.
//
// Every factor of its products is the sum of three bf16 parts, which hold its 24 bits (their
// rests are exact), and six of the nine products of parts are formed, on
// v_mfma_f32_32x32x16_bf16 (the scores on 16x16x32): the second part is up to 2^-8 of a
// value and the third up to 2^-17, so what the other three leave out is below 2^-24 of a
// product, one rounding.  Six of these take 3/8 of the time of the fp32 instructions for the
// same elements; a forward of 8 x 2048 x 32 heads of 128 x 128 took 595 us with those, 440
// with the parts, and takes 322 with wavefronts of their own for the rows and the scores
// (floor 240: what is left is the state wavefronts' chain, at 40% of the matrix units' time
// and a third of the vector units').  256 wide, a lane holds 128 numbers of the state and
// four wavefronts of it spill, 52 to 64 bytes a lane.  What is infinite, or would round to it in
// bf16, has no such parts and gives NaN.
#include "attn_util.hpp"

namespace ssd {
namespace {

constexpr int kC = 32, kPad = 4;   // rows of x padded by 16 bytes: its columns are read from all banks

// A tile's rows, read to registers at any alignment and length (get), put into LDS later:
// as three planes of bf16 parts of `plane` bytes each, or (SPLIT 0) as they are.
template <int W, int NTH, bool SPLIT> struct StageF {
    static constexpr int PR = W / 4, N = kC * PR / NTH, RS = NTH / PR;
    Piece<float> piece;
    int row0, col;
    u32x4 v[N];
    __device__ __forceinline__ StageF(int tid, int col0, int d) : piece(col0 + tid % PR * 4, d) {
        row0 = tid / PR;
        col = tid % PR * 4;
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
    __device__ __forceinline__ void put(uint32_t tile, int r0, bool whole, const Minus& minus) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int row = row0 + k * RS;
            u32x4 w = v[k];
            if (!whole) {
                w = piece.shifted(w);
                if (row < r0) w = u32x4{0, 0, 0, 0};
            }
            if constexpr (!SPLIT) {
                lds_store4(tile + 4 * (row * (W + kPad) + col), w);
            } else {
                const float f[4] = {__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3])};
                u32x2 part[3];
                parts(f, minus, part);
                const uint32_t at = tile + 2 * tile_at<W / 8>(row, col);
#pragma unroll
                for (int p = 0; p < 3; ++p) lds_store2(at + p * (2 * kC * W), part[p]);
            }
        }
    }
    // four values as bf16 parts
    static __device__ __forceinline__ void parts(const float (&f)[4], const Minus& minus, u32x2 (&part)[3]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            part[0][e] = pack2(f[2 * e], f[2 * e + 1]);
            const float lo = minus.dot(part[0][e], minus.low, f[2 * e]), hi = minus.dot(part[0][e], minus.high, f[2 * e + 1]);
            part[1][e] = pack2(lo, hi);
            part[2][e] = minus.rest(lo, hi, part[1][e]);
        }
    }
};

// product k of the six: the parts of its factors, large products last
__device__ constexpr int kLeft[6] = {0, 2, 1, 0, 1, 0}, kRight[6] = {2, 0, 1, 1, 0, 0};
__device__ __forceinline__ f32x16 product(const bf16x8 (&a)[3], const bf16x8 (&b)[3], f32x16 c) {
#pragma unroll
    for (int k = 0; k < 6; ++k) c = mfma32(a[kLeft[k]], b[kRight[k]], c);
    return c;
}

// KD: contracted elements held; NW state wavefronts, 32 columns each, and as many that bring the
// rows, split them and form the scores.  In two phases of a chunk the state wavefronts
//     multiply S and a                 while the others put the next chunk's rows into LDS,
//     multiply P and x, move S on      while the others form the next chunk's scores
// with two sets of tiles; 256 wide, where LDS holds one, the rows are put there in a phase
// of their own.
template <int KD, int NW> constexpr int f32_sets() { return KD == 256 ? 1 : 2; }
template <int KD, int NW> constexpr int f32_waves() { return NW == 4 || KD == 64 ? 2 : 1; }   // of a SIMD
template <int KD, int NW, bool FULL>
__global__ __launch_bounds__(128 * NW, (f32_waves<KD, NW>())) void k_attn_f32(const AttnArgs A) {
    constexpr int NTH = 64 * NW, NT = KD / 32, CPR = KD / 8, XW = 32 * NW, XR = XW + kPad, SETS = f32_sets<KD, NW>();
    constexpr uint32_t RB = 2 * KD, PLANE = kC * RB, PB = 2 * kC * kC;       // bytes of a row, of a plane of parts
    __shared__ __attribute__((aligned(16))) u16 sA[FULL ? SETS * 3 * kC * KD : 8];
    __shared__ __attribute__((aligned(16))) u16 sK[SETS * 3 * kC * KD];
    __shared__ __attribute__((aligned(16))) float sX[SETS * kC * XR];
    __shared__ __attribute__((aligned(16))) u16 sP[FULL ? SETS * 3 * kC * kC : 8];   // scores, [i][j]
    // powers of gamma: plain, with the scale of the scores, with that of x from the chunk's end
    __shared__ __attribute__((aligned(16))) float sG[kC + 4], sGp[kC], sGw[kC];

    AttnPlace w;
    if (!attn_place(A, XW, &w)) return;
    const AttnPass& P = A.p[w.walk];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, hi = lane >> 5;
    const int rev = P.rev;
    const int chunks = (w.len + kC - 1) / kC;
    const int c0 = w.seg * w.cps, c1 = c0 + w.cps < chunks ? c0 + w.cps : chunks;
    if (!FULL && c0 + w.cps >= chunks) return;   // no segment follows: its end is not asked for
    const Minus minus;
    const Decay g = log2_decay(A.log_decay[w.h]);
    const uint32_t a_at = lds_addr(sA), k_at = lds_addr(sK), x_at = lds_addr(sX), p_at = lds_addr(sP);
    auto first_row = [&](int c) { return c == chunks - 1 ? chunks * kC - w.len : 0; };
    auto set = [&](int c) { return SETS == 2 ? (c - c0) & 1 : 0; };

    if (wave >= NW) {
        // ================= rows and scores =================
        const int at = tid - NTH;
        if (at <= kC) {
            const float p = at <= w.len ? decay_pow(g, at) : 0.f;   // see attn_walk.hpp
            sG[at] = p;
            if (at < kC) {
                sGp[at] = P.scale_p * p;
                sGw[kC - 1 - at] = P.scale_w * p;
            }
        }
        const float* Ab = FULL ? static_cast<const float*>(P.a) + w.b * P.ab + (w.h / P.ag) * P.cd : nullptr;
        const float* Cb = static_cast<const float*>(P.c) + w.b * P.cb + (w.h / P.cg) * P.cd;
        const float* Xb = static_cast<const float*>(P.x) + w.b * P.xb + (w.h / P.xg) * P.xd;
        const bool wide = P.cd == KD, xwide = w.x0 + XW <= P.xd;
        StageF<KD, NTH, true> ga(at, 0, P.cd), gc(at, 0, P.cd);
        StageF<XW, NTH, false> gx(at, w.x0, P.xd);
        auto get = [&](int c) {
            const int r0 = first_row(c);
            const int64_t t0 = c * kC - r0, m0 = rev ? w.len - kC - t0 : t0;
            if constexpr (FULL) ga.get(Ab + m0 * (int64_t)P.ar, P.ar, rev, r0, P.cd);
            gc.get(Cb + m0 * (int64_t)P.cr, P.cr, rev, r0, P.cd);
            gx.get(Xb + m0 * (int64_t)P.xr, P.xr, rev, r0, P.xd);
        };
        auto put = [&](int c) {
            const int r0 = first_row(c), buf = set(c);
            const bool whole = wide && r0 == 0;
            if constexpr (FULL) ga.put(a_at + buf * 3 * PLANE, r0, whole, minus);
            gc.put(k_at + buf * 3 * PLANE, r0, whole, minus);
            gx.put(x_at + buf * 4 * kC * XR, r0, xwide && r0 == 0, minus);
        };
        // scores: 16 x 16 tiles (I, J) = (t / 2, t % 2); register r is row j = 4 (lane / 16) + r,
        // the lane column i = lane % 16
        const int l16 = lane & 15, g4 = lane >> 4;
        auto scores = [&](int t, int buf) {
            const int I = t >> 1, J = t & 1;
            f32x4 s = {0.f, 0.f, 0.f, 0.f};
            if (I >= J) {
                const uint32_t at = fresh(2 * tile_at<CPR>(l16, 8 * g4));   // rows 16 apart have the same swizzle
#pragma unroll
                for (int k = 0; k < KD / 32; ++k) {
                    bf16x8 cf[3], af[3];
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        cf[p] = lds_piece((at ^ (64 * k)) + k_at + buf * 3 * PLANE + J * 16 * RB + p * PLANE);
                        af[p] = lds_piece((at ^ (64 * k)) + a_at + buf * 3 * PLANE + I * 16 * RB + p * PLANE);
                    }
#pragma unroll
                    for (int n = 0; n < 6; ++n)
                        s = mfma16x16x32(cf[kLeft[n]], af[kRight[n]], s);
                }
            }
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int back = 16 * (I - J) + l16 - (4 * g4 + e);
                const float f = sGp[back & (kC - 1)];
                v[e] = back >= 0 ? s[e] * f : 0.f;   // steps ahead are replaced
            }
            u32x2 part[3];
            StageF<KD, NTH, true>::parts(v, minus, part);
            const int i = 16 * I + l16;
            const uint32_t at = p_at + buf * 3 * PB + i * 64 + 16 * ((2 * J + (g4 >> 1)) ^ ((i >> 2) & 3)) + 8 * (g4 & 1);
#pragma unroll
            for (int p = 0; p < 3; ++p) lds_store2(at + p * PB, part[p]);
        };
        auto form = [&](int c) {
            if constexpr (FULL) {
#pragma unroll
                for (int t = 0; t < 4; t += NW) scores(t + wave - NW, set(c));
            }
        };
        if (c0 < c1) get(c0);
        if constexpr (SETS == 2) {
            if (c0 < c1) put(c0);
            if (c0 + 1 < c1) get(c0 + 1);
            sync_lds();
            if (FULL && c0 < c1) form(c0);
            if (FULL) sync_lds();
            for (int c = c0; c < c1; ++c) {
                if (c + 1 < c1) put(c + 1);
                if (c + 2 < c1) get(c + 2);
                sync_lds();
                if constexpr (FULL) {
                    if (c + 1 < c1) form(c + 1);
                    sync_lds();
                }
            }
        } else {
            for (int c = c0; c < c1; ++c) {
                put(c);
                if (c + 1 < c1) get(c + 1);
                sync_lds();
                form(c);
                if (FULL) sync_lds();
                sync_lds();
            }
        }
        return;
    }

    // ================= the state =================
    // columns and state rows in the order of attn_walk.hpp: a lane's registers 8h .. 8h+7
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
        if (P.sc == 1 && P.cd % 8 == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int e = element(nt, r & 8);
                    const f32x4 v = *reinterpret_cast<const f32x4_any*>(col + (e < P.cd ? e + (r & 4) : 0));
#pragma unroll
                    for (int k = 0; k < 4; ++k) S[nt][r + k] = v[k];
                }
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 16; ++r) S[nt][r] = col[(element(nt, r) < P.cd ? element(nt, r) : 0) * P.sc];
        }
        int cd = P.cd;
        asm volatile("" : "+s"(cd));   // or the comparisons above stay in scalar registers till here
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[nt][r] = mine && element(nt, r) < cd ? S[nt][r] : 0.f;
    }
    auto save = [&](float* to, float f) {
        float* col = to + (int64_t)xc * P.sx;
        int cd = P.cd;
        asm volatile("" : "+s"(cd));
        if (P.sc == 1 && cd % 8 == 0) {
            if (mine) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 16; r += 4)
                        if (element(nt, r & 8) < cd)
                            *reinterpret_cast<f32x4_any*>(col + element(nt, r)) =
                                f32x4{f * S[nt][r], f * S[nt][r + 1], f * S[nt][r + 2], f * S[nt][r + 3]};
            }
            return;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (mine && element(nt, r) < cd) col[element(nt, r) * P.sc] = f * S[nt][r];
    };

    const uint32_t row_at0 = 2 * tile_at<CPR>(l32, 8 * hi);
    // see attn_walk.hpp
    const int trow = 8 * hi + ((lane & 15) >> 2), tq = lane & 3;
    const int tcol = (lane & 16) + 4 * (tq == 1 ? 2 : tq == 2 ? 1 : tq);
    const uint32_t tr_at0 = 2 * tile_at<CPR>(trow, tcol), four = 16 * tile_bits<CPR>(4);
    if constexpr (SETS == 2) {
        sync_lds();                // the first tiles
        if (FULL) sync_lds();      // the first scores
    }

    for (int c = c0; c < c1; ++c) {
        const int r0 = first_row(c), lead = rev && c == 0 ? 0 : 1;
        const uint32_t ta = a_at + set(c) * 3 * PLANE, tk = k_at + set(c) * 3 * PLANE, tp = p_at + set(c) * 3 * PB;
        if constexpr (SETS == 1) sync_lds();   // the rows are there
        float xv[2][8];                // column xl of steps 16 s + 8 hi + 0 .. 7
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) xv[s][e] = sX[(set(c) * kC + 16 * s + 8 * hi + e) * XR + xl];

        if constexpr (FULL) {
            f32x16 Y = zero16();
            const uint32_t row_at = fresh(row_at0);
            bf16x8 sf[2][3], af[2][3];
            auto ready = [&](int st) {     // the operands of 16 contracted elements
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = S[st >> 1][8 * (st & 1) + e];
                split3(v, minus, true, sf[st & 1]);
#pragma unroll
                for (int p = 0; p < 3; ++p) af[st & 1][p] = lds_piece((row_at ^ (32 * st)) + ta + p * PLANE);
            };
            ready(0);
#pragma unroll
            for (int st = 0; st < 2 * NT; ++st) {
                if (st + 1 < 2 * NT) ready(st + 1);
                Y = product(sf[st & 1], af[st & 1], Y);
            }
            const int n = l32 - r0 + lead;
            const float f = P.scale_in * sG[n > 0 ? n : 0];
#pragma unroll
            for (int r = 0; r < 16; ++r) Y[r] *= f;
            sync_lds();                // one set of tiles: the scores are there
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                bf16x8 xf[3], pf[3];
                split3(xv[s], minus, true, xf);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    pf[p] = lds_piece(tp + l32 * 64 + 16 * ((2 * s + hi) ^ ((l32 >> 2) & 3)) + p * PB);
                Y = product(xf, pf, Y);
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

        const float through = sG[kC - 1 - r0 + lead];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] *= through;
        const uint32_t tr = fresh(tr_at0);
        bf16x8 cf[2][3], xs[2][3];
        auto column = [&](int i) {         // c^T of steps 16 (i / NT) .., rows 32 (i % NT) ..
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const uint32_t base = tk + 16 * (i / NT) * RB + p * PLANE, b = 64 * (i % NT);
                cf[i & 1][p] = lds_transposed((tr ^ b) + base, (tr ^ (b ^ four)) + (base + 4 * RB));
            }
        };
        auto weigh = [&](int s) {
            float v[8];
            const f32x4* pw = reinterpret_cast<const f32x4*>(&sGw[16 * s + 8 * hi]);
            const f32x4 w0 = pw[0], w1 = pw[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = xv[s][e] * (e < 4 ? w0[e & 3] : w1[e & 3]);
            split3(v, minus, true, xs[s]);
        };
        column(0);
        weigh(0);
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            if (i + 1 < 2 * NT) column(i + 1);
            if (i == 0) weigh(1);
            S[i % NT] = product(cf[i & 1], xs[i / NT], S[i % NT]);
        }
        sync_lds();
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
    if (attn_columns(A.p[0].xd) == 128) k_attn_f32<KD, 4, FULL><<<grid, 512, 0, st>>>(A);
    else k_attn_f32<KD, 2, FULL><<<grid, 256, 0, st>>>(A);
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
