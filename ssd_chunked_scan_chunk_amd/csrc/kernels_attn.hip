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
#include <type_traits>

#include "attn_util.hpp"

namespace ssd {
namespace {

constexpr int kC = kAttnChunkBf16;

template <int PR> __device__ __forceinline__ int tile_bits(int r) { return swzbits<(PR > 16 ? 16 : PR)>(r); }
template <int PR> __device__ __forceinline__ int tile_at(int row, int col) {
    return row * (PR * 8) + ((((col >> 3) ^ tile_bits<PR>(row)) << 3) | (col & 7));
}

// A tile of 64 rows with PR pieces of 16 bytes each, brought from memory to LDS by the
// workgroup's NW wavefronts.  Its first row is memory row 0 of `base` (63 against time), rows are
// rs elements apart; rows before r0 are read as r0.
//
// FAST: copied to LDS as it comes (rows and strides of whole aligned pieces), the tile's
// swizzle made by the order in which the lanes take a row's pieces.  Pieces past a
// row's end are not copied: the tile was cleared once.
template <int PR, int NW> struct Copy {
    static constexpr int N = PR / NW, RS = NW * 64 / PR;   // copies of a wavefront, rows between them
    int row0;
    uint32_t lds0;
    __device__ __forceinline__ Copy(int wave, int lane) {
        row0 = wave * (64 / PR) + lane / PR;
        lds0 = (uint32_t)wave * 1024;
    }
    __device__ __forceinline__ void operator()(const u16* base, uint32_t rs, int rev, int r0, int col0, int d, u16* tile,
                                               int lane) const {
        const uintptr_t at = reinterpret_cast<uintptr_t>(base);   // the same in all lanes, into scalar registers
        const void* from = reinterpret_cast<const void*>((uintptr_t)uniform((uint32_t)(at >> 32)) << 32 | uniform((uint32_t)at));
#pragma unroll
        for (int k = 0; k < N; ++k) {
            int r = row0 + k * RS;
            const int col = col0 + ((lane % PR) ^ tile_bits<PR>(r)) * 8;
            r = r < r0 ? r0 : r;
            const uint32_t off = __umul24((uint32_t)(rev ? kC - 1 - r : r), 2 * rs) + 2 * col;
            if (col < d) dma16(from, off, lds_addr(tile) + lds0 + (uint32_t)k * NW * 1024);
        }
    }
};

// Otherwise: read to registers at any alignment and length, put into the tile later.
template <int PR, int NW> struct Stage {
    static constexpr int NTH = 64 * NW, N = kC * PR / NTH, RS = NTH / PR;   // pieces of a thread, rows between them
    Piece<u16> piece;
    int row0, col;
    u32x4 v[N];
    __device__ __forceinline__ Stage(int tid, int col0, int d) : piece(col0 + tid % PR * 8, d) {
        row0 = tid / PR;
        col = tid % PR * 8;
    }
    __device__ __forceinline__ void get(const u16* base, uint32_t rs, int rev, int r0, int d) {
        const bool shortrow = d < 8;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            int r = row0 + k * RS;
            r = r < r0 ? r0 : r;
            const u16* row = base + (uint32_t)(rev ? kC - 1 - r : r) * rs;
            if (!shortrow) v[k] = load16(row + piece.at);
            else v[k] = piece.load_short(row, d);
        }
    }
    __device__ __forceinline__ void put(u16* tile, int r0) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int r = row0 + k * RS;
            const u32x4 w = r < r0 ? u32x4{0, 0, 0, 0} : piece.shifted(v[k]);
            *reinterpret_cast<u32x4*>(tile + tile_at<PR>(r, col)) = w;
        }
    }
};
struct Nothing {
    __device__ __forceinline__ Nothing(int, int, int) {}
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
// state; else the states at the segments' ends.  FAST: see Copy.
//
// A chunk's a and x are free once its scores are formed and their products with the
// state made, so the next chunk's are copied there then, behind the second half of the
// chunk's work; c is needed to its end and has two tiles.  At 128 x 128 that is 79 KB: two
// workgroups to a CU, one's matrix work behind the other's barriers.
template <int KD, int NW, bool FULL, bool FAST>
__global__ __launch_bounds__(64 * NW, KD > 128 ? 1 : 2) void k_attn(const AttnArgs A) {
    constexpr int NT = KD / 32, CPR = KD / 8, XW = 32 * NW, XPR = XW / 8;
    constexpr int KB = FAST ? 2 : 1, XB = FAST && !FULL ? 2 : 1;
    __shared__ __attribute__((aligned(16))) u16 sA[FULL ? kC * KD : 8];
    __shared__ __attribute__((aligned(16))) u16 sK[KB][kC * KD];
    __shared__ __attribute__((aligned(16))) u16 sX[XB][kC * XW];
    __shared__ __attribute__((aligned(16))) u16 sP[FULL ? 3 : 1][FULL ? 2 * 32 * 32 : 8];   // scores, [i][j], high, low
    // powers of gamma: plain, with the scale of the scores (32 zeros ahead), with that of x
    __shared__ __attribute__((aligned(16))) float sG[kC + 4], sGp[32 + kC], sGw[kC];

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
    if (tid <= kC) {
        const float p = decay_pow(g, tid);
        sG[tid] = p;
        if (tid < kC) {
            sGp[32 + tid] = P.scale_p * p;
            sGw[tid] = P.scale_w * p;
        }
        if (tid < 32) sGp[tid] = 0.f;
    }

    const u16* Ab = FULL ? static_cast<const u16*>(P.a) + w.b * P.ab + (w.h / P.ag) * P.cd : nullptr;
    const u16* Cb = static_cast<const u16*>(P.c) + w.b * P.cb + (w.h / P.cg) * P.cd;
    const u16* Xb = static_cast<const u16*>(P.x) + w.b * P.xb + (w.h / P.xg) * P.xd;
    const Copy<CPR, NW> copy_c(wave, lane);
    const Copy<XPR, NW> copy_x(wave, lane);
    using StageC = typename std::conditional<FAST, Nothing, Stage<CPR, NW>>::type;
    using StageX = typename std::conditional<FAST, Nothing, Stage<XPR, NW>>::type;
    StageC ga(tid, 0, P.cd), gc(tid, 0, P.cd);
    StageX gx(tid, w.x0, P.xd);
    // A partial chunk's steps are the last rows of its tile (rows of x before are zero), so
    // that what follows it by 63 - j steps does so there too.
    auto first_row = [&](int64_t c) { return c == chunks - 1 ? (int)(chunks * kC - w.len) : 0; };
    auto memory_row = [&](int64_t c, int r0) {      // of tile row 0, or 63 against time
        const int64_t t0 = c * kC - r0;
        return rev ? w.len - kC - t0 : t0;
    };
    auto fetch_c = [&](int64_t c, int buf) {
        const int r0 = first_row(c);
        const u16* base = Cb + memory_row(c, r0) * (int64_t)P.cr;
        if constexpr (FAST) copy_c(base, P.cr, rev, r0, 0, P.cd, sK[buf], lane);
        else gc.get(base, P.cr, rev, r0, P.cd);
    };
    auto fetch_ax = [&](int64_t c, int buf) {
        const int r0 = first_row(c);
        const int64_t m = memory_row(c, r0);
        if constexpr (FAST) {
            if constexpr (FULL) copy_c(Ab + m * P.ar, P.ar, rev, r0, 0, P.cd, sA, lane);
            copy_x(Xb + m * P.xr, P.xr, rev, r0, w.x0, P.xd, sX[buf], lane);
        } else {
            if constexpr (FULL) ga.get(Ab + m * P.ar, P.ar, rev, r0, P.cd);
            gx.get(Xb + m * P.xr, P.xr, rev, r0, P.xd);
        }
    };
    if constexpr (FAST) {
        if (P.cd < KD || w.x0 + XW > P.xd) {
            const u32x4 z = {0, 0, 0, 0};
            for (int i = tid * 8; i < kC * KD; i += 512 * NW) {
                if constexpr (FULL) *reinterpret_cast<u32x4*>(&sA[i]) = z;
                *reinterpret_cast<u32x4*>(&sK[0][i]) = z;
                *reinterpret_cast<u32x4*>(&sK[KB - 1][i]) = z;
            }
            for (int i = tid * 8; i < kC * XW; i += 512 * NW) {
                *reinterpret_cast<u32x4*>(&sX[0][i]) = z;
                *reinterpret_cast<u32x4*>(&sX[XB - 1][i]) = z;
            }
            sync_lds();
        }
    }
    if (c0 < c1) {
        fetch_ax(c0, 0);
        fetch_c(c0, 0);
    }

    // Lane l32 of a wavefront holds column x = x0 + 32 wave + sigma: the column quads of
    // each 16 come in the order 0, 2, 1, 3, so that register r of a 32x32 product's rows
    // is row 16 (r / 8) + 8 hi + r % 8, eight consecutive columns (or contracted elements)
    // to a half, one 16-byte piece.
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

    // scores: wavefronts 0 .. 2 (0 and 1 of two) form tiles (I, J) = (0,0), (1,1), (1,0) of
    // 32 x 32; register r is row j = 8 (r / 4) + 4 hi + r % 4, the lane column i
    auto scores = [&](int t, const u16* tk) {
        const int I = t > 0 ? 1 : 0, J = t == 1 ? 1 : 0;
        f32x16 s = zero16();
#pragma unroll
        for (int k = 0; k < KD / 16; ++k) {
            const int col = 16 * k + 8 * hi;
            const bf16x8 cf = as_bf16x8(*reinterpret_cast<const u32x4*>(&tk[tile_at<CPR>(32 * J + l32, col)]));
            const bf16x8 af = as_bf16x8(*reinterpret_cast<const u32x4*>(&sA[tile_at<CPR>(32 * I + l32, col)]));
            s = mfma32(cf, af, s);
        }
        u16* row = &sP[t][l32 * 32];
        const float* pw = &sGp[32 + 32 * (I - J) + l32 - 4 * hi];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int back = 32 * (I - J) + l32 - 4 * hi - (8 * q + e);
                // steps ahead are replaced, not multiplied by 0
                v[e] = back >= 0 ? s[4 * q + e] * pw[-(8 * q + e)] : 0.f;
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

    for (int64_t c = c0; c < c1; ++c) {
        const int buf = FAST ? (int)((c - c0) & 1) : 0, xb = XB == 2 ? buf : 0;
        const int r0 = first_row(c), lead = rev && c == 0 ? 0 : 1;   // against time the given state is the last step's own
        u16* tk = sK[buf];
        u16* tx = sX[xb];
        if constexpr (FAST) {
            vm_wait_all();             // this wavefront's copies have landed ...
            sync_lds();                // ... and the others'; the scores and the older c are free
            if (r0 > 0) {
                for (int i = tid; i < r0 * XPR; i += 64 * NW) *reinterpret_cast<u32x4*>(&tx[i * 8]) = u32x4{0, 0, 0, 0};
                sync_lds();
            }
            if (c + 1 < c1) {
                fetch_c(c + 1, buf ^ 1);
                if constexpr (!FULL) fetch_ax(c + 1, buf ^ 1);
            }
        } else {
            sync_lds();                // the tiles' readers are done
            if constexpr (FULL) ga.put(sA, r0);
            gc.put(tk, r0);
            gx.put(tx, r0);
            if (c + 1 < c1) {
                fetch_ax(c + 1, 0);
                fetch_c(c + 1, 0);
            }
            sync_lds();
        }

        bf16x8 xf[4];                  // x^T: lane = column, k = step 16 s + 8 hi + 0 .. 7
#pragma unroll
        for (int s = 0; s < 4; ++s)
            xf[s] = join8(lds_tr4(&tx[tile_at<XPR>(16 * s + 8 * hi + trow, 32 * wave + tcol)]),
                          lds_tr4(&tx[tile_at<XPR>(16 * s + 8 * hi + 4 + trow, 32 * wave + tcol)]));

        if constexpr (FULL) {
            if constexpr (NW == 4) {
                if (wave < 3) scores(wave, tk);
            } else {
                scores(wave, tk);
                if (wave == 0) scores(2, tk);
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
                const float f = P.scale_in * sG[n > 0 ? n : 0];
#pragma unroll
                for (int r = 0; r < 16; ++r) Y[I][r] *= f;
            }
            sync_lds();                // the scores are there; a and x are free
            if constexpr (FAST) {
                if (c + 1 < c1) fetch_ax(c + 1, 0);
            }
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
                        if (FAST || x + 8 <= P.xd) {
                            if (x < P.xd) {
                                *reinterpret_cast<f32x4_any*>(y) = f32x4{Y[I][8 * h], Y[I][8 * h + 1], Y[I][8 * h + 2], Y[I][8 * h + 3]};
                                *reinterpret_cast<f32x4_any*>(y + 4) = f32x4{Y[I][8 * h + 4], Y[I][8 * h + 5], Y[I][8 * h + 6], Y[I][8 * h + 7]};
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (x + e < P.xd) y[e] = Y[I][8 * h + e];
                        }
                    } else {
                        u16* y = static_cast<u16*>(P.y) + at + x;
                        const u32x4 v = as_u32x4(acc_half(Y[I], h));
                        if (FAST || x + 8 <= P.xd) {
                            if (x < P.xd) *reinterpret_cast<u32x4_any*>(y) = v;
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (x + e < P.xd) y[e] = (u16)(v[e / 2] >> (16 * (e & 1)));
                        }
                    }
                }
            }
        }

        // ---- the state after the chunk ----
        const float through = sG[kC - 1 - r0 + lead];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt] *= through;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const f32x4* pw = reinterpret_cast<const f32x4*>(&sGw[kC - 8 - (16 * s + 8 * hi)]);
            const f32x4 late = pw[0], early = pw[1];
            const float wt[8] = {early[3], early[2], early[1], early[0], late[3], late[2], late[1], late[0]};
            bf16x8 xs[3];
            split3(xf[s], wt, xs);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const bf16x8 cf = join8(lds_tr4(&tk[tile_at<CPR>(16 * s + 8 * hi + trow, 32 * nt + tcol)]),
                                        lds_tr4(&tk[tile_at<CPR>(16 * s + 8 * hi + 4 + trow, 32 * nt + tcol)]));
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
        for (int64_t t = e0 + tid / XW; t < e1; t += 64 * NW / XW) {
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

template <bool FULL, int KD, bool FAST>
hipError_t launch(const AttnArgs& A, unsigned grid, hipStream_t st) {
    if (attn_waves(A.p.xd) == 4) k_attn<KD, 4, FULL, FAST><<<grid, 256, 0, st>>>(A);
    else k_attn<KD, 2, FULL, FAST><<<grid, 128, 0, st>>>(A);
    return hipGetLastError();
}
template <bool FULL, bool FAST> hipError_t launch(const AttnArgs& A, hipStream_t st) {
    const unsigned grid = (unsigned)((A.items + kXcds - 1) / kXcds * kXcds);
    switch (attn_width(A.p.cd)) {
        case 64: return launch<FULL, 64, FAST>(A, grid, st);
        case 128: return launch<FULL, 128, FAST>(A, grid, st);
        default: return launch<FULL, 256, FAST>(A, grid, st);
    }
}

// whole 16-byte pieces at whole 16-byte places, a tile's rows within 24 bits of each other
bool whole_pieces(const void* p, int64_t bs, uint32_t rs, int d) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bs % 8 == 0 && rs % 8 == 0 && d % 8 == 0 && rs < (1u << 22);
}

}  // namespace

hipError_t launch_attn_bf16(const AttnArgs& A, bool full, hipStream_t st) {
    const AttnPass& p = A.p;
    const bool fast = (!full || whole_pieces(p.a, p.ab, p.ar, p.cd)) && whole_pieces(p.c, p.cb, p.cr, p.cd) &&
                      whole_pieces(p.x, p.xb, p.xr, p.xd);
    if (full) return fast ? launch<true, true>(A, st) : launch<true, false>(A, st);
    return fast ? launch<false, true>(A, st) : launch<false, false>(A, st);
}

}  // namespace ssd
