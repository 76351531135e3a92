// attn_walk.hpp -- linear attention with a decay per head, bf16: one walk over the
// sequences in chunks of C steps, 64 where 128 x 128 elements are held and 32 otherwise
// (AttnPass in attn_launch.hpp has the recurrence).
//
// With gamma the head's decay and S the state before the chunk,
//     y_i = sum_{j<=i} gamma^(i-j) (a_i . c_j) x_j + gamma^(i+1) S a_i
//     S'  = gamma^C S + sum_j gamma^(C-1-j) x_j c_j^T
// on v_mfma_f32_32x32x16_bf16.  A workgroup owns a (batch,
// head), 64 or 128 columns x and a segment of the chunks.  Each of its state wavefronts keeps 32
// columns of the state in accumulators.  As many more wavefronts bring the rows to LDS, two
// chunks ahead, and form the decayed scores, one chunk ahead: neither the copies, which hold
// a wavefront for 170 cycles each while HBM is busy, nor the scores' chain of reads, products
// and splits (2300 cycles) stands in the state wavefronts' way, and the workgroup meets at
// one barrier per chunk.
//
// Precision.  The rows are bf16 and their products exact, but three factors are made
// here and have to be rounded to multiply on: the decayed scores and the state in
// the product with a are split into a high and a low bf16 part (17 bits); the decayed x,
// whose errors stay in the states (an fp32 output), into three parts (25 bits), or two
// where no state is asked for (dq, dk).  y is off by its own rounding, 2^-8 of it, and by 2^-17
// of the sum of its terms' magnitudes, of which the rounding is the larger unless they cancel
// to less than 2^-9 of that sum (32-bit factors would leave 2^-24 of it).  One part each would put y
// 1.7 roundings off in place of one and the states at 2e-3 in place of 1e-7.
//
// Bound by HBM where every CU has a workgroup (8 x 2048 x 32 heads of 128 x 128: 137 us, 4.0 of the
// 4.5 TB/s of a large copy), else by the state wavefronts' chain, 6000 cycles to a chunk of 64 steps:
// 2270 the product with the state, 760 that with the scores, 2800 the state's step.  256 wide, a
// lane holds 128 numbers of the state, and four wavefronts of it spill, 44 to 52 bytes a lane.
#pragma once
#include <type_traits>

#include "attn_util.hpp"

namespace ssd {
namespace {

// A tile of C rows with PR pieces of 16 bytes each, brought from memory to LDS by W
// wavefronts.  Its first row is memory row 0 of `base` (C - 1 against time), rows are rs
// elements apart; rows before r0 are no part of the sequence.
//
// FAST: copied to LDS as it comes (rows and strides of whole aligned pieces), the tile's
// swizzle made by the order in which the lanes take a row's pieces.  Pieces past a row's
// end are not copied (clear() once), rows before r0 cleared.
template <int C, int PR, int W> struct Copy {
    static constexpr int N = C * PR / 64 / W, RS = W * 64 / PR;     // copies of a wavefront, rows between them
    uint32_t off[N];
    int row0, wave;
    uint32_t on;               // bit k: the lane's piece of copy k lies in the row
    __device__ __forceinline__ Copy(int wave_, int lane, uint32_t rs, int rev, int col0, int d) {
        wave = wave_;
        row0 = wave * (64 / PR) + lane / PR;
        on = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int r = row0 + k * RS, col = col0 + ((lane % PR) ^ tile_bits<PR>(r)) * 8;
            off[k] = __umul24((uint32_t)(rev ? C - 1 - r : r), 2 * rs) + 2 * col;
            on |= (col < d ? 1u : 0u) << k;
        }
    }
    __device__ __forceinline__ void clear(u16* tile, int lane) const {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (!(on >> k & 1))
                lds_store4(lds_addr(tile) + (uint32_t)(k * W + wave) * 1024 + 16 * lane, u32x4{0, 0, 0, 0});
    }
    __device__ __forceinline__ void get(const u16*, uint32_t, int, int, int) {}
    __device__ __forceinline__ void put(const u16* base, u16* tile, int r0, int lane) const {
        const uintptr_t at = reinterpret_cast<uintptr_t>(base);   // the same in all lanes, into scalar registers
        const void* from = reinterpret_cast<const void*>((uintptr_t)uniform((uint32_t)(at >> 32)) << 32 | uniform((uint32_t)at));
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t lds = lds_addr(tile) + (uint32_t)(k * W + wave) * 1024;
            if ((on >> k & 1) && row0 + k * RS >= r0) dma16(from, off[k], lds);
            else if (row0 + k * RS < r0) lds_store4(lds + 16 * lane, u32x4{0, 0, 0, 0});
        }
    }
};

// Otherwise: read to registers at any alignment and length, put into the tile later.  A row's
// last piece, if it is not whole, is read from where a whole one is left and shifted (Piece),
// by lanes of its own, a row each: were all lanes to shift as one of a row needs to, 4 x 2048 x 32
// heads of 109 x 99 would take 170 us, so they take 147 (104 x 104, aligned: 97).  Pieces past
// it are cleared once.
template <int C, int PR, int W> struct Stage {
    static constexpr int NTH = 64 * W, N = C * PR / NTH, RS = NTH / PR;   // pieces of a thread, rows between them
    static constexpr int TR = C / W;                                      // rows whose last piece a wavefront takes
    static_assert(TR <= 64, "one to a lane");
    Piece<u16> last;
    int row0, at, col, full, tail, trow;   // whole pieces of the tile's rows; 1 if a last one follows; its row, or -1: none for this lane
    u32x4 v[N], t;
    __device__ __forceinline__ Stage(int wave, int lane, uint32_t, int, int col0, int d)
        : last(col0 + (d - col0) / 8 * 8, d) {
        full = (d - col0) / 8 < PR ? (d - col0) / 8 : PR;
        row0 = (64 * wave + lane) / PR;
        col = lane % PR * 8;
        at = full > 0 ? col0 + (col < 8 * full ? col : 0) : 0;   // read and dropped past them
        tail = full < PR && d % 8 != 0 ? 1 : 0;
        trow = tail && lane < TR ? wave * TR + lane : -1;
    }
    __device__ __forceinline__ void get(const u16* base, uint32_t rs, int rev, int r0, int d) {
        auto row = [&](int r) {
            r = r < r0 ? r0 : r;
            return base + (uint32_t)(rev ? C - 1 - r : r) * rs;
        };
        const int tr = trow < 0 ? 0 : trow;    // read and dropped: a condition would have the read wait
        if (d >= 8) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = load16(row(row0 + k * RS) + at);
            t = load16(row(tr) + last.at);
        } else {
            t = last.load_short(row(tr), d);
        }
    }
    __device__ __forceinline__ void clear(u16* tile, int) const {
        if (col >= 8 * (full + tail)) {    // not the last pieces: other wavefronts may have put them already
#pragma unroll
            for (int k = 0; k < N; ++k)
                lds_store4(lds_addr(tile) + 2 * tile_at<PR>(row0 + k * RS, col), u32x4{0, 0, 0, 0});
        }
    }
    __device__ __forceinline__ void put(const u16*, u16* tile, int r0, int) {
        if (col < 8 * full) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int r = row0 + k * RS;
                lds_store4(lds_addr(tile) + 2 * tile_at<PR>(r, col), r < r0 ? u32x4{0, 0, 0, 0} : v[k]);
            }
        }
        if (trow >= 0)
            lds_store4(lds_addr(tile) + 2 * tile_at<PR>(trow, 8 * full), trow < r0 ? u32x4{0, 0, 0, 0} : last.shifted(t));
    }
};

// KD: contracted elements held (64, 128 or 256); NW state wavefronts, and as many others; C
// steps to a chunk.  FULL: y and the last state; else the states at the segments' ends.
// FAST: see Copy.  EX: the decayed x in three parts; YF: y in fp32.
//
// While the state wavefronts work on chunk c, a and c of chunk c + 2, x of chunk c + 1 and
// the scores of chunk c + 1 are made.  At 128 x 128 in chunks of 64 that is 153 KB, one
// workgroup and two wavefronts per SIMD to a CU, with 256 registers each (8 x 2048 x 32 heads:
// two workgroups of six wavefronts whose copies and scores share the chunk's halves took
// 157 us); the other sizes take chunks of 32, as they fit two to four workgroups or
// (256 wide) one.
template <int KD, int NW> constexpr int attn_steps() { return KD == 128 && NW == 4 ? 64 : 32; }
template <int KD, int NW> constexpr int waves_per_simd() { return KD == 64 ? 4 : KD == 256 && NW == 2 ? 1 : 2; }
template <int KD, int NW, bool FULL> struct Tiles {
    static constexpr int C = attn_steps<KD, NW>(), XW = 32 * NW, NP = C / 32 * (C / 32 + 1) / 2;
    __attribute__((aligned(16))) u16 sA[FULL ? 3 : 1][FULL ? C * KD : 8];
    __attribute__((aligned(16))) u16 sK[3][C * KD];
    __attribute__((aligned(16))) u16 sX[2][C * XW];
    // decayed scores [i][j] in blocks of 32 x 32, (0,0), (1,1), (1,0), high parts, low parts
    __attribute__((aligned(16))) u16 sP[FULL ? 2 : 1][FULL ? NP : 1][FULL ? 2 * 32 * 32 : 8];
    // powers of gamma: plain, with the scale of the scores (32 zeros ahead), with that of x
    __attribute__((aligned(16))) float sG[C + 4], sGp[32 + C], sGw[C];
};
template <int KD, int NW, bool FULL, bool FAST, bool EX, bool YF>
__device__ __forceinline__ void walk(const AttnArgs& A, const AttnPass& P, const AttnPlace& w, Tiles<KD, NW, FULL>& T) {
    constexpr int C = attn_steps<KD, NW>(), CB = C / 32, CS = C / 16;   // steps; blocks of 32, products' steps of 16
    constexpr int NT = KD / 32, CPR = KD / 8, XW = 32 * NW, XPR = XW / 8, NP = CB * (CB + 1) / 2;
    auto &sA = T.sA;
    auto &sK = T.sK;
    auto &sX = T.sX;
    auto &sP = T.sP;
    auto &sG = T.sG;
    auto &sGp = T.sGp;
    auto &sGw = T.sGw;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, hi = lane >> 5;
    const int rev = P.rev;
    const int chunks = (w.len + C - 1) / C;
    const int c0 = w.seg * w.cps, c1 = c0 + w.cps < chunks ? c0 + w.cps : chunks;
    if (!FULL && c0 + w.cps >= chunks) return;   // no segment follows: its end is not asked for

    // A partial chunk's steps are the last rows of its tile (rows before are zero), so
    // that what follows it by C - 1 - j steps does so there too.
    auto first_row = [&](int c) { return c == chunks - 1 ? chunks * C - w.len : 0; };
    auto memory_row = [&](int c, int r0) -> int64_t {      // of tile row 0, or C - 1 against time
        const int t0 = c * C - r0;
        return rev ? w.len - C - t0 : t0;
    };
    constexpr uint32_t RB = 2 * KD;            // bytes of a row
    // Places in a tile: piece p + q of a row, q in the low bits of it alone, is at the place of
    // piece q exclusive or 16 p, as the swizzle moves pieces by an exclusive or.  row_at:
    // piece hi of row l32.
    const uint32_t row_at0 = 2 * tile_at<CPR>(l32, 8 * hi);
    const uint32_t a_base = lds_addr(sA[0]), x_base = lds_addr(sX[0]), k_base = lds_addr(sK[0]);
    const Minus minus;
    const Decay gamma = log2_decay(A.log_decay[w.h]);

    constexpr int W = NW / 2;                  // wavefronts that copy
    if (wave >= 2 * NW - W) {
        // ================= rows to LDS =================
        const int at = wave - (2 * NW - W);
        const u16* Ab = FULL ? static_cast<const u16*>(P.a) + w.b * P.ab + (w.h / P.ag) * P.cd : nullptr;
        const u16* Cb = static_cast<const u16*>(P.c) + w.b * P.cb + (w.h / P.cg) * P.cd;
        const u16* Xb = static_cast<const u16*>(P.x) + w.b * P.xb + (w.h / P.xg) * P.xd;
        // through registers: a chunk ahead of their place in LDS (backward of 2 x 1024 x 20 heads of 109 x 99
        // 82 us, else 92; 256 wide it costs more spills than it hides: 301 us at 250 x 222, else 295)
        constexpr bool AHEAD = !FAST && KD < 256;
        using RowsC = typename std::conditional<FAST, Copy<C, CPR, W>, Stage<C, CPR, W>>::type;
        using RowsX = typename std::conditional<FAST, Copy<C, XPR, W>, Stage<C, XPR, W>>::type;
        RowsC ga(at, lane, P.ar, rev, 0, P.cd), gc(at, lane, P.cr, rev, 0, P.cd);
        RowsX gx(at, lane, P.xr, rev, w.x0, P.xd);
        auto get_ac = [&](int c) {
            const int r0 = first_row(c);
            const int64_t m = memory_row(c, r0);
            if constexpr (FULL) ga.get(Ab + m * P.ar, P.ar, rev, r0, P.cd);
            gc.get(Cb + m * P.cr, P.cr, rev, r0, P.cd);
        };
        auto get_x = [&](int c) { gx.get(Xb + memory_row(c, first_row(c)) * P.xr, P.xr, rev, first_row(c), P.xd); };
        auto put_ac = [&](int c, int buf) {
            const int r0 = first_row(c);
            const int64_t m = memory_row(c, r0);
            if constexpr (FULL) ga.put(Ab + m * P.ar, sA[FULL ? buf : 0], r0, lane);
            gc.put(Cb + m * P.cr, sK[buf], r0, lane);
        };
        auto put_x = [&](int c, int buf) { gx.put(Xb + memory_row(c, first_row(c)) * P.xr, sX[buf], first_row(c), lane); };
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if constexpr (FULL) ga.clear(sA[FULL ? i : 0], lane);
            gc.clear(sK[i], lane);
            if (i < 2) gx.clear(sX[i], lane);
        }
        if (c0 < c1) {
            get_ac(c0);
            get_x(c0);
            put_ac(c0, 0);
            put_x(c0, 0);
            if (c0 + 1 < c1) {
                get_ac(c0 + 1);
                put_ac(c0 + 1, 1);
            }
            if (AHEAD && c0 + 1 < c1) get_x(c0 + 1);
            if (AHEAD && c0 + 2 < c1) get_ac(c0 + 2);
        }
        if constexpr (FAST) vm_wait_all();
        sync_lds();                    // the first two chunks' a and c, the first's x
        sync_lds();                    // the first chunk's scores
        int b3 = 2;                    // chunk c + 2's tiles
        for (int c = c0; c < c1; ++c) {
            if (!AHEAD && c + 1 < c1) get_x(c + 1);
            if (!AHEAD && c + 2 < c1) get_ac(c + 2);
            if (c + 1 < c1) put_x(c + 1, (c + 1 - c0) & 1);
            if (c + 2 < c1) put_ac(c + 2, b3);
            if (AHEAD && c + 2 < c1) get_x(c + 2);
            if (AHEAD && c + 3 < c1) get_ac(c + 3);
            b3 = b3 == 2 ? 0 : b3 + 1;
            if constexpr (FAST) vm_wait_all();  // they have landed
            sync_lds();
        }
        return;
    }
    if (wave >= NW) {
        // ================= scores =================
        const int at = tid - 64 * NW;
        if (at < 64) {
            // powers past the sequence's length meet nothing but its missing rows' zeros: 0, as growth
            // may make infinities of them that the sequence itself does not reach
            for (int n = at; n <= C; n += 64) {
                const float p = n <= w.len ? decay_pow(gamma, n) : 0.f;
                sG[n] = p;
                if (n < C) {
                    sGp[32 + n] = P.scale_p * p;
                    sGw[n] = P.scale_w * p;
                }
                if (n < 32) sGp[n] = 0.f;
            }
        }
        // block t of (I, J) = (0,0), (1,1), (1,0); register r is row j = 8 (r / 4) + 4 hi + r % 4,
        // the lane column i = l32
        auto block = [&](int t, int b3, int pb, uint32_t row_at) {
            const int I = t > 0 ? 1 : 0, J = t == 1 ? 1 : 0;
            const uint32_t ka = k_base + b3 * C * RB + 32 * J * RB, aa = a_base + b3 * C * RB + 32 * I * RB;
            const float* pw = &sGp[32 + 32 * (I - J) + l32 - 4 * hi];
            float pv[16];
            f32x16 s = zero16();
            bf16x8 cf[4], af[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                cf[k] = lds_piece((row_at ^ (32 * k)) + ka);
                af[k] = lds_piece((row_at ^ (32 * k)) + aa);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) pv[r] = pw[-(8 * (r >> 2) + (r & 3))];
#pragma unroll
            for (int k = 0; k < KD / 16; ++k) {
                s = mfma32(cf[k & 3], af[k & 3], s);
                if (k + 4 < KD / 16) {
                    cf[k & 3] = lds_piece((row_at ^ (32 * (k + 4))) + ka);
                    af[k & 3] = lds_piece((row_at ^ (32 * (k + 4))) + aa);
                }
            }
            const uint32_t row = lds_addr(sP[FULL ? pb : 0][FULL ? t : 0]) + (uint32_t)l32 * 64 + 8 * hi;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)   // steps ahead are replaced, not multiplied by 0
                    v[e] = 32 * (I - J) + l32 - 4 * hi >= 8 * q + e ? s[4 * q + e] * pv[4 * q + e] : 0.f;
                const uint32_t h01 = pack2(v[0], v[1]), h23 = pack2(v[2], v[3]);
                const uint32_t to = row + 16 * (q ^ ((l32 >> 2) & 3));
                lds_store2(to, u32x2{h01, h23});
                lds_store2(to + 2 * 32 * 32, u32x2{minus.rest(v[0], v[1], h01), minus.rest(v[2], v[3], h23)});
            }
        };

        const int who = wave - NW;
        auto scores = [&](int b3, int pb) {
            if constexpr (FULL) {
                const uint32_t row_at = fresh(row_at0);
                if (who == 0) {
                    block(0, b3, pb, row_at);
                    if constexpr (CB == 2) block(2, b3, pb, row_at);
                } else if (CB == 2) {
                    block(1, b3, pb, row_at);
                }
            }
        };
        sync_lds();
        if (c0 < c1) scores(0, 0);
        sync_lds();
        int b3 = 1;
        for (int c = c0; c < c1; ++c) {
            if (c + 1 < c1) scores(b3, (c + 1 - c0) & 1);
            b3 = b3 == 2 ? 0 : b3 + 1;
            sync_lds();
        }
        return;
    }

    // ================= the state, c by x =================
    // Lane l32 holds column x = x0 + 32 wave + sigma: the quads of each 16 columns come in
    // the order 0, 2, 1, 3, and so do the rows of c, so that registers 8h .. 8h+7 of a 32x32
    // product are rows 16 h + 8 hi + 0 .. 7: the eight consecutive c of one 16-byte read of a
    // row of a, the eight columns of one store.
    const int quad = (l32 >> 2) & 3, swapped = quad == 1 ? 2 : quad == 2 ? 1 : quad;
    const int xc = w.x0 + 32 * wave + (l32 & 16) + 4 * swapped + (l32 & 3);
    const bool mine = xc < P.xd;
    f32x16 S[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) S[t] = zero16();
    const int64_t SE = (int64_t)P.cd * P.xd;
    auto element = [&](int t, int r) { return 32 * t + 16 * (r >> 3) + 8 * hi + (r & 7); };
    const float* from = w.seg == 0 ? (P.first ? P.first + w.state * SE : nullptr)
                      : FULL ? A.slots[w.walk] + (w.slot + w.seg - 1) * SE : nullptr;
    if (from && (w.seg == 0 || c0 < chunks)) {
        // read at a clamped place and dropped: a condition around each read would have it
        // wait for its own value
        const float* col = from + (int64_t)(mine ? xc : 0) * P.sx;
        if (P.sc == 1 && P.cd % 8 == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int e = element(t, r & 8);
                    const f32x4 v = *reinterpret_cast<const f32x4_any*>(col + (e < P.cd ? e + (r & 4) : 0));
#pragma unroll
                    for (int k = 0; k < 4; ++k) S[t][r + k] = v[k];
                }
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) S[t][r] = col[(element(t, r) < P.cd ? element(t, r) : 0) * P.sc];
        }
        int cd = P.cd;
        asm volatile("" : "+s"(cd));   // or the comparisons above stay in scalar registers till here
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[t][r] = mine && element(t, r) < cd ? S[t][r] : 0.f;
    }
    auto save = [&](float* to, float f) {
        float* col = to + (int64_t)xc * P.sx;
        int cd = P.cd;
        asm volatile("" : "+s"(cd));
        if (P.sc == 1 && cd % 8 == 0) {
            if (mine) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 16; r += 4)
                        if (element(t, r & 8) < cd)
                            *reinterpret_cast<f32x4_any*>(col + element(t, r)) =
                                f32x4{f * S[t][r], f * S[t][r + 1], f * S[t][r + 2], f * S[t][r + 3]};
            }
            return;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (mine && element(t, r) < cd) col[element(t, r) * P.sc] = f * S[t][r];
    };

    // tr_at: where a lane points in a transposing read, which gives it four rows of its
    // column (the lanes of a group of 16 point at four rows and four quads of columns), for
    // rows 8 hi + 0 .. 3; the next four rows' swizzle is another by a constant, as it is
    // linear in the row's bits.
    const int trow = 8 * hi + ((lane & 15) >> 2), tq = lane & 3;
    const int tcol = (lane & 16) + 4 * (tq == 1 ? 2 : tq == 2 ? 1 : tq);
    const uint32_t tr_at0 = 2 * tile_at<CPR>(trow, tcol), x_at0 = 2 * tile_at<XPR>(trow, 32 * wave + tcol);
    const uint32_t four = 16 * tile_bits<CPR>(4), xfour = 16 * tile_bits<XPR>(4);
    // y's rows of a chunk: lane l32 has two steps, 32 I + l32, of 2 x 8 columns each
    const int x = w.x0 + 32 * wave + 8 * hi;
    constexpr uint32_t es = YF ? 4 : 2;
    const uint32_t yr = A.H * P.xd * es;       // bytes of a row; 64 rows are within 32 bits
    const uint32_t o0 = (uint32_t)(rev ? C - 1 - l32 : l32) * yr + x * es;
    sync_lds();                // the first tiles
    sync_lds();                // the first scores
    int b3 = 0;

    for (int c = c0; c < c1; ++c) {
        const int buf = (c - c0) & 1;
        const int r0 = first_row(c), lead = rev && c == 0 ? 0 : 1;   // against time the given state is the last step's own
        const uint32_t ta = a_base + b3 * C * RB, tk = k_base + b3 * C * RB, tx = x_base + buf * C * 2 * XW;
        b3 = b3 == 2 ? 0 : b3 + 1;
        bf16x8 xf[CS];                 // x^T: lane = column, k = step 16 s + 8 hi + 0 .. 7
#pragma unroll
        for (int s = 0; s < CS; ++s)
            xf[s] = lds_transposed(x_at0 + (tx + 32 * s * XW), (x_at0 ^ xfour) + (tx + 32 * s * XW + 8 * XW));

        f32x16 Y[CB];
        if constexpr (FULL) {
            // ---- from the state: y^T, rows the columns x, lane = step 32 I + l32 ----
            const uint32_t row_at = fresh(row_at0);
#pragma unroll
            for (int I = 0; I < CB; ++I) Y[I] = zero16();
            bf16x8 sh[2], sl[2], af[2][CB];
            auto ready = [&](int st) {     // the operands of 16 contracted elements
                const f32x16& v = S[st >> 1];
                const int h = st & 1, i = st & 1;
                u32x4 up, lo;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    up[k] = pack2(v[8 * h + 2 * k], v[8 * h + 2 * k + 1]);
                    lo[k] = minus.rest(v[8 * h + 2 * k], v[8 * h + 2 * k + 1], up[k]);
                }
                sh[i] = as_bf16x8(up);
                sl[i] = as_bf16x8(lo);
#pragma unroll
                for (int I = 0; I < CB; ++I) af[i][I] = lds_piece((row_at ^ (32 * st)) + (ta + 32 * I * RB));
            };
            ready(0);
#pragma unroll
            for (int st = 0; st < 2 * NT; ++st) {
                const int i = st & 1;
                if (st + 1 < 2 * NT) ready(st + 1);
#pragma unroll
                for (int I = 0; I < CB; ++I) Y[I] = mfma32(sh[i], af[i][I], Y[I]);
#pragma unroll
                for (int I = 0; I < CB; ++I) Y[I] = mfma32(sl[i], af[i][I], Y[I]);
            }
#pragma unroll
            for (int I = 0; I < CB; ++I) {
                const int n = 32 * I + l32 - r0 + lead;
                const float f = P.scale_in * sG[n > 0 ? n : 0];
#pragma unroll
                for (int r = 0; r < 16; ++r) Y[I][r] *= f;
            }
            // ---- from inside the chunk ----
            const uint32_t p_at = lds_addr(sP[FULL ? buf : 0][0]) + (uint32_t)l32 * 64;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                bf16x8 pf[NP][2];
#pragma unroll
                for (int t = 0; t < NP; ++t)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        pf[t][part] = lds_piece(p_at + 16 * ((2 * s + hi) ^ ((l32 >> 2) & 3)) + (t * 2 + part) * 2 * 32 * 32);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    Y[0] = mfma32(xf[s], pf[0][part], Y[0]);
                    if constexpr (CB == 2) {
                        Y[CB - 1] = mfma32(xf[s], pf[NP - 1][part], Y[CB - 1]);
                        Y[CB - 1] = mfma32(xf[CS - 2 + s], pf[NP - 2][part], Y[CB - 1]);
                    }
                }
            }
        }
        char* const yb = FULL ? static_cast<char*>(P.y) + ((w.b * A.L + memory_row(c, r0)) * A.H + w.h) * P.xd * es : nullptr;
        if constexpr (FULL && !FAST) {
#pragma unroll
            for (int I = 0; I < CB; ++I) {
                if (32 * I + l32 < r0) continue;
                char* y = yb + (o0 + (rev ? -32 * I : 32 * I) * yr);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 v = as_u32x4(acc_half(Y[I], h));
                    if (x + 16 * h + 8 <= P.xd) {
                        if constexpr (YF) {
#pragma unroll
                            for (int e = 0; e < 8; e += 4)
                                *reinterpret_cast<f32x4_any*>(y + 4 * (16 * h + e)) =
                                    f32x4{Y[I][8 * h + e], Y[I][8 * h + e + 1], Y[I][8 * h + e + 2], Y[I][8 * h + e + 3]};
                        } else {
                            *reinterpret_cast<u32x4_any*>(y + 2 * 16 * h) = v;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (x + 16 * h + e < P.xd) {
                                if constexpr (YF) reinterpret_cast<float*>(y)[16 * h + e] = Y[I][8 * h + e];
                                else reinterpret_cast<u16*>(y)[16 * h + e] = (u16)(v[e / 2] >> (16 * (e & 1)));
                            }
                    }
                }
            }
        }
        // FAST: whole pieces, stored one by one among the products that follow, without a branch,
        // which would end the stretch of code that is scheduled as one: lanes without a
        // column or a step are past the buffer's end
        constexpr int YN = FULL && FAST ? (YF ? 4 : 2) * CB : 0;
        u32x4 yp[CB][2];
        __amdgpu_buffer_rsrc_t yd;
        uint32_t yo[CB][2];
        if constexpr (YN > 0) {
            yd = __builtin_amdgcn_make_buffer_rsrc(yb, 0, (int)0xffe00000u, 0x00020000);
#pragma unroll
            for (int I = 0; I < CB; ++I)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (!YF) yp[I][h] = as_u32x4(acc_half(Y[I], h));
                    yo[I][h] = 32 * I + l32 >= r0 && x + 16 * h < P.xd ? o0 + (rev ? -32 * I : 32 * I) * yr + 16 * h * es
                                                                      : 0xfff00000u;
                }
        }
        auto store = [&](int k) {
            if constexpr (YN > 0) {
                const int I = k % CB, h = k / CB & 1, e4 = k / CB >> 1;
                if constexpr (YF) {
                    const int e = 8 * h + 4 * e4;
                    const u32x4 v = {__float_as_uint(Y[I][e]), __float_as_uint(Y[I][e + 1]), __float_as_uint(Y[I][e + 2]),
                                     __float_as_uint(Y[I][e + 3])};
                    __builtin_amdgcn_raw_buffer_store_b128(v, yd, yo[I][h], 16 * e4, 0);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b128(yp[I][h], yd, yo[I][h], 0, 0);
                }
            }
        };

        // ---- the state after the chunk ----
        const uint32_t t0 = fresh(tr_at0);
        bf16x8 cf[2], xs[2][3];
        auto column = [&](int i) {         // c^T of steps 16 (i / NT) .., rows 32 (i % NT) ..
            const uint32_t base = tk + 16 * (i / NT) * RB, b = 64 * (i % NT);
            return lds_transposed((t0 ^ b) + base, (t0 ^ (b ^ four)) + (base + 4 * RB));
        };
        auto weigh = [&](int s) {
            const f32x4* pw = reinterpret_cast<const f32x4*>(&sGw[C - 8 - (16 * s + 8 * hi)]);
            const f32x4 late = pw[0], early = pw[1];
            const float wt[8] = {early[3], early[2], early[1], early[0], late[3], late[2], late[1], late[0]};
            split3(xf[s], wt, minus, EX, xs[s & 1]);
        };
        cf[0] = column(0);
        weigh(0);
        const float through = sG[C - 1 - r0 + lead];
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] *= through;
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            if (s + 1 < CS) weigh(s + 1);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int i = s * NT + t;
                if (i + 1 < CS * NT) cf[(i + 1) & 1] = column(i + 1);
                S[t] = mfma32(cf[i & 1], xs[s & 1][0], S[t]);
                S[t] = mfma32(cf[i & 1], xs[s & 1][1], S[t]);
                if constexpr (EX) S[t] = mfma32(cf[i & 1], xs[s & 1][2], S[t]);
#pragma unroll
                for (int k = 0; k < YN; ++k)
                    if (k * (CS * NT / 2) / (YN > 0 ? YN : 1) == i) store(k);   // in the first half
            }
        }
        sync_lds();
    }

    if constexpr (FULL) {
        if (P.last && (chunks > 0 ? c0 < chunks && c1 == chunks : w.seg == 0))
            save(P.last + w.state * SE, rev && chunks > 0 ? decay_pow(gamma, 1) : 1.f);
        // rows behind the sequence's end
        const int64_t e0 = c0 * C > w.len ? c0 * C : w.len;
        const int64_t e1 = w.seg + 1 == w.nseg ? A.L : (c0 + w.cps) * C;
        for (int64_t t = e0 + tid / XW; t < e1; t += 64 * NW / XW) {
            const int col = w.x0 + tid % XW;
            const int64_t at = ((w.b * A.L + t) * A.H + w.h) * P.xd + col;
            if (col < P.xd) {
                if constexpr (YF) static_cast<float*>(P.y)[at] = 0.f;
                else static_cast<u16*>(P.y)[at] = 0;
            }
        }
    } else {
        save(A.slots[w.walk] + (w.slot + w.seg) * SE, 1.f);
    }
}

// Each of a launch's walks has its own EX and YF.
template <int KD, int NW, bool FULL, bool FAST>
__global__ __launch_bounds__(128 * NW, (waves_per_simd<KD, NW>())) void k_attn(const AttnArgs A) {
    __shared__ Tiles<KD, NW, FULL> T;
    AttnPlace w;
    if (!attn_place(A, 32 * NW, &w)) return;
    const AttnPass& P = A.p[w.walk];
    if (FULL && P.y_f32) {
        if (P.exact) walk<KD, NW, FULL, FAST, true, true>(A, P, w, T);
        else walk<KD, NW, FULL, FAST, false, true>(A, P, w, T);
    } else {
        if (P.exact) walk<KD, NW, FULL, FAST, true, false>(A, P, w, T);
        else walk<KD, NW, FULL, FAST, false, false>(A, P, w, T);
    }
}

template <bool FULL, bool FAST> hipError_t launch(const AttnArgs& A, hipStream_t st) {
    const unsigned grid = attn_grid(A);
    const int kd = attn_width(A.p[0].cd);   // attn_chunk() goes by it too
    if (attn_columns(A.p[0].xd) == 128) {
        if (kd == 64) k_attn<64, 4, FULL, FAST><<<grid, 512, 0, st>>>(A);
        else if (kd == 128) k_attn<128, 4, FULL, FAST><<<grid, 512, 0, st>>>(A);
        else k_attn<256, 4, FULL, FAST><<<grid, 512, 0, st>>>(A);
    } else {
        if (kd == 64) k_attn<64, 2, FULL, FAST><<<grid, 256, 0, st>>>(A);
        else if (kd == 128) k_attn<128, 2, FULL, FAST><<<grid, 256, 0, st>>>(A);
        else k_attn<256, 2, FULL, FAST><<<grid, 256, 0, st>>>(A);
    }
    return hipGetLastError();
}
template <bool FAST> hipError_t launch(const AttnArgs& A, bool full, hipStream_t st) {
    return full ? launch<true, FAST>(A, st) : launch<false, FAST>(A, st);
}

}  // namespace
}  // namespace ssd
