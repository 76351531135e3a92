// attn_util.hpp -- device-side pieces shared by the linear attention kernels: rows
// loaded 16 bytes at a time at any alignment and length, the walk's bookkeeping, the
// states' places in memory, tiles in LDS, and values as sums of bf16 parts.
#pragma once
#include "attn_launch.hpp"
#include "mfma_util.hpp"

namespace ssd {

// Up to three walks of one instance in a launch.  The first `whole` (batch, head) pairs are
// walked by a workgroup each (and slice of columns), the others by `segs` of them.
struct AttnArgs {
    AttnPass p[3];
    float* slots[3];         // states at the segments' ends, [pairs - whole][nseg - 1][Dv * Dk]
    const float* log_decay;
    const int32_t* lens;
    int64_t L;
    int cps, nseg;           // chunks of a segment, segments of a pair
    unsigned walks, H, slices, pairs, whole, segs;   // segs: those of this launch
    unsigned skip_whole;     // 1 for the segments' ends, which whole pairs do not have
};
// items of a launch: of whole pairs, and of segments
inline __host__ __device__ unsigned attn_first(const AttnArgs& A) { return A.skip_whole ? 0 : A.whole * A.slices * A.walks; }
inline __host__ __device__ unsigned attn_rest(const AttnArgs& A) { return (A.pairs - A.whole) * A.segs * A.slices * A.walks; }
inline unsigned attn_grid(const AttnArgs& A) { return (attn_first(A) + kXcds - 1) / kXcds * kXcds + (attn_rest(A) + kXcds - 1) / kXcds * kXcds; }

__device__ __forceinline__ int64_t attn_length(const int32_t* lens, int64_t b, int64_t L) {
    if (!lens) return L;
    const int64_t n = lens[b];
    return n < 0 ? 0 : n > L ? L : n;
}

// log_decay in powers of two, as the sum of two floats, bounded to finite values:
// gamma^0 is then 1 whatever the decay, and a decay of -infinity forgets all at once.
struct Decay {
    float hi, lo;
};
__device__ __forceinline__ Decay log2_decay(float log_decay) {
    const float v = log_decay * kLog2e, most = 3.402823466e38f;
    if (!(fabsf(v) < 1e30f)) return Decay{fabsf(v) > most ? copysignf(most, v) : v, 0.f};
    return Decay{v, fmaf(log_decay, kLog2e, -v) + log_decay * 1.9259629911e-8f};   // log2(e) - float(log2(e))
}
// gamma^n, n a whole number >= 0.  What the exponent's roundings lose is carried along:
// alone they would move the result by |exponent| roundings.
__device__ __forceinline__ float decay_pow(const Decay& g, int n) {
    const float f = (float)n, e = g.hi * f, v = fast_exp2(e);
    const float lo = fmaf(g.lo, f, fmaf(g.hi, f, -e));
    return fabsf(e) < 200.f ? fmaf(v, lo * 0.69314718f, v) : v;
}

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ u32x4 load16(const u16* p) { return *reinterpret_cast<const u32x4_any*>(p); }
__device__ __forceinline__ u32x4 load16(const float* p) { return *reinterpret_cast<const u32x4_any4*>(p); }

// A thread's 16-byte piece of every row of a tile: elements [col, col + E) of rows of
// `d` elements.  It is read from where a whole piece of the row is left (at +
// shifted(...) the elements then move down by `skip`), so that no read passes the
// row's end; rows shorter than a piece are read an element at a time.
template <typename T> struct Piece {
    static constexpr int E = 16 / sizeof(T);
    int at, skip;
    __device__ __forceinline__ Piece(int col, int d) {
        const bool shortrow = d < E;
        const int most = d - E;
        at = shortrow ? 0 : col < most ? col : most;
        skip = shortrow ? (col < d ? 0 : E) : col - at;
        if (skip > E) skip = E;
    }
    __device__ __forceinline__ u32x4 load_short(const T* row, int d) const {
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t bits = (uint32_t)raw(row[e < d ? e : 0]);
            if constexpr (E == 8) v[e / 2] |= (e < d ? bits : 0u) << (16 * (e & 1));
            else v[e] = e < d ? bits : 0u;
        }
        return v;
    }
    // what belongs at col.., zeros past the row's end
    __device__ __forceinline__ u32x4 shifted(u32x4 v) const {
        if constexpr (E == 8) {
            if (skip & 4) v = u32x4{v[2], v[3], 0, 0};
            if (skip & 2) v = u32x4{v[1], v[2], v[3], 0};
            if (skip & 1)
                v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
            if (skip & 8) v = u32x4{0, 0, 0, 0};
        } else {
            if (skip & 2) v = u32x4{v[2], v[3], 0, 0};
            if (skip & 1) v = u32x4{v[1], v[2], v[3], 0};
            if (skip & 4) v = u32x4{0, 0, 0, 0};
        }
        return v;
    }
    static __device__ __forceinline__ uint32_t raw(u16 v) { return v; }
    static __device__ __forceinline__ uint32_t raw(float v) { return __float_as_uint(v); }
};

// A workgroup's place: its walk, batch, head, first column, segment; the sequence's length.  All of
// it the same for the workgroup, and in scalar registers (the copies to LDS take their base
// from there).
struct AttnPlace {
    int64_t b;
    int walk, seg, nseg, cps, len, h, x0;
    int64_t state, slot;     // indices of the pair's state, and of its first segment's among the slots
};
__device__ __forceinline__ unsigned uniform(unsigned v) { return (unsigned)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ bool attn_place(const AttnArgs& A, int width, AttnPlace* w) {
    // Workgroups alternate over the XCDs: those of one take neighbouring items, so that the
    // walks of a pair, the slices of a head and the heads of a row meet in one L2.
    const unsigned first = attn_first(A), rest = attn_rest(A), xcd = blockIdx.x % kXcds;
    const unsigned per = (first + kXcds - 1) / kXcds, more = (rest + kXcds - 1) / kXcds;
    unsigned j = blockIdx.x / kXcds, i, segs = 1;
    if (j < per) {
        i = xcd * per + j;
        if (i >= first) return false;
    } else {
        j -= per;
        i = xcd * more + j;
        if (j >= more || i >= rest) return false;
        segs = 0;
    }
    w->walk = (int)uniform(i % A.walks);
    i /= A.walks;
    w->x0 = (int)uniform(i % A.slices) * width;
    i /= A.slices;
    const unsigned in = segs ? A.whole : A.pairs - A.whole, pair = uniform(i % in + (segs ? 0 : A.whole));
    w->seg = (int)uniform(i / in);
    w->nseg = segs ? 1 : A.nseg;
    w->cps = segs ? 1 << 26 : A.cps;
    w->b = uniform(pair / A.H);
    w->h = (int)uniform(pair % A.H);
    w->len = (int)uniform((unsigned)attn_length(A.lens, w->b, A.L));
    w->state = pair;
    w->slot = (int64_t)(pair - A.whole) * (A.nseg - 1);
    return true;
}

// Places in a tile of rows of PR 16-byte pieces, swizzled.
template <int PR> __device__ __forceinline__ int tile_bits(int r) { return swzbits<(PR > 16 ? 16 : PR)>(r); }
template <int PR> __device__ __forceinline__ int tile_at(int row, int col) {
    return row * (PR * 8) + ((((col >> 3) ^ tile_bits<PR>(row)) << 3) | (col & 7));
}

// LDS by byte address
__device__ __forceinline__ bf16x8 lds_piece(uint32_t at) {
    return as_bf16x8(*reinterpret_cast<__attribute__((address_space(3))) const u32x4*>(at));
}
__device__ __forceinline__ bf16x8 lds_transposed(uint32_t first, uint32_t second) {
    return join8(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(first)),
                 __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(second)));
}
__device__ __forceinline__ void lds_store4(uint32_t at, u32x4 v) {
    *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(at) = v;
}
__device__ __forceinline__ void lds_store2(uint32_t at, u32x2 v) {
    *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(at) = v;
}
// The compiler would keep every address that a loop derives from `at` in a register of its
// own; after this it derives them where they are used.
__device__ __forceinline__ uint32_t fresh(uint32_t at) {
    asm volatile("" : "+v"(at));
    return at;
}

// What a rounding to bf16 left of the low and the high value of `pair`, exact: one
// v_dot2_f32_bf16 each, with (-1, 0) or (0, -1), in place of a shift or mask and a
// subtraction.  The factors come in registers: as a literal the low one is taken for the
// inline constant -1.0, whose one is in the high half.
struct Minus {
    uint32_t low, high;
    __device__ __forceinline__ Minus() : low(0x0000bf80u), high(0xbf800000u) { asm volatile("" : "+s"(low), "+s"(high)); }
    static __device__ __forceinline__ float dot(uint32_t pair, uint32_t one, float v) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, one), v, false);
    }
    __device__ __forceinline__ uint32_t rest(float v, float w, uint32_t pair) const {   // rounded in turn
        return pack2(dot(pair, low, v), dot(pair, high, w));
    }
};

// v as a sum of bf16 parts: three, or two and no third
__device__ __forceinline__ void split3(const float (&v)[8], const Minus& minus, bool three, bf16x8 (&o)[3]) {
    u32x4 part[3] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        part[0][e] = pack2(v[2 * e], v[2 * e + 1]);
        const float lo = minus.dot(part[0][e], minus.low, v[2 * e]), hi = minus.dot(part[0][e], minus.high, v[2 * e + 1]);
        part[1][e] = pack2(lo, hi);
        if (three) part[2][e] = minus.rest(lo, hi, part[1][e]);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) o[p] = as_bf16x8(part[p]);
}
// eight bf16 times w, split
__device__ __forceinline__ void split3(const bf16x8& v, const float (&w)[8], const Minus& minus, bool three,
                                       bf16x8 (&o)[3]) {
    const u32x4 u = as_u32x4(v);
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = w[2 * e] * __uint_as_float(u[e] << 16);
        f[2 * e + 1] = w[2 * e + 1] * __uint_as_float(u[e] & 0xffff0000u);
    }
    split3(f, minus, three, o);
}

}  // namespace ssd
