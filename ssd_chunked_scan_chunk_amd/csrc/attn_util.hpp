// attn_util.hpp -- device-side pieces shared by the linear attention kernels: rows
// loaded 16 bytes at a time at any alignment and length, the walk's bookkeeping,
// and the states' places in memory.
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

}  // namespace ssd
