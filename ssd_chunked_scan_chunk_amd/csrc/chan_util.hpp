// chan_util.hpp -- device-side pieces shared by the per-channel scan's kernels.
//
// Lane layout of a wavefront: c = lane % 16 picks R consecutive channels, q =
// lane / 16 a quarter of the states (NR = padded states / 4 of them per lane).
// In registers a lane therefore holds R x NR states; sums over the states are
// finished across the four rows of 16 lanes, and B and C, which all channels of
// a group share, are the same for the 16 lanes of a row.  Steps are taken in
// batches of 16 / R: unit j (16 bytes: S = 4 / R steps of R channels) of a batch
// belongs to row q = j, whose lanes load, transform and store it, so that
// per-(step, channel) work is done once.
#pragma once
#include "layer_launch.hpp"
#include "ssd_device.hpp"

namespace ssd {

struct ChanArgs {
    ChanIn in;
    int64_t L, D, ub, ur, db, dr, zb, zr, Bb, Br, Cb, Cr;
    int64_t seg, nseg;
    int N, per, tpg, tiles;   // states, channels and wavefronts per group, wavefronts in all
    int softplus, wide;       // wide: rows allow R elements at once
    void* y;
    float *hfin, *S, *sumdt;
};

// R consecutive elements of a row as stored
template <typename T, int R> struct Elems { T v[R]; };

template <typename T, int R>
__device__ __forceinline__ Elems<T, R> load_elems(const T* p, int live, bool wide) {
    Elems<T, R> e;
    if (R == 4 && wide && live == R) {
        if constexpr (sizeof(T) == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            __builtin_memcpy(&e, &v, sizeof(e) < 8 ? sizeof(e) : 8);
        } else {
            const float4 v = *reinterpret_cast<const float4*>(p);
            __builtin_memcpy(&e, &v, sizeof(e) < 16 ? sizeof(e) : 16);
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) e.v[r] = r < live ? p[r] : T(0);
    }
    return e;
}
template <typename T, int R>
__device__ __forceinline__ void store_elems(T* p, const float* f, int live, bool wide) {
    if (R == 4 && wide && live == R) {
        if constexpr (sizeof(T) == 2) {
            uint2 v;
            v.x = (uint32_t)f32_to_bf_bits(f[0]) | ((uint32_t)f32_to_bf_bits(f[1 % R]) << 16);
            v.y = (uint32_t)f32_to_bf_bits(f[2 % R]) | ((uint32_t)f32_to_bf_bits(f[3 % R]) << 16);
            *reinterpret_cast<uint2*>(p) = v;
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1 % R], f[2 % R], f[3 % R]);
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r < live) Elem<T>::store(p + r, f[r]);
    }
}
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(u16 v) { return bf_bits_to_f32(v); }

// e^-|x| to about an ulp: the product with log2(e) is carried in two parts, as
// its rounding alone would cost |x| ulps.
__device__ __forceinline__ float exp_neg_abs(float x) {
    const float a = -fabsf(x), p = a * kLog2e;
    const float lo = fmaf(a, kLog2e, -p) + a * 1.9259629911e-8f;   // log2(e) - float(log2(e))
    const float e = fast_exp2(p);
    return fmaf(e, lo * 0.69314718f, e);
}
// log(1 + y) for y in [0, 1] to a few ulps of the result: 2 artanh(s) with
// s = y / (2 + y) <= 1/3, whose series after s^13 leaves less than 2^-26.
__device__ __forceinline__ float log1p_unit(float y) {
    const float s = y * __builtin_amdgcn_rcpf(2.f + y), q = s * s;
    float p = fmaf(q, 1.f / 13, 1.f / 11);
    p = fmaf(q, p, 1.f / 9);
    p = fmaf(q, p, 1.f / 7);
    p = fmaf(q, p, 1.f / 5);
    p = fmaf(q, p, 1.f / 3);
    return 2.f * fmaf(s * q, p, s);
}
__device__ __forceinline__ float softplus_of(float x) { return fmaxf(x, 0.f) + log1p_unit(exp_neg_abs(x)); }
__device__ __forceinline__ float sigmoid_of(float x) {
    const float e = exp_neg_abs(x), r = __builtin_amdgcn_rcpf(1.f + e);
    return x >= 0.f ? r : e * r;
}

// Four values per lane, one for each row of 16 lanes: row j receives the sum
// of v[j] over the four rows.  permlane32_swap exchanges the upper half of its
// first operand with the lower half of its second, permlane16_swap the odd rows
// of the first with the even rows of the second: six instructions.
__device__ __forceinline__ float sum_to_rows(float v0, float v1, float v2, float v3) {
    auto bits = [](float f) { return __builtin_bit_cast(unsigned, f); };
    auto flt = [](unsigned u) { return __builtin_bit_cast(float, u); };
    const auto a = __builtin_amdgcn_permlane32_swap(bits(v0), bits(v2), false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(bits(v1), bits(v3), false, false);
    const float x = flt(a[0]) + flt(a[1]), y = flt(b[0]) + flt(b[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(bits(x), bits(y), false, false);
    return flt(c[0]) + flt(c[1]);
}
__device__ __forceinline__ float sum_rows(float v) { return sum_to_rows(v, v, v, v); }

__device__ __forceinline__ int64_t chan_length(const int32_t* lens, int64_t b, int64_t L) {
    if (!lens) return L;
    const int64_t n = lens[b];
    return n < 0 ? 0 : n > L ? L : n;
}

// LDS written and read within one wavefront: its accesses complete in order, the
// compiler is kept from moving them across
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

}  // namespace ssd
