// chan_util.hpp -- device-side pieces shared by the per-channel scan's kernels.
#pragma once
#include "layer_launch.hpp"
#include "ssd_device.hpp"

namespace ssd {

struct ChanArgs {
    ChanIn in;
    int64_t L, D, ub, db, zb, Bb, Cb;      // batch strides in elements
    uint32_t ur, dr, zr, Br, Cr;           // step strides in bytes
    int64_t seg, nseg;
    int N, per, tpg;          // states; channels of a group and its workgroups
    int softplus;
    void* y;
    float *hfin, *S, *sumdt;
};

// A row that is the same for the whole wavefront: a base in scalar registers, to
// which a lane adds its 32-bit byte offset.  The empty asm keeps the offset's
// extension to 64 bits beside the access, where it is free: hoisted out of a loop
// it took two vector registers per access and an addition each time.  It works on
// the caller's variable: on a copy, every access in a loop costs the move of it.
typedef __attribute__((address_space(1))) char GlobalByte;
typedef GlobalByte* RowOut;
typedef const GlobalByte* RowIn;
__device__ __forceinline__ RowIn row_in(const void* p, int64_t bytes) { return (RowIn)(uintptr_t)p + bytes; }
__device__ __forceinline__ RowOut row_out(void* p, int64_t bytes) { return (RowOut)(uintptr_t)p + bytes; }
template <typename T> __device__ __forceinline__ T load_at(RowIn row, uint32_t& off) {
    asm volatile("" : "+v"(off));
    return *reinterpret_cast<const __attribute__((address_space(1))) T*>(row + off);
}
__device__ __forceinline__ void store_at(RowOut row, uint32_t& off, float v, float) {
    asm volatile("" : "+v"(off));
    *reinterpret_cast<__attribute__((address_space(1))) float*>(row + off) = v;
}
__device__ __forceinline__ void store_at(RowOut row, uint32_t& off, float v, u16) {
    asm volatile("" : "+v"(off));
    *reinterpret_cast<__attribute__((address_space(1))) u16*>(row + off) = f32_to_bf_bits(v);
}

// four consecutive elements of a row, at any element's alignment
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef u16 u16x4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void load_quad(const float* p, float (&f)[4]) {
    const f32x4_any v = *reinterpret_cast<const f32x4_any*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = v[k];
}
__device__ __forceinline__ void load_quad(const u16* p, float (&f)[4]) {
    const u16x4_any v = *reinterpret_cast<const u16x4_any*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = bf_bits_to_f32(v[k]);
}
// Values n0 .. of a channel's N, 0 past them.  All are read, those past N as the last:
// a condition around each read would have it wait for its own value, one memory
// latency after the other.
template <int NR> __device__ __forceinline__ void load_values(const float* p, int n0, int N, float (&v)[NR]) {
#pragma unroll
    for (int i = 0; i < NR; ++i) v[i] = p[n0 + i < N ? n0 + i : N - 1];
#pragma unroll
    for (int i = 0; i < NR; ++i) v[i] = n0 + i < N ? v[i] : 0.f;
}
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(u16 v) { return bf_bits_to_f32(v); }

// A log2(e), what dt is multiplied by in a decay's exponent.  Products that overflow, and
// infinities, become the largest finite value: with dt = 0 (steps past the end, masked
// steps, segments of neither) the exponent is then 0 and the state stays, and with any
// other dt down to 1e-36 the decay is 0 (or infinite) as it was.
__device__ __forceinline__ float log2_rate(float A) {
    const float v = A * kLog2e, most = 3.402823466e38f;
    return fabsf(v) > most ? copysignf(most, v) : v;
}

// e^-|x|.  EXACT carries the product with log2(e) in two parts, as its rounding
// alone moves the result by |x| roundings; without it the error stays below
// |x| 2^-24, which bf16 inputs do not need less than.
template <bool EXACT> __device__ __forceinline__ float exp_neg_abs(float x) {
    const float a = -fabsf(x), p = a * kLog2e;
    const float e = fast_exp2(p);
    if constexpr (EXACT) {
        const float lo = fmaf(a, kLog2e, -p) + a * 1.9259629911e-8f;   // log2(e) - float(log2(e))
        // below 2e-5 in size wherever e is not 0; an infinity or NaN where p overflowed (x
        // beyond 2.3e38: masks of the lowest value, infinities), which e = 0 has to win over
        return fmaf(e, __builtin_amdgcn_fmed3f(lo, -1.f, 1.f) * 0.69314718f, e);
    }
    return e;
}
// log(1 + y), y in [0, 1], to a few roundings of the result: the part of y that
// 1 + y loses is added back (it is below 2^-24, so its slope may be taken as 1).
__device__ __forceinline__ float log1p_unit(float y) {
    const float w = 1.f + y, lost = y - (w - 1.f);
    return fmaf(__builtin_amdgcn_logf(w), 0.69314718f, lost);
}
template <bool EXACT> __device__ __forceinline__ float softplus_of(float x) {
    return fmaxf(x, 0.f) + log1p_unit(exp_neg_abs<EXACT>(x));
}
__device__ __forceinline__ float sigmoid_of(float x) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * x));
}

__device__ __forceinline__ int64_t chan_length(const int32_t* lens, int64_t b, int64_t L) {
    if (!lens) return L;
    const int64_t n = lens[b];
    return n < 0 ? 0 : n > L ? L : n;
}

inline ChanArgs chan_args(const ChanShape& s, const ChanIn& in) {
    ChanArgs a = {};
    a.in = in;
    a.L = s.L; a.D = s.D; a.N = (int)s.N;
    a.ub = s.ub; a.db = s.db; a.Bb = s.Bb; a.Cb = s.Cb;
    a.zb = in.gate ? s.zb : s.ub;   // without a gate the kernels load u in its place
    const uint32_t es = s.bf16 ? 2 : 4;
    a.ur = (uint32_t)s.ur * es; a.dr = (uint32_t)s.dr * es; a.zr = (uint32_t)(in.gate ? s.zr : s.ur) * es;
    a.Br = (uint32_t)s.Br * es; a.Cr = (uint32_t)s.Cr * es;
    a.per = (int)(s.D / s.G);
    a.softplus = s.softplus;
    return a;
}

}  // namespace ssd
