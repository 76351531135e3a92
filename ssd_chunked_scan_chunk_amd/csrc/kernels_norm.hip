// kernels_norm.hip -- the norm over groups of channels of one row, its activation or
// gate, and their gradients.
//
//     u = x, or x act(gate) with the gate first;  n = (u - mean) r,  r = 1 / sqrt(var + eps)
//     p = weight n + bias;  y = act(p), p act(gate), or p with the gate first
// and backward, with dp the gradient of p and dn = weight dp,
//     du = r (dn - [mean(dn)] - n mean(dn n)),  dweight = sum dp n,  dbias = sum dp.
//
// HBM-bound: every row is read once and stays in registers through the sums (the mean
// first, then the squares about it).  A thread owns 16 bytes of channels, the same in
// every row it walks, so weight and bias are loaded once and the parameters'
// gradients add up in registers.  A group is a power of two of lanes of a wavefront, or
// a workgroup with its sums joined in LDS.
#include "attn_launch.hpp"
#include "chan_util.hpp"

namespace ssd {
namespace {

struct NormArgs {
    const void *x, *gate, *dy;
    const float *weight, *bias;
    const int32_t* lens;
    void *y, *dx, *dgate;
    float* parts;
    int64_t rows, L, C, xb, xr, zb, zr;
    int m, G, lanes, gw, rw;      // channels of a group, groups, lanes of one; groups and rows of a workgroup
    float eps, size, inv;         // size: m; inv: 1 / m
    int center, silu, flat;
};

// the sum over `lanes` lanes (a power of two), the same bits in each of them
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    if (lanes > 1) v += dpp<0xb1>(v);         // quad_perm 1, 0, 3, 2
    if (lanes > 2) v += dpp<0x4e>(v);         // quad_perm 2, 3, 0, 1
    if (lanes > 4) v += dpp<0x141>(v);        // row_half_mirror
    if (lanes > 8) v += dpp<0x140>(v);        // row_mirror
    if (lanes > 16) v += __shfl_xor(v, 16, 64);
    if (lanes > 32) v += __shfl_xor(v, 32, 64);
    return v;
}

template <bool BLOCK> struct Sums {
    float* lds;          // BLOCK: two alternating sets of 2 x 16 floats
    int lanes, turn;
    // one or two sums over the group's lanes
    __device__ __forceinline__ void operator()(float& a, float& b, bool two) {
        a = lanes_sum(a, BLOCK ? 64 : lanes);
        if (two) b = lanes_sum(b, BLOCK ? 64 : lanes);
        if constexpr (BLOCK) {
            float* s = lds + 32 * turn;
            turn ^= 1;   // the set before this one may still be read
            const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
            if ((threadIdx.x & 63) == 0) {
                s[wave] = a;
                s[16 + wave] = b;
            }
            lds_barrier();
            a = b = 0.f;
            for (int i = 0; i < waves; ++i) {
                a += s[i];
                b += s[16 + i];
            }
        }
    }
};

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
template <typename T, int V> struct Vec;
template <> struct Vec<u16, 8> {
    typedef u16 raw __attribute__((ext_vector_type(8), aligned(2)));
};
template <> struct Vec<float, 4> {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
};
template <typename T> struct Vec<T, 1> {
    typedef T raw __attribute__((ext_vector_type(1)));
};
__device__ __forceinline__ u16 to_elem(float v, u16) { return f32_to_bf_bits(v); }
__device__ __forceinline__ float to_elem(float v, float) { return v; }

// The exponential and the reciprocal are the hardware's, an ulp each; in fp32 the exponential's
// argument is in two parts, as its rounding alone would move a sigmoid by |x| roundings.
template <typename T> __device__ __forceinline__ float sigmoid_as(float x) {
    if constexpr (sizeof(T) == 2) return sigmoid_of(x);
    const float e = exp_neg_abs<true>(x), d = __builtin_amdgcn_rcpf(1.f + e);
    return x >= 0.f ? d : e * d;
}

// GATE: 0 none, 1 after the norm, 2 before it.  WHOLE: a group is a whole number of pieces;
// otherwise its last one starts early and its first `skip` elements are another thread's
// (with that test at every element the bf16 backward needs 121 registers and 10% longer).
// 16 channels a lane (groups above 8192) do not fit the backward's 128 registers: 396 to 484 bytes
// of scratch with a gate, 120 to 208 without (2 x 2048 x 16384 gated bf16 742 us, floor 148; fp32
// 2 x 1024 x 16384 530, floor 148), and up to 60 in the gated fp32 forward (104 us, floor 89).  8 of
// them in fp32 (groups above 4096) spill 20 to 28 bytes: 4 x 2048 x 5120, gate first, 177 us.
template <typename T, int V, int NP, bool BLOCK, int GATE, bool BWD, bool WHOLE>
__global__ __launch_bounds__(BLOCK ? 1024 : 512, BWD ? 4 : 1) void k_norm(const NormArgs A) {
    using R = typename Vec<T, V>::raw;
    __shared__ float lds[BLOCK ? 64 : 1];
    const int tid = threadIdx.x;
    Sums<BLOCK> sums{lds, A.lanes, 0};
    const int slot = BLOCK ? 0 : tid / A.lanes, first = BLOCK ? tid : tid % A.lanes;
    const int stride = BLOCK ? blockDim.x : A.lanes;
    const int group = blockIdx.x * A.gw + slot % A.gw, rowat = slot / A.gw;
    const bool on = group < A.G && rowat < A.rw;
    const int64_t ch = (int64_t)(on ? group : 0) * A.m;
    int at[NP], skip[NP];          // elements skip .. V-1 of a piece are the thread's own; WHOLE: all or none
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int col = (first + k * stride) * V, most = A.m - V;
        at[k] = col < most ? col : most;
        skip[k] = !on ? V : col - at[k] < V ? col - at[k] : V;
    }
    float wt[NP][V], bs[NP][V], dw[NP][V], db[NP][V];
#pragma unroll
    for (int k = 0; k < NP; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            wt[k][e] = A.weight ? A.weight[ch + at[k] + e] : 1.f;
            bs[k][e] = A.bias ? A.bias[ch + at[k] + e] : 0.f;
            dw[k][e] = db[k][e] = 0.f;
        }
    const float inv = A.inv;
    // sum / m, rounded once: a constant group has n = 0 and a constant gradient dx = 0 wherever the sum
    // is exact, as every sum of up to 16384 equal bf16 values is.  The product with 1 / m alone is an
    // ulp off for up to three in ten m, and n that ulp over sqrt(eps): 0.5 for 30080 and m = 7.
    auto mean_of = [&](float sum) {
        const float q = sum * inv;
        return fmaf(fmaf(-q, A.size, sum), inv, q);
    };
    const int64_t step = (int64_t)gridDim.y * A.rw;
    R xr[NP], zr[NP], dr[NP];
    bool live = false;
    auto own = [&](int k, int e) { return WHOLE ? skip[k] == 0 : e >= skip[k]; };
    auto read = [&](const T* p, R (&to)[NP]) {
#pragma unroll
        for (int k = 0; k < NP; ++k) to[k] = *reinterpret_cast<const R*>(p + at[k]);
    };
    // in fp32; rows that are not there, and pieces of no group, are zeros
    auto values = [&](const R (&from)[NP], bool here, float (&v)[NP][V]) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if constexpr (WHOLE && V > 1) {
                u32x4 w = __builtin_bit_cast(u32x4, from[k]);
                const uint32_t mask = here && skip[k] == 0 ? 0xffffffffu : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j] &= mask;
                    if constexpr (V == 8) {
                        v[k][2 * j] = __uint_as_float(w[j] << 16);
                        v[k][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                    } else {
                        v[k][j] = __uint_as_float(w[j]);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = here && own(k, e) ? as_f32(from[k][e]) : 0.f;
            }
        }
    };
    auto fetch = [&](int64_t row) {
        int64_t b = 0, t = row;
        if (!A.flat) {
            b = (uint32_t)row / (uint32_t)A.L;
            t = row - b * A.L;
        }
        live = row < A.rows && (!A.lens || t < A.lens[b]);
        if (!live) return;
        read(static_cast<const T*>(A.x) + b * A.xb + t * A.xr + ch, xr);
        if constexpr (GATE != 0) read(static_cast<const T*>(A.gate) + b * A.zb + t * A.zr + ch, zr);
        if constexpr (BWD) read(static_cast<const T*>(A.dy) + row * A.C + ch, dr);
    };
    auto put = [&](void* to, int64_t row, const float (&v)[NP][V]) {
        T* p = static_cast<T*>(to) + row * A.C + ch;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            R o;
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = to_elem(v[k][e], T{});
            if (skip[k] == 0) *reinterpret_cast<R*>(p + at[k]) = o;
            else if (!WHOLE && skip[k] < V) {
#pragma unroll
                for (int e = 1; e < V; ++e)
                    if (e >= skip[k]) p[at[k] + e] = o[e];
            }
        }
    };

    // every thread of a workgroup takes the same number of turns: a row of its own or none
    int64_t row = (int64_t)blockIdx.y * A.rw + rowat;
    const int64_t turns = ((int64_t)blockIdx.y * A.rw < A.rows) ? (A.rows - (int64_t)blockIdx.y * A.rw + step - 1) / step : 0;
    if (turns > 0) fetch(row);
    for (int64_t i = 0; i < turns; ++i, row += step) {
        const bool here = live, in = row < A.rows;
        float x[NP][V], z[NP][V], d[NP][V];
        values(xr, here, x);
        if constexpr (GATE != 0) values(zr, here, z);
        if constexpr (BWD) values(dr, here, d);
        if (i + 1 < turns) fetch(row + step);

        // ---- the normalised row ----
        float n[NP][V], act[NP][V], sg[NP][V];   // act(gate) and its sigmoid
        float sum = 0.f, other = 0.f;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if constexpr (GATE != 0) {
                    sg[k][e] = A.silu ? sigmoid_as<T>(z[k][e]) : 1.f;
                    act[k][e] = z[k][e] * sg[k][e];
                }
                n[k][e] = GATE == 2 ? x[k][e] * act[k][e] : x[k][e];
                sum += n[k][e];
            }
        if (A.center) {
            sums(sum, other, false);
            const float mean = mean_of(sum);
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) n[k][e] = own(k, e) ? n[k][e] - mean : 0.f;
        }
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) sq = fmaf(n[k][e], n[k][e], sq);
        sums(sq, other, false);
        const float r = here ? rsqrtf(fmaf(sq, inv, A.eps)) : 0.f;   // zeros of eps 0 have none
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) n[k][e] *= r;

        if constexpr (!BWD) {
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = fmaf(wt[k][e], n[k][e], bs[k][e]);
                    float y = p;
                    if constexpr (GATE == 1) y = p * act[k][e];
                    else if (GATE == 0 && A.silu) y = p * sigmoid_as<T>(p);
                    x[k][e] = here ? y : 0.f;
                }
            if (in) put(A.y, row, x);
        } else {
            auto slope = [&](float v, float s) { return s * fmaf(v, 1.f - s, 1.f); };   // of v sigmoid(v), s its sigmoid
            float c1 = 0.f, c2 = 0.f;
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = fmaf(wt[k][e], n[k][e], bs[k][e]);
                    if constexpr (GATE == 1) {
                        const float dz = d[k][e] * p * (A.silu ? slope(z[k][e], sg[k][e]) : 1.f);
                        d[k][e] *= act[k][e];
                        z[k][e] = dz;
                    } else if (GATE == 0 && A.silu) {
                        d[k][e] *= slope(p, sigmoid_as<T>(p));
                    }
                    dw[k][e] = fmaf(d[k][e], n[k][e], dw[k][e]);
                    db[k][e] += d[k][e];
                    d[k][e] *= wt[k][e];
                    c1 += d[k][e];
                    c2 = fmaf(d[k][e], n[k][e], c2);
                }
            sums(c1, c2, true);
            c1 = A.center ? mean_of(c1) : 0.f;
            c2 *= inv;
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float du = r * (d[k][e] - c1 - n[k][e] * c2);
                    if constexpr (GATE == 2) {
                        z[k][e] = du * x[k][e] * (A.silu ? slope(z[k][e], sg[k][e]) : 1.f);
                        du *= act[k][e];
                    }
                    if constexpr (GATE != 0) z[k][e] = here ? z[k][e] : 0.f;
                    d[k][e] = here ? du : 0.f;
                }
            if (in) {
                put(A.dx, row, d);
                if constexpr (GATE != 0) put(A.dgate, row, z);
            }
        }
    }
    if constexpr (BWD) {
        if (!A.parts) return;
        bool mine = on;
        if constexpr (!BLOCK) {
            // Rows beside each other in a workgroup add their columns up here.  With a part for each
            // of them (up to 256) the sum over the parts read more than the rows hold: 4 x 2048
            // rows of 64 channels took 211 us, now 22, 100000 fp32 rows of 8 channels 1637, now 35.
            if (A.rw > 1) {
                __shared__ float part[2][512];
                const int apart = A.gw * A.lanes;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    part[0][tid] = dw[0][e];
                    part[1][tid] = db[0][e];
                    lds_barrier();
                    if (on && rowat == 0)
                        for (int i = 1; i < A.rw; ++i) {
                            dw[0][e] += part[0][tid + i * apart];
                            db[0][e] += part[1][tid + i * apart];
                        }
                    lds_barrier();
                }
                mine = on && rowat == 0;
            }
        }
        float* p = A.parts + (int64_t)blockIdx.y * 2 * A.C + ch;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (mine && own(k, e)) {
                    p[at[k] + e] = dw[k][e];
                    p[A.C + at[k] + e] = db[k][e];
                }
    }
}

// Sums of the parts, in a fixed order: 64 columns to a workgroup, sixteen wavefronts take
// every sixteenth part, four at a time.  80 workgroups for 5120 columns, so what bounds
// them is the way of a load: 512 parts 6.8 us, by four
// wavefronts 15.8.
constexpr int kParamWaves = 16;
__global__ __launch_bounds__(64 * kParamWaves) void k_norm_params(const float* parts, int64_t n, int64_t C,
                                                                  float* dweight, float* dbias) {
    __shared__ float s[2][kParamWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float w[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < C) {
        for (int64_t i = wave; i < n; i += 4 * kParamWaves) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t at = i + kParamWaves * k, j = at < n ? at : i;
                const float vw = parts[2 * j * C + c], vb = parts[(2 * j + 1) * C + c];
                w[k] += at < n ? vw : 0.f;
                b[k] += at < n ? vb : 0.f;
            }
        }
    }
    s[0][wave][lane] = (w[0] + w[1]) + (w[2] + w[3]);
    s[1][wave][lane] = (b[0] + b[1]) + (b[2] + b[3]);
    __syncthreads();
    if (wave < 2 && c < C) {
        float* out = wave == 0 ? dweight : dbias;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kParamWaves; ++k) sum += s[wave][k][lane];
        if (out) out[c] = sum;
    }
}

template <typename T, int V, int NP, bool BLOCK, bool BWD, bool WHOLE>
void go(const NormArgs& A, int gate, dim3 grid, int threads, hipStream_t st) {
    if (gate == 0) k_norm<T, V, NP, BLOCK, 0, BWD, WHOLE><<<grid, threads, 0, st>>>(A);
    else if (gate == 1) k_norm<T, V, NP, BLOCK, 1, BWD, WHOLE><<<grid, threads, 0, st>>>(A);
    else k_norm<T, V, NP, BLOCK, 2, BWD, WHOLE><<<grid, threads, 0, st>>>(A);
}
template <typename T, int V, int NP, bool BLOCK, bool BWD>
void go(const NormArgs& A, int gate, dim3 grid, int threads, hipStream_t st) {
    if (A.m % V == 0) go<T, V, NP, BLOCK, BWD, true>(A, gate, grid, threads, st);
    else if constexpr (V > 1) go<T, V, NP, BLOCK, BWD, false>(A, gate, grid, threads, st);
}

template <typename T, bool BWD> hipError_t run(const NormShape& s, const NormLayout& l, const NormArgs& A, hipStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int gate = !A.gate ? 0 : s.gate_first ? 2 : 1;
    const dim3 grid((unsigned)l.across, (unsigned)l.down);
    if (l.vec == 1) go<T, 1, 1, false, BWD>(A, gate, grid, l.threads, st);
    else if (!l.block) go<T, V, 1, false, BWD>(A, gate, grid, l.threads, st);
    else if (l.pieces == 1) go<T, V, 1, true, BWD>(A, gate, grid, l.threads, st);
    else if (l.pieces == 2) go<T, V, 2, true, BWD>(A, gate, grid, l.threads, st);
    else if constexpr (V == 4) go<T, V, 4, true, BWD>(A, gate, grid, l.threads, st);   // kNormMost / (1024 V)
    return hipGetLastError();
}

NormArgs norm_args(const NormShape& s, const NormLayout& l, const NormIn& in) {
    NormArgs A = {};
    A.x = in.x; A.gate = in.gate; A.weight = in.weight; A.bias = in.bias; A.lens = in.lens;
    A.rows = s.Bz * s.L; A.L = s.L; A.C = s.C;
    A.xb = s.xb; A.xr = s.xr; A.zb = s.zb; A.zr = s.zr;
    A.m = (int)(s.C / s.G); A.G = (int)s.G;
    A.lanes = l.lanes; A.gw = l.gw; A.rw = l.rw;
    A.eps = s.eps; A.size = (float)A.m; A.inv = 1.f / A.size; A.center = s.center; A.silu = s.silu;
    A.flat = !in.lens && (s.Bz == 1 || (s.xb == s.L * s.xr && (!in.gate || s.zb == s.L * s.zr)));
    return A;
}

}  // namespace

hipError_t launch_norm_fwd(const NormShape& s, const NormIn& in, void* y, hipStream_t st) {
    const NormLayout l = norm_layout(s, false);
    NormArgs A = norm_args(s, l, in);
    A.y = y;
    return s.bf16 ? run<u16, false>(s, l, A, st) : run<float, false>(s, l, A, st);
}

hipError_t launch_norm_bwd(const NormShape& s, const NormIn& in, const void* dy, void* dx, void* dgate, float* dweight,
                           float* dbias, float* parts, hipStream_t st) {
    const NormLayout l = norm_layout(s, true);
    NormArgs A = norm_args(s, l, in);
    A.dy = dy; A.dx = dx; A.dgate = dgate;
    A.parts = dweight || dbias ? parts : nullptr;
    hipError_t e = s.bf16 ? run<u16, true>(s, l, A, st) : run<float, true>(s, l, A, st);
    if (e != hipSuccess || !A.parts) return e;
    k_norm_params<<<(unsigned)((s.C + 63) / 64), 64 * kParamWaves, 0, st>>>(parts, norm_bwd_parts(s), s.C, dweight, dbias);
    return hipGetLastError();
}

}  // namespace ssd
