// kernels_conv.hip -- the short causal convolution on gfx950: forward,
// backward and the single-token step.
//
// One filter of W taps (2..4) per channel along the sequence,
//     pre[t] = bias + sum_k w[k] x'[t - (W-1) + k],   y = silu(pre) or pre,
// with x' continued to the left by a window or zeros.  About one flop per byte:
// bound by HBM.  A thread owns four consecutive channels (one in pieces of fewer;
// eight in bf16 measured 3 to 5% slower, their registers leaving two wavefronts per
// SIMD in the backward) and walks `rows` steps with the
// last W-1 inputs in registers, so every input row is read once but for the W-1
// rows ahead of each walk; a wavefront's accesses are one contiguous run.
//
// Backward, with dpre[t] = dy[t] act'(pre[t]) (0 outside the sequence):
//     dx[t] = sum_k w[k] dpre[t + W-1 - k],  dw[k] = sum_t dpre[t] x'[t-(W-1)+k],
//     dbias = sum_t dpre[t].
// The walk recomputes pre, keeps the last W-1 dpre in registers and runs W-1
// steps past its rows to finish their dx.  dw and dbias are summed in registers
// along the walk, over the workgroup's four wavefronts in LDS, and over the
// workgroups by a second kernel in a fixed order.
#include "layer_launch.hpp"
#include "ssd_device.hpp"

namespace ssd {

namespace {

constexpr int kWaves = kConvWaves;   // consecutive in time

struct ConvArgs {
    int64_t L, C, xb, xr;
    int64_t end0, end1;      // first channels of the second and third piece
    int64_t pw[3];
    int64_t rows;            // steps of one wavefront's walk
    unsigned across, first1, first2;   // threads across the channels, the first of the second and third piece
    unsigned cblocks, tblocks;
};

// V consecutive elements of a row as stored.  Rows need no alignment beyond an
// element's: the hardware takes wide accesses anywhere.
template <typename T, int V> struct Row {
    T v[V];
};
template <typename T> struct Wide;
template <> struct Wide<u16> { typedef u16 type __attribute__((ext_vector_type(4), aligned(2))); };
template <> struct Wide<float> { typedef float type __attribute__((ext_vector_type(4), aligned(4))); };

template <typename T, int V> __device__ __forceinline__ Row<T, V> load_row(const T* p) {
    Row<T, V> r;
    if constexpr (V == 1) {
        r.v[0] = *p;
    } else {
        const typename Wide<T>::type q = *reinterpret_cast<const typename Wide<T>::type*>(p);
        __builtin_memcpy(&r, &q, sizeof(r));
    }
    return r;
}
template <typename T, int V> __device__ __forceinline__ void store_raw(T* p, const Row<T, V>& r) {
    if constexpr (V == 1) {
        *p = r.v[0];
    } else {
        typename Wide<T>::type q;
        __builtin_memcpy(&q, &r, sizeof(q));
        *reinterpret_cast<typename Wide<T>::type*>(p) = q;
    }
}
template <typename T, int V> __device__ __forceinline__ Row<T, V> zero_row() {
    Row<T, V> r;
    __builtin_memset(&r, 0, sizeof(r));
    return r;
}
template <int V> __device__ __forceinline__ void widen(const Row<float, V>& r, float* f) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = r.v[i];
}
template <int V> __device__ __forceinline__ void widen(const Row<u16, V>& r, float* f) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = bf_bits_to_f32(r.v[i]);
}
template <int V> __device__ __forceinline__ void store_row(float* p, const float* f) {
    Row<float, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = f[i];
    store_raw<float, V>(p, r);
}
template <int V> __device__ __forceinline__ void store_row(u16* p, const float* f) {
    Row<u16, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = f32_to_bf_bits(f[i]);
    store_raw<u16, V>(p, r);
}

// V * W consecutive filter taps and V biases
template <int V, int W>
__device__ __forceinline__ void load_filter(const float* __restrict__ weight, const float* __restrict__ bias,
                                            int64_t c, float (&w)[V][W], float (&bs)[V]) {
    float* wf = &w[0][0];
#pragma unroll
    for (int i = 0; i < V * W; i += V) widen<V>(load_row<float, V>(weight + c * W + i), wf + i);
    if (bias) {
        widen<V>(load_row<float, V>(bias + c), bs);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) bs[i] = 0.f;
    }
}

__device__ __forceinline__ float sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * v));
}

template <typename P> struct Pieces { P p[3]; };

// The V channels of thread t across: c of all, pc of their piece, which is pw wide.
// The last thread of a piece whose width V does not divide starts earlier and repeats
// some of its neighbour's channels, with the same results.
template <int V, typename P> struct Cut {
    int64_t c, pc, pw, left;   // left: channels from where the thread would have started
    P p;
    __device__ __forceinline__ Cut(const ConvArgs& a, const Pieces<P>& y, unsigned t) {
        const bool p1 = t >= a.first1, p2 = t >= a.first2;
        pw = p2 ? a.pw[2] : p1 ? a.pw[1] : a.pw[0];
        p = p2 ? y.p[2] : p1 ? y.p[1] : y.p[0];
        pc = (int64_t)(t - (p2 ? a.first2 : p1 ? a.first1 : 0)) * V;
        left = pw - pc;
        if (left < V) pc = pw - V;
        c = pc + (p2 ? a.end1 : p1 ? a.end0 : 0);
    }
};

__device__ __forceinline__ int64_t length_of(const int32_t* lens, int64_t b, int64_t L) {
    if (!lens) return L;
    const int64_t n = lens[b];
    return n < 0 ? 0 : n > L ? L : n;
}

// x' at step t - (W-1) .. t - 1 as stored: the window (or zeros) left of the
// sequence; steps at or past n are not read
template <typename T, int V, int W>
__device__ __forceinline__ void load_history(const T* xc, int64_t xr, const T* win0, int64_t C, int64_t t, int64_t n,
                                             Row<T, V> (&h)[W - 1]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t s = t - (W - 1) + j;
        h[j] = zero_row<T, V>();
        if (s >= 0) { if (s < n) h[j] = load_row<T, V>(xc + s * xr); }
        else if (win0) h[j] = load_row<T, V>(win0 + (s + W - 1) * C);
    }
}

template <typename T, int V, int W, bool SILU>
__global__ __launch_bounds__(64 * kWaves) void k_conv_fwd(ConvArgs a, const T* __restrict__ x,
                                                          const float* __restrict__ weight,
                                                          const float* __restrict__ bias,
                                                          const T* __restrict__ win0,
                                                          const int32_t* __restrict__ lens, Pieces<T*> y,
                                                          T* __restrict__ win1)
{
    constexpr int U = 8;   // rows in flight
    const unsigned cb = blockIdx.x % a.cblocks, tb = blockIdx.x / a.cblocks;
    const int64_t b = blockIdx.y;
    const unsigned across = cb * 64 + (threadIdx.x & 63);
    const int64_t t0 = ((int64_t)tb * kWaves + (threadIdx.x >> 6)) * a.rows;
    if (across >= a.across || (t0 >= a.L && t0 > 0)) return;
    const Cut<V, T*> cut(a, y, across);
    const int64_t c = cut.c, pw = cut.pw;
    const int64_t t1 = t0 + a.rows < a.L ? t0 + a.rows : a.L;
    const int64_t n = length_of(lens, b, a.L);
    const int64_t te = t1 < n ? t1 : n;      // steps t0 .. te are computed, te .. t1 are zero
    const T* xc = x + b * a.xb + c;
    const T* w0 = win0 ? win0 + b * (W - 1) * a.C + c : nullptr;
    T* yp = cut.p + b * a.L * pw + cut.pc;

    float w[V][W], bs[V];
    load_filter<V, W>(weight, bias, c, w, bs);
    Row<T, V> hist[W - 1];
    load_history<T, V, W>(xc, a.xr, w0, a.C, t0, n, hist);
    float xf[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) widen<V>(hist[j], xf[j]);

    for (int64_t t = t0; t < te; t += U) {
        Row<T, V> in[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (t + j < te) in[j] = load_row<T, V>(xc + (t + j) * a.xr);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (t + j < te) {
                widen<V>(in[j], xf[W - 1]);
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s = bs[v];
#pragma unroll
                    for (int k = 0; k < W; ++k) s = fmaf(w[v][k], xf[k][v], s);
                    o[v] = SILU ? s * sigmoid(s) : s;
                }
                store_row<V>(yp + (t + j) * pw, o);
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v) xf[k][v] = xf[k + 1][v];
            }
        }
    }
    const float zero[V] = {};
    for (int64_t t = te > t0 ? te : t0; t < t1; ++t) store_row<V>(yp + t * pw, zero);
    // the walk that reaches the sequence's end holds its last W-1 inputs
    if (win1 && ((te == n && te > t0) || (n == 0 && t0 == 0))) {
        T* w1 = win1 + b * (W - 1) * a.C + c;
        // xf[j] is exactly representable: it was widened from T
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_row<V>(w1 + j * a.C, xf[j]);
    }
}

template <typename T, int V, int W, bool SILU>
__global__ __launch_bounds__(64 * kWaves) void k_conv_bwd(ConvArgs a, const T* __restrict__ x,
                                                          const float* __restrict__ weight,
                                                          const float* __restrict__ bias,
                                                          const T* __restrict__ win0,
                                                          const int32_t* __restrict__ lens, Pieces<const T*> dy,
                                                          const T* __restrict__ dwin1, T* __restrict__ dx,
                                                          T* __restrict__ dwin0, float* __restrict__ parts)
{
    constexpr int U = 4;   // rows in flight
    constexpr int NA = V * (W + 1);
    __shared__ float red[(kWaves - 1) * NA * 64];
    const unsigned cb = blockIdx.x % a.cblocks, tb = blockIdx.x / a.cblocks;
    const int64_t b = blockIdx.y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool on = cb * 64 + lane < a.across;
    const Cut<V, const T*> cut(a, dy, on ? cb * 64 + lane : a.across - 1);
    const int64_t c = cut.c, pw = cut.pw;
    const int64_t t0 = ((int64_t)tb * kWaves + wave) * a.rows;
    float dw[V][W] = {}, db[V] = {};
    if (on && (t0 < a.L || t0 == 0)) {
        const int64_t t1 = t0 + a.rows < a.L ? t0 + a.rows : a.L;
        const int64_t n = length_of(lens, b, a.L);
        const T* xc = x + b * a.xb + c;
        const T* w0 = win0 ? win0 + b * (W - 1) * a.C + c : nullptr;
        const T* g1 = dwin1 ? dwin1 + b * (W - 1) * a.C + c : nullptr;
        T* g0 = dwin0 ? dwin0 + b * (W - 1) * a.C + c : nullptr;
        T* dxc = dx + b * a.L * a.C + c;
        const T* dyp = cut.p + b * a.L * pw + cut.pc;

        float w[V][W], bs[V];
        load_filter<V, W>(weight, bias, c, w, bs);
        Row<T, V> hist[W - 1];
        load_history<T, V, W>(xc, a.xr, w0, a.C, t0, n, hist);
        float xf[W][V], dp[W][V] = {};
#pragma unroll
        for (int j = 0; j < W - 1; ++j) widen<V>(hist[j], xf[j]);

        const int64_t tlast = t1 + W - 1;
        const int64_t te = t1 < n ? t1 : n;   // steps whose terms of dw and db are this walk's
        for (int64_t t = t0; t < tlast; t += U) {
            Row<T, V> in[U], gin[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                in[j] = gin[j] = zero_row<T, V>();
                if (t + j < n && t + j < tlast) {
                    in[j] = load_row<T, V>(xc + (t + j) * a.xr);
                    gin[j] = load_row<T, V>(dyp + (t + j) * pw);
                }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t r = t + j;
                if (r >= tlast) break;
                float g[V], o[V];
                widen<V>(in[j], xf[W - 1]);
                widen<V>(gin[j], g);
                // of these alone: past the end d is 0, but the inputs may be infinite or NaN
                const bool own = r < te;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float d = g[v];
                    if constexpr (SILU) {
                        float s = bs[v];
#pragma unroll
                        for (int k = 0; k < W; ++k) s = fmaf(w[v][k], xf[k][v], s);
                        const float sg = sigmoid(s);
                        d *= sg * fmaf(s, 1.f - sg, 1.f);
                    }
                    d = r < n ? d : 0.f;
                    dp[W - 1][v] = d;
                    if (own) {
                        db[v] += d;
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[v][k] = fmaf(d, xf[k][v], dw[v][k]);
                    }
                    // row r of the sequence with its window ahead: steps r-(W-1) .. r
                    float s = 0.f;
#pragma unroll
                    for (int k = 0; k < W; ++k) s = fmaf(w[v][k], dp[W - 1 - k][v], s);
                    o[v] = s;
                }
                if (g1 && r >= n && r < n + W - 1) {
                    float e[V];
                    widen<V>(load_row<T, V>(g1 + (r - n) * a.C), e);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] += e[v];
                }
                if (r >= t0 + W - 1) store_row<V>(dxc + (r - (W - 1)) * a.C, o);
                else if (t0 == 0 && g0) store_row<V>(g0 + r * a.C, o);
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v) { xf[k][v] = xf[k + 1][v]; dp[k][v] = dp[k + 1][v]; }
            }
        }
    }
    // sum over the workgroup's wavefronts, in their order
    if (wave > 0) {
        float* q = red + (wave - 1) * NA * 64 + lane;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int k = 0; k < W; ++k) q[(k * V + v) * 64] = dw[v][k];
            q[(W * V + v) * 64] = db[v];
        }
    }
    __syncthreads();
    if (wave == 0 && on) {
        float* out = parts + ((int64_t)b * a.tblocks + tb) * (W + 1) * a.C + c;
#pragma unroll
        for (int k = 0; k <= W; ++k) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = k < W ? dw[v][k < W ? k : 0] : db[v];
#pragma unroll
                for (int q = 0; q < kWaves - 1; ++q) s += red[(q * NA + k * V + v) * 64 + lane];
                out[(int64_t)k * a.C + v] = s;
            }
        }
    }
}

// dweight and dbias from the workgroups' parts [np][W + 1][C]: a workgroup
// sums 64 columns, its wavefronts every kWaves-th part, in a fixed order
__global__ __launch_bounds__(64 * kWaves) void k_conv_sum(const float* __restrict__ parts, int64_t np, int64_t C,
                                                          int W, float* __restrict__ dweight,
                                                          float* __restrict__ dbias)
{
    __shared__ float red[kWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane, cols = (int64_t)(W + 1) * C;
    float s = 0.f;
    if (col < cols) {
        int64_t p = wave;
        for (; p + 3 * kWaves < np; p += 4 * kWaves) {
            const float v0 = parts[p * cols + col], v1 = parts[(p + kWaves) * cols + col];
            const float v2 = parts[(p + 2 * kWaves) * cols + col], v3 = parts[(p + 3 * kWaves) * cols + col];
            s += (v0 + v1) + (v2 + v3);
        }
        for (; p < np; p += kWaves) s += parts[p * cols + col];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < cols) {
        s = red[0][lane];
#pragma unroll
        for (int q = 1; q < kWaves; ++q) s += red[q][lane];
        const int64_t k = col / C, c = col - k * C;
        if (k < W) dweight[c * W + k] = s;
        else if (dbias) dbias[c] = s;
    }
}

template <typename T, int V, int W, bool SILU>
__device__ __forceinline__ void conv_step(const ConvArgs& a, T* wp, const T* xp, const float* __restrict__ weight,
                                          const float* __restrict__ bias, int64_t c, T* yp)
{
    Row<T, V> in[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k] = load_row<T, V>(wp + k * a.C);
    in[W - 1] = load_row<T, V>(xp);
    float w[V][W], o[V];
    load_filter<V, W>(weight, bias, c, w, o);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float f[V];
        widen<V>(in[k], f);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(w[v][k], f[v], o[v]);
    }
    if constexpr (SILU) {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= sigmoid(o[v]);
    }
    store_row<V>(yp, o);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_raw<T, V>(wp + k * a.C, in[k + 1]);
}

template <typename T, int V, int W, bool SILU>
__global__ __launch_bounds__(256) void k_conv_step(ConvArgs a, T* __restrict__ window, const T* __restrict__ x,
                                                   const float* __restrict__ weight, const float* __restrict__ bias,
                                                   Pieces<T*> y, int64_t items)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items) return;
    const int64_t b = i / a.across;
    const Cut<V, T*> cut(a, y, (unsigned)(i - b * a.across));
    T* wp = window + b * (W - 1) * a.C;
    const T* xp = x + b * a.xb;
    T* yp = cut.p + b * cut.pw;
    if (cut.left >= V) {
        conv_step<T, V, W, SILU>(a, wp + cut.c, xp + cut.c, weight, bias, cut.c, yp + cut.pc);
    } else {   // in place: no channel may be shifted twice
        for (int64_t k = V - cut.left; k < V; ++k)
            conv_step<T, 1, W, SILU>(a, wp + cut.c + k, xp + cut.c + k, weight, bias, cut.c + k, yp + cut.pc + k);
    }
}

ConvArgs args_of(const ConvShape& s, int vec, int64_t rows) {
    ConvArgs a;
    a.L = s.L; a.C = s.C; a.xb = s.xb; a.xr = s.xr;
    a.end0 = s.piece[1] ? s.piece[0] : s.C;
    a.end1 = s.piece[2] ? s.piece[0] + s.piece[1] : s.C;
    for (int i = 0; i < 3; ++i) a.pw[i] = s.piece[i];
    a.rows = rows;
    const auto threads = [&](int i) { return (unsigned)((s.piece[i] + vec - 1) / vec); };
    a.first1 = threads(0);
    a.first2 = a.first1 + threads(1);
    a.across = a.first2 + threads(2);
    a.cblocks = (a.across + 63) / 64;
    a.tblocks = (unsigned)conv_time_blocks(s, rows);
    return a;
}

// run f(T, V, W, SILU) for the shape's types and sizes
template <typename T, int V, typename F> hipError_t by_width(const ConvShape& s, F f) {
    if (s.silu) {
        if (s.W == 4) return f.template go<T, V, 4, true>();
        if (s.W == 3) return f.template go<T, V, 3, true>();
        return f.template go<T, V, 2, true>();
    }
    if (s.W == 4) return f.template go<T, V, 4, false>();
    if (s.W == 3) return f.template go<T, V, 3, false>();
    return f.template go<T, V, 2, false>();
}
template <typename F> hipError_t by_type(const ConvShape& s, int vec, F f) {
    if (s.bf16) return vec > 1 ? by_width<u16, 4>(s, f) : by_width<u16, 1>(s, f);
    return vec > 1 ? by_width<float, 4>(s, f) : by_width<float, 1>(s, f);
}

template <typename T, typename P> Pieces<T> pieces_of(const ConvShape& s, const P* y) {
    Pieces<T> p;
    for (int i = 0; i < 3; ++i) p.p[i] = s.piece[i] ? (T)y[i] : nullptr;
    return p;
}

struct FwdCall {
    const ConvShape& s;
    ConvArgs a;
    const void* x;
    const float *weight, *bias;
    const void* win0;
    const int32_t* lens;
    void* const* y;
    void* win1;
    hipStream_t st;
    template <typename T, int V, int W, bool SILU> hipError_t go() {
        hipLaunchKernelGGL((k_conv_fwd<T, V, W, SILU>), dim3(a.cblocks * a.tblocks, (unsigned)s.Bz), dim3(64 * kWaves),
                           0, st, a, (const T*)x, weight, bias, (const T*)win0, lens, (pieces_of<T*>(s, y)), (T*)win1);
        return hipGetLastError();
    }
};
struct BwdCall {
    const ConvShape& s;
    ConvArgs a;
    const void* x;
    const float *weight, *bias;
    const void* win0;
    const int32_t* lens;
    const void* const* dy;
    const void* dwin1;
    void *dx, *dwin0;
    float* parts;
    hipStream_t st;
    template <typename T, int V, int W, bool SILU> hipError_t go() {
        hipLaunchKernelGGL((k_conv_bwd<T, V, W, SILU>), dim3(a.cblocks * a.tblocks, (unsigned)s.Bz), dim3(64 * kWaves),
                           0, st, a, (const T*)x, weight, bias, (const T*)win0, lens, (pieces_of<const T*>(s, dy)),
                           (const T*)dwin1, (T*)dx, (T*)dwin0, parts);
        return hipGetLastError();
    }
};
struct StepCall {
    const ConvShape& s;
    ConvArgs a;
    void* window;
    const void* x;
    const float *weight, *bias;
    void* const* y;
    hipStream_t st;
    template <typename T, int V, int W, bool SILU> hipError_t go() {
        const int64_t items = s.Bz * a.across;
        hipLaunchKernelGGL((k_conv_step<T, V, W, SILU>), dim3((unsigned)((items + 255) / 256)), dim3(256), 0, st, a,
                           (T*)window, (const T*)x, weight, bias, (pieces_of<T*>(s, y)), items);
        return hipGetLastError();
    }
};

}  // namespace

hipError_t launch_conv_fwd(const ConvShape& s, const void* x, const float* weight, const float* bias,
                           const void* win0, const int32_t* lens, void* const* y, void* win1, hipStream_t st)
{
    const int vec = conv_vec(s);
    return by_type(s, vec, FwdCall{s, args_of(s, vec, conv_rows(s, false)), x, weight, bias, win0, lens, y, win1, st});
}

hipError_t launch_conv_bwd(const ConvShape& s, const void* x, const float* weight, const float* bias,
                           const void* win0, const int32_t* lens, const void* const* dy, const void* dwin1,
                           void* dx, float* dweight, float* dbias, void* dwin0, float* parts, hipStream_t st)
{
    const int vec = conv_vec(s);
    hipError_t e = by_type(s, vec, BwdCall{s, args_of(s, vec, conv_rows(s, true)), x, weight, bias, win0, lens,
                                           dy, dwin1, dx, dwin0, parts, st});
    if (e != hipSuccess) return e;
    const int64_t cols = (s.W + 1) * s.C;
    hipLaunchKernelGGL(k_conv_sum, dim3((unsigned)((cols + 63) / 64)), dim3(64 * kWaves), 0, st, parts,
                       conv_bwd_parts(s), s.C, s.W, dweight, dbias);
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvShape& s, void* window, const void* x, const float* weight,
                            const float* bias, void* const* y, hipStream_t st)
{
    const int vec = conv_vec(s);
    return by_type(s, vec, StepCall{s, args_of(s, vec, 1), window, x, weight, bias, y, st});
}

}  // namespace ssd
