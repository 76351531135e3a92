// kernels_attn_aux.hip -- linear attention around its walks: the segments' states
// joined, gradients of shared keys and values added up, the single-token step.
#include "attn_util.hpp"

namespace ssd {
namespace {

template <int V> struct StepVec;
template <> struct StepVec<4> { typedef f32x4_any type; };
template <> struct StepVec<1> { typedef float type __attribute__((ext_vector_type(1))); };

// The states at the segments' ends, each from nothing but the first, to the states that
// the next segments start from: one thread walks V elements over the segments, four where a
// state holds whole fours (64 pairs of 128 x 128 in four segments: 6.4 us, one by one 15).
template <int V>
__global__ __launch_bounds__(256) void k_attn_join(float* slots0, float* slots1, const float* log_decay,
                                                   const int32_t* lens, int64_t L, int64_t H, int64_t whole,
                                                   int64_t nslots, int64_t steps, int64_t SE, unsigned blocks) {
    using F = typename StepVec<V>::type;
    float* slots = blockIdx.y ? slots1 : slots0;
    const int64_t i = blockIdx.x / blocks, s = whole + i, e = ((int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x) * V;
    if (e >= SE) return;
    const int64_t len = attn_length(lens, s / H, L);
    const float f = decay_pow(log2_decay(log_decay[s % H]), (int)steps);   // every segment that another follows is whole
    float* p = slots + i * nslots * SE + e;
    // as many as have steps after them; eight reads in flight
    int64_t n = len > 0 ? (len - 1) / steps : 0;
    if (n > nslots) n = nslots;
    F carry = {};
    for (int64_t k = 0; k < n; k += 8) {
        F v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const F*>(p + (k + j < n ? k + j : n - 1) * SE);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k + j >= n) break;
#pragma unroll
            for (int x = 0; x < V; ++x) carry[x] = k + j == 0 ? v[0][x] : fmaf(f, carry[x], v[j][x]);
            *reinterpret_cast<F*>(p + (k + j) * SE) = carry;
        }
    }
}

// Gradients of shared keys (blockIdx.y 0) and values (1): sums over the heads that share, V
// elements to a thread (3 x 1301 steps of 16 heads on 4 of 64 x 64: 6.2 us, one by one 9.3).
template <typename T, int V>
__global__ __launch_bounds__(256) void k_attn_share(const float* in0, const float* in1, T* out0, T* out1, int64_t heads,
                                                    int each, int D0, int D1) {
    using F = typename StepVec<V>::type;
    const float* in = blockIdx.y ? in1 : in0;
    T* out = blockIdx.y ? out1 : out0;
    const int D = blockIdx.y ? D1 : D0;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < heads * D; i += (int64_t)gridDim.x * 256 * V) {
        const int64_t head = i / D;               // i: (row, shared head, element)
        const float* p = in + head * each * D + i % D;
        F v = {};
        for (int k = 0; k < each; ++k) v += *reinterpret_cast<const F*>(p + (int64_t)k * D);
        if constexpr (V == 1) Elem<T>::store(out + i, v[0]);
        else if constexpr (sizeof(T) == 4) *reinterpret_cast<F*>(out + i) = v;
        else *reinterpret_cast<u32x2_any*>(out + i) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
    }
}

// One token: S <- gamma S + v k^T, y = scale S q.  HBM-bound by the state, read and written
// once: 16 bytes to a lane, `lanes` of them (a power of two) to a row of keys, so that a
// wavefront has 64 / lanes rows at a time and kUnroll such groups in flight.  256 requests of 40
// heads of 128 x 128: 5.7 TB/s, 4 bytes to a lane 2.6.
__device__ __forceinline__ float row_sum(float v, int lanes) {
    for (int d = 1; d < lanes; d *= 2) v += __shfl_xor(v, d, 64);
    return v;
}

constexpr int kUnroll = 8;
template <typename T, int V>
__global__ __launch_bounds__(256) void k_attn_step(float* state, const T* q, const T* k, const T* v,
                                                   const float* log_decay, T* y, int H, int each, int Dk, int Dv,
                                                   int lanes, int64_t qb, int64_t kb, int64_t vb, float scale) {
    using F = typename StepVec<V>::type;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned bh = blockIdx.x, b = bh / (unsigned)H, h = bh % (unsigned)H;
    const float f = decay_pow(log2_decay(log_decay[h]), 1);
    const T *qp = q + b * qb + (int64_t)h * Dk, *kp = k + b * kb + (int64_t)(h / each) * Dk;
    const T* vp = v + b * vb + (int64_t)(h / each) * Dv;
    // the last piece of a row whose length is no multiple of V starts early, its first
    // `skip` elements being another lane's
    const int want = lane % lanes * V, most = Dk - V, at = want < most ? want : most;
    const int skip = want < Dk ? want - at : V;
    float qv[V], kv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        qv[i] = i >= skip ? Elem<T>::load(qp + at + i) : 0.f;
        kv[i] = Elem<T>::load(kp + at + i);
    }
    const int rows = 64 / lanes, first = (blockIdx.y * 4 + wave) * rows * kUnroll + lane / lanes;
    float* S = state + (int64_t)bh * Dk * Dv + at;
    F s[kUnroll];
    float x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int r = first + u * rows, c = r < Dv ? r : Dv - 1;
        s[u] = __builtin_nontemporal_load(reinterpret_cast<const F*>(S + (int64_t)c * Dk));
        x[u] = Elem<T>::load(vp + c);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int r = first + u * rows;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[u][i] = fmaf(x[u], kv[i], f * s[u][i]);
            sum = i >= skip ? fmaf(s[u][i], qv[i], sum) : sum;
        }
        sum = row_sum(sum, lanes);
        if (r >= Dv) continue;
        if (skip == 0) {
            __builtin_nontemporal_store(s[u], reinterpret_cast<F*>(S + (int64_t)r * Dk));
        } else {
#pragma unroll
            for (int i = 1; i < V; ++i)
                if (i >= skip) S[(int64_t)r * Dk + i] = s[u][i];
        }
        if (lane % lanes == 0) Elem<T>::store(y + (int64_t)bh * Dv + r, scale * sum);
    }
}

}  // namespace

hipError_t launch_attn_bf16(const AttnArgs& A, bool full, hipStream_t st);
hipError_t launch_attn_f32(const AttnArgs& A, bool full, hipStream_t st);

static hipError_t launch_walks(const AttnShape& s, const AttnPlan& pl, const AttnPass* p, float* const* slots, int n,
                               const float* log_decay, const int32_t* lens, bool full, hipStream_t st) {
    AttnArgs A = {};
    const int64_t chunk = attn_chunk(s.bf16, p[0].cd, p[0].xd);
    for (int i = 0; i < n; ++i) {
        A.p[i] = p[i];
        A.slots[i] = slots[i];
    }
    A.log_decay = log_decay; A.lens = lens; A.L = s.L;
    A.cps = (int)((pl.steps + chunk - 1) / chunk);
    A.nseg = (int)pl.nseg;
    A.walks = (unsigned)n; A.H = (unsigned)s.H;
    A.slices = (unsigned)attn_slices(p[0].xd);
    A.pairs = (unsigned)(s.Bz * s.H);
    A.whole = (unsigned)pl.whole;
    A.segs = (unsigned)(full ? pl.nseg : pl.nseg - 1);
    if (!full) A.skip_whole = 1;
    return s.bf16 ? launch_attn_bf16(A, full, st) : launch_attn_f32(A, full, st);
}

// walks whose rows have the same sizes share a launch
static bool same_instance(const AttnPass& p, const AttnPass& q) {
    return attn_width(p.cd) == attn_width(q.cd) && attn_columns(p.xd) == attn_columns(q.xd) &&
           attn_slices(p.xd) == attn_slices(q.xd);
}
static hipError_t launch_grouped(const AttnShape& s, const AttnPlan& pl, const AttnPass* p, float* const* slots, int n,
                                 const float* log_decay, const int32_t* lens, bool full, hipStream_t st) {
    for (int i = 0; i < n;) {
        int k = i + 1;
        while (k < n && same_instance(p[i], p[k])) ++k;
        const hipError_t e = launch_walks(s, pl, p + i, slots + i, k - i, log_decay, lens, full, st);
        if (e != hipSuccess) return e;
        i = k;
    }
    return hipSuccess;
}

hipError_t launch_attn_states(const AttnShape& s, const AttnPlan& pl, const AttnPass* p, float* const* slots, int n,
                              const float* log_decay, const int32_t* lens, hipStream_t st) {
    const int64_t cut = s.Bz * s.H - pl.whole;
    if (pl.nseg < 2 || cut < 1) return hipSuccess;
    const hipError_t e = launch_grouped(s, pl, p, slots, n, log_decay, lens, false, st);
    if (e != hipSuccess) return e;
    const int64_t SE = s.Dk * s.Dv;
    const bool four = SE % 4 == 0;
    const unsigned blocks = (unsigned)((SE + (four ? 1023 : 255)) / (four ? 1024 : 256));
    auto join = four ? k_attn_join<4> : k_attn_join<1>;
    join<<<dim3((unsigned)cut * blocks, (unsigned)n), 256, 0, st>>>(
        slots[0], n > 1 ? slots[1] : nullptr, log_decay, lens, s.L, s.H, pl.whole, pl.nseg - 1, pl.steps, SE, blocks);
    return hipGetLastError();
}

hipError_t launch_attn_walks(const AttnShape& s, const AttnPlan& pl, const AttnPass* p, float* const* slots, int n,
                             const float* log_decay, const int32_t* lens, hipStream_t st) {
    return launch_grouped(s, pl, p, slots, n, log_decay, lens, true, st);
}

hipError_t launch_attn_share(const AttnShape& s, const float* dk_heads, const float* dv_heads, void* dk, void* dv,
                             hipStream_t st) {
    const int V = s.Dk % 4 == 0 && s.Dv % 4 == 0 ? 4 : 1;
    const int64_t heads = s.Bz * s.L * s.K, n = (heads * (s.Dk > s.Dv ? s.Dk : s.Dv) + 256 * V - 1) / (256 * V);
    const dim3 grid((unsigned)(n < 65536 ? n : 65536), 2);
    auto run = [&](auto kernel, auto* k, auto* v) {
        kernel<<<grid, 256, 0, st>>>(dk_heads, dv_heads, k, v, heads, (int)(s.H / s.K), (int)s.Dk, (int)s.Dv);
    };
    if (s.bf16) run(V == 4 ? k_attn_share<u16, 4> : k_attn_share<u16, 1>, static_cast<u16*>(dk), static_cast<u16*>(dv));
    else run(V == 4 ? k_attn_share<float, 4> : k_attn_share<float, 1>, static_cast<float*>(dk), static_cast<float*>(dv));
    return hipGetLastError();
}

hipError_t launch_attn_step(const AttnShape& s, float* state, const void* q, const void* k, const void* v,
                            const float* log_decay, void* y, hipStream_t st) {
    const int V = s.Dk < 4 ? 1 : 4;
    int lanes = 1;
    while (lanes * V < s.Dk) lanes *= 2;
    const int64_t rows = 64 / lanes * kUnroll * 4;
    const dim3 grid((unsigned)(s.Bz * s.H), (unsigned)((s.Dv + rows - 1) / rows));
    auto go = [&](auto t) {
        using T = decltype(t);
        auto run = [&](auto kernel) {
            kernel<<<grid, 256, 0, st>>>(state, static_cast<const T*>(q), static_cast<const T*>(k),
                                         static_cast<const T*>(v), log_decay, static_cast<T*>(y), (int)s.H,
                                         (int)(s.H / s.K), (int)s.Dk, (int)s.Dv, lanes, s.qb, s.kb, s.vb, s.scale);
        };
        if (V == 4) run(k_attn_step<T, 4>);
        else run(k_attn_step<T, 1>);
    };
    if (s.bf16) go(u16{});
    else go(float{});
    return hipGetLastError();
}

}  // namespace ssd
