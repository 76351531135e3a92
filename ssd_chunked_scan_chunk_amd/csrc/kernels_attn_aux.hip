// kernels_attn_aux.hip -- linear attention around its walks: the segments' states
// joined, gradients of shared keys and values added up, the single-token step.
#include "attn_util.hpp"

namespace ssd {
namespace {

// The states at the segments' ends, each from nothing but the first, to the states that
// the next segments start from: one thread walks an element over the segments.
__global__ __launch_bounds__(256) void k_attn_join(float* slots, const float* log_decay, const int32_t* lens, int64_t L,
                                                   int64_t H, int64_t nslots, int64_t steps, int64_t SE, unsigned blocks) {
    const int64_t s = blockIdx.x / blocks, e = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x;
    if (e >= SE) return;
    const int64_t len = attn_length(lens, s / H, L);
    const float f = decay_pow(log2_decay(log_decay[s % H]), (int)steps);   // every segment that another follows is whole
    float* p = slots + s * nslots * SE + e;
    float carry = 0.f;
    for (int64_t k = 0; k < nslots && (k + 1) * steps < len; ++k) {
        carry = k == 0 ? p[0] : fmaf(f, carry, p[k * SE]);
        p[k * SE] = carry;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_attn_share(const float* in, T* out, int64_t n, int each, int D) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t head = i / D;               // i: (row, shared head, element)
        const float* p = in + head * each * D + i % D;
        float v = 0.f;
        for (int k = 0; k < each; ++k) v += p[(int64_t)k * D];
        Elem<T>::store(out + i, v);
    }
}

// One token.  A wavefront takes the state's rows of one (batch, head) in turn, 64 lanes
// over the keys; HBM-bound by the state, read and written once.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_step(float* state, const T* q, const T* k, const T* v,
                                                   const float* log_decay, T* y, int H, int each, int Dk, int Dv,
                                                   int64_t qb, int64_t kb, int64_t vb, float scale) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t bh = blockIdx.x, b = bh / H;
    const int h = (int)(bh % H);
    const float f = decay_pow(log2_decay(log_decay[h]), 1);
    const T *qp = q + b * qb + (int64_t)h * Dk, *kp = k + b * kb + (int64_t)(h / each) * Dk;
    const T* vp = v + b * vb + (int64_t)(h / each) * Dv;
    float* S = state + bh * Dk * Dv;
    float qv[4], kv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane + 64 * i;
        qv[i] = c < Dk ? Elem<T>::load(qp + c) : 0.f;
        kv[i] = c < Dk ? Elem<T>::load(kp + c) : 0.f;
    }
    for (int x = blockIdx.y * 4 + wave; x < Dv; x += gridDim.y * 4) {
        const float xv = Elem<T>::load(vp + x);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane + 64 * i;
            if (c < Dk) {
                const float s = fmaf(xv, kv[i], f * S[(int64_t)x * Dk + c]);
                S[(int64_t)x * Dk + c] = s;
                sum = fmaf(s, qv[i], sum);
            }
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
        if (lane == 0) Elem<T>::store(y + bh * Dv + x, scale * sum);
    }
}

}  // namespace

hipError_t launch_attn_bf16(const AttnArgs& A, bool full, hipStream_t st);
hipError_t launch_attn_f32(const AttnArgs& A, bool full, hipStream_t st);

static AttnArgs attn_args(const AttnShape& s, const AttnPlan& pl, const AttnPass& p, const float* log_decay,
                          const int32_t* lens, float* slots, int64_t segs) {
    AttnArgs A;
    A.p = p; A.log_decay = log_decay; A.lens = lens; A.slots = slots;
    A.L = s.L; A.cps = (int)((pl.steps + attn_chunk(s.bf16, p.cd, p.xd) - 1) / attn_chunk(s.bf16, p.cd, p.xd)); A.nseg = (int)pl.nseg; A.walked = (unsigned)segs; A.H = (unsigned)s.H;
    A.slices = (unsigned)attn_slices(p.xd);
    A.items = (unsigned)(s.Bz * s.H * A.slices * segs);
    return A;
}

hipError_t launch_attn_states(const AttnShape& s, const AttnPlan& pl, const AttnPass& p, const float* log_decay,
                              const int32_t* lens, float* slots, hipStream_t st) {
    if (pl.nseg < 2) return hipSuccess;
    AttnArgs A = attn_args(s, pl, p, log_decay, lens, slots, pl.nseg - 1);
    const hipError_t e = s.bf16 ? launch_attn_bf16(A, false, st) : launch_attn_f32(A, false, st);
    if (e != hipSuccess) return e;
    const int64_t SE = s.Dk * s.Dv;
    const unsigned blocks = (unsigned)((SE + 255) / 256);
    k_attn_join<<<(unsigned)(s.Bz * s.H) * blocks, 256, 0, st>>>(slots, log_decay, lens, s.L, s.H, pl.nseg - 1,
                                                                 pl.steps, SE, blocks);
    return hipGetLastError();
}

hipError_t launch_attn_pass(const AttnShape& s, const AttnPlan& pl, const AttnPass& p, const float* log_decay,
                            const int32_t* lens, const float* slots, hipStream_t st) {
    const AttnArgs A = attn_args(s, pl, p, log_decay, lens, const_cast<float*>(slots), pl.nseg);
    return s.bf16 ? launch_attn_bf16(A, true, st) : launch_attn_f32(A, true, st);
}

hipError_t launch_attn_share(const float* in, void* out, int64_t rows, int64_t H, int64_t K, int64_t D, bool bf16,
                             hipStream_t st) {
    const int64_t n = rows * K * D;
    const unsigned grid = (unsigned)(n < (int64_t)65536 * 256 ? (n + 255) / 256 : 65536);
    if (bf16) k_attn_share<<<grid, 256, 0, st>>>(in, static_cast<u16*>(out), n, (int)(H / K), (int)D);
    else k_attn_share<<<grid, 256, 0, st>>>(in, static_cast<float*>(out), n, (int)(H / K), (int)D);
    return hipGetLastError();
}

hipError_t launch_attn_step(const AttnShape& s, float* state, const void* q, const void* k, const void* v,
                            const float* log_decay, void* y, hipStream_t st) {
    const dim3 grid((unsigned)(s.Bz * s.H), (unsigned)((s.Dv + 31) / 32));
    auto go = [&](auto t) {
        using T = decltype(t);
        k_attn_step<T><<<grid, 256, 0, st>>>(state, static_cast<const T*>(q), static_cast<const T*>(k),
                                             static_cast<const T*>(v), log_decay, static_cast<T*>(y), (int)s.H,
                                             (int)(s.H / s.K), (int)s.Dk, (int)s.Dv, s.qb, s.kb, s.vb, s.scale);
    };
    if (s.bf16) go(u16{});
    else go(float{});
    return hipGetLastError();
}

}  // namespace ssd
