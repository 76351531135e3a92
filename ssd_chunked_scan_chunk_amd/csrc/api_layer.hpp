// api_layer.hpp -- the C ABI of the operators around the chunked scan: the short
// causal convolution and the per-channel scan.  Included once, at the end of
// api.cpp, whose error state and range checks it shares.
#include "layer_launch.hpp"

namespace {

constexpr int64_t kMaxSize = (int64_t)1 << 40;
constexpr int64_t kMaxRow = (int64_t)1 << 24;   // elements between steps of the per-channel scan's inputs

// bytes from the first to past the last element of rows of `n` elements at
// b * bs + t * rs
int64_t span_bytes(int64_t Bz, int64_t L, int64_t n, int64_t bs, int64_t rs, int64_t es) {
    return Bz > 0 && L > 0 ? ((Bz - 1) * bs + (L - 1) * rs + n) * es : 0;
}

// Bz batches at bs and L steps at rs elements stay within 2^41 elements
ssd_status check_stride(const char* name, int64_t Bz, int64_t bs, int64_t L, int64_t rs) {
    if (bs < 0 || rs < 0)
        return fail(SSD_ERR_SHAPE, "%s: strides must not be negative (got %lld, %lld)", name, (long long)bs,
                    (long long)rs);
    if ((Bz > 0 && bs > kMaxSize / Bz) || (L > 0 && rs > kMaxSize / L))
        return fail(SSD_ERR_UNSUPPORTED, "%s: strides beyond the supported range", name);
    return SSD_OK;
}

ssd_status check_disjoint(const Range* out, int no, const Range* in, int ni) {
    for (int o = 0; o < no; ++o) {
        for (int i = 0; i < ni; ++i)
            if (overlap(out[o], in[i])) return fail(SSD_ERR_ALIAS, "%s overlaps %s", out[o].name, in[i].name);
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out[q])) return fail(SSD_ERR_ALIAS, "%s overlaps %s", out[o].name, out[q].name);
    }
    return SSD_OK;
}

ssd_status check_aligned(const char* name, const void* p, size_t n) {
    if (p && !aligned(p, n)) return fail(SSD_ERR_ALIGN, "%s is not %zu-byte aligned", name, n);
    return SSD_OK;
}

#define SSD_CHECK(call)                          \
    do {                                         \
        const ssd_status st_ = (call);           \
        if (st_ != SSD_OK) return st_;           \
    } while (0)

ssd_status conv_shape(const ssd_conv_desc* d, ssd::ConvShape* s) {
    if (!d) return fail(SSD_ERR_NULL, "desc is NULL");
    if (d->batch < 0 || d->seqlen < 0 || d->channels < 1)
        return fail(SSD_ERR_SHAPE, "sizes must be batch>=0, seqlen>=0, channels>=1 (got %lld,%lld,%lld)",
                    (long long)d->batch, (long long)d->seqlen, (long long)d->channels);
    if (d->width < 2 || d->width > 4)
        return fail(SSD_ERR_UNSUPPORTED, "width must be 2, 3 or 4 (got %lld)", (long long)d->width);
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16)
        return fail(SSD_ERR_DTYPE, "dtype %d is not SSD_F32 or SSD_BF16", (int)d->dtype);
    if ((d->silu != 0 && d->silu != 1) || d->reserved != 0)
        return fail(SSD_ERR_SHAPE, "silu must be 0 or 1, reserved 0");
    if (d->npieces < 1 || d->npieces > 3) return fail(SSD_ERR_SHAPE, "npieces must be 1, 2 or 3");
    // the grid is (channel blocks x time blocks, batch) of 256 threads
    if (d->batch > 65535 || d->seqlen > ((int64_t)1 << 31) || d->channels > ((int64_t)1 << 24) ||
        d->batch * d->seqlen > kMaxSize / d->channels)
        return fail(SSD_ERR_UNSUPPORTED, "sizes beyond the supported range");
    SSD_CHECK(check_stride("x", d->batch, d->x_bstride, d->seqlen, d->x_rstride));
    int64_t sum = 0;
    for (int i = 0; i < 3; ++i) {
        s->piece[i] = i < d->npieces ? d->piece[i] : 0;
        if (i < d->npieces && (d->piece[i] < 1 || d->piece[i] > d->channels))
            return fail(SSD_ERR_SHAPE, "piece %d must be 1 .. channels wide (got %lld)", i, (long long)d->piece[i]);
        sum += s->piece[i];
    }
    if (sum != d->channels)
        return fail(SSD_ERR_SHAPE, "the pieces hold %lld channels, not %lld", (long long)sum, (long long)d->channels);
    s->Bz = d->batch; s->L = d->seqlen; s->C = d->channels; s->W = (int)d->width;
    s->xb = d->x_bstride; s->xr = d->x_rstride;
    s->bf16 = d->dtype == SSD_BF16; s->silu = d->silu == 1;
    // worst case of one channel per thread; the step's threads in workgroups of 256
    const int64_t blocks = ((s->C + 63) / 64) * ssd::conv_time_blocks(*s, ssd::conv_rows(*s, true));
    const int64_t fblocks = ((s->C + 63) / 64) * ssd::conv_time_blocks(*s, ssd::conv_rows(*s, false));
    if ((blocks > fblocks ? blocks : fblocks) * 256 >= ((int64_t)1 << 32) || s->Bz * s->C > ((int64_t)1 << 32) - 256)
        return fail(SSD_ERR_UNSUPPORTED, "seqlen*channels or batch*channels too large for one launch");
    return SSD_OK;
}

size_t conv_bwd_bytes(const ssd::ConvShape& s) {
    return s.Bz > 0 ? (size_t)ssd::conv_bwd_parts(s) * (s.W + 1) * s.C * sizeof(float) : 0;
}

// the pieces of y or dy: present, aligned; their ranges go to r
ssd_status check_pieces(const ssd::ConvShape& s, const char* name, const void* const* y, Range* r) {
    const int64_t es = s.bf16 ? 2 : 4;
    const bool empty = s.Bz == 0 || s.L == 0;
    for (int i = 0; i < 3; ++i) {
        const void* p = s.piece[i] && y ? y[i] : nullptr;
        if (s.piece[i] && !p && !empty) return fail(SSD_ERR_NULL, "%s: piece %d is NULL", name, i);
        SSD_CHECK(check_aligned(name, p, es));
        r[i] = rng(name, p, s.Bz * s.L * s.piece[i] * es);
    }
    return SSD_OK;
}

ssd_status chan_shape(const ssd_channel_desc* d, ssd::ChanShape* s) {
    if (!d) return fail(SSD_ERR_NULL, "desc is NULL");
    if (d->batch < 0 || d->seqlen < 0 || d->channels < 1 || d->dstate < 1 || d->ngroups < 1)
        return fail(SSD_ERR_SHAPE,
                    "sizes must be batch>=0, seqlen>=0, channels,dstate,ngroups>=1 (got %lld,%lld,%lld,%lld,%lld)",
                    (long long)d->batch, (long long)d->seqlen, (long long)d->channels, (long long)d->dstate,
                    (long long)d->ngroups);
    if (d->channels % d->ngroups != 0)
        return fail(SSD_ERR_SHAPE, "channels (%lld) must be a multiple of ngroups (%lld)", (long long)d->channels,
                    (long long)d->ngroups);
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16)
        return fail(SSD_ERR_DTYPE, "dtype %d is not SSD_F32 or SSD_BF16", (int)d->dtype);
    if (d->softplus != 0 && d->softplus != 1) return fail(SSD_ERR_SHAPE, "softplus must be 0 or 1");
    if (d->dstate > 64)
        return fail(SSD_ERR_UNSUPPORTED, "dstate must be at most 64 (got %lld)", (long long)d->dstate);
    // grid limits, and 32-bit steps and offsets inside a segment
    if (d->batch > 65535 || d->ngroups > 65535 || d->seqlen > ((int64_t)1 << 30) || d->channels > ((int64_t)1 << 20) ||
        d->batch * d->seqlen > kMaxSize / d->channels)
        return fail(SSD_ERR_UNSUPPORTED, "sizes beyond the supported range");
    SSD_CHECK(check_stride("u", d->batch, d->u_bstride, d->seqlen, d->u_rstride));
    SSD_CHECK(check_stride("delta", d->batch, d->delta_bstride, d->seqlen, d->delta_rstride));
    SSD_CHECK(check_stride("gate", d->batch, d->gate_bstride, d->seqlen, d->gate_rstride));
    SSD_CHECK(check_stride("B", d->batch, d->B_bstride, d->seqlen, d->B_rstride));
    SSD_CHECK(check_stride("C", d->batch, d->C_bstride, d->seqlen, d->C_rstride));
    // the per-state kernels launch a thread for every (batch, channel, state), of
    // channels rounded up to 64 for every group
    const int64_t padded = d->ngroups * ((d->channels / d->ngroups + 63) / 64 * 64);
    if (d->batch * padded * 64 >= ((int64_t)1 << 32))
        return fail(SSD_ERR_UNSUPPORTED, "batch*channels too large for one launch");
    s->Bz = d->batch; s->L = d->seqlen; s->D = d->channels; s->N = d->dstate; s->G = d->ngroups;
    s->ub = d->u_bstride; s->ur = d->u_rstride; s->db = d->delta_bstride; s->dr = d->delta_rstride;
    s->zb = d->gate_bstride; s->zr = d->gate_rstride;
    s->Bb = d->B_bstride; s->Br = d->B_rstride; s->Cb = d->C_bstride; s->Cr = d->C_rstride;
    // the kernels reach the rows of a batch of steps by 32-bit byte offsets
    int64_t* rows[] = {&s->ur, &s->dr, &s->zr, &s->Br, &s->Cr};
    for (int64_t* r : rows) {
        if (s->L <= 1) *r = 0;
        if (*r > kMaxRow) return fail(SSD_ERR_UNSUPPORTED, "step strides must be at most 2^24 elements");
    }
    s->bf16 = d->dtype == SSD_BF16; s->softplus = d->softplus == 1;
    return SSD_OK;
}

// u .. seqlens: present and aligned; their ranges go to r[0 .. 9]
constexpr int kChanIn = 10;
ssd_status check_chan_in(const ssd::ChanShape& s, const ssd::ChanIn& in, Range* r) {
    const int64_t es = s.bf16 ? 2 : 4;
    if (!in.A || (s.Bz > 0 && s.L > 0 && (!in.u || !in.delta || !in.B || !in.C)))
        return fail(SSD_ERR_NULL, "u, delta, A, B and C are required");
    SSD_CHECK(check_aligned("u", in.u, es));
    SSD_CHECK(check_aligned("delta", in.delta, es));
    SSD_CHECK(check_aligned("gate", in.gate, es));
    SSD_CHECK(check_aligned("B", in.B, es));
    SSD_CHECK(check_aligned("C", in.C, es));
    SSD_CHECK(check_aligned("A", in.A, 4));
    SSD_CHECK(check_aligned("skip", in.skip, 4));
    SSD_CHECK(check_aligned("delta_bias", in.dbias, 4));
    SSD_CHECK(check_aligned("initial_state", in.h0, 4));
    SSD_CHECK(check_aligned("seqlens", in.lens, 4));
    r[0] = rng("u", in.u, span_bytes(s.Bz, s.L, s.D, s.ub, s.ur, es));
    r[1] = rng("delta", in.delta, span_bytes(s.Bz, s.L, s.D, s.db, s.dr, es));
    r[2] = rng("gate", in.gate, span_bytes(s.Bz, s.L, s.D, s.zb, s.zr, es));
    r[3] = rng("B", in.B, span_bytes(s.Bz, s.L, s.G * s.N, s.Bb, s.Br, es));
    r[4] = rng("C", in.C, span_bytes(s.Bz, s.L, s.G * s.N, s.Cb, s.Cr, es));
    r[5] = rng("A", in.A, s.D * s.N * 4);
    r[6] = rng("skip", in.skip, s.D * 4);
    r[7] = rng("delta_bias", in.dbias, s.D * 4);
    r[8] = rng("initial_state", in.h0, s.Bz * s.D * s.N * 4);
    r[9] = rng("seqlens", in.lens, s.Bz * 4);
    return SSD_OK;
}

// The sums of dB and dC launch a thread for every (batch, step, group, B or C,
// padded state).
ssd_status check_chan_bwd(const ssd::ChanShape& s) {
    if (s.Bz * s.L > ((int64_t)1 << 31) / (s.G * 128))
        return fail(SSD_ERR_UNSUPPORTED, "batch*seqlen*ngroups too large for one launch of the backward");
    return SSD_OK;
}

ssd_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need > 0 && (!ws || have < need))
        return fail(SSD_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu%s)", need, have, ws ? "" : ", NULL");
    return need > 0 ? check_aligned("workspace", ws, 16) : SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_short_conv_fwd(const ssd_conv_desc* desc, const void* x, const float* weight, const float* bias,
                              const void* initial_window, const int32_t* seqlens, void* const* y,
                              void* final_window, void* stream) {
    ssd::ConvShape s;
    SSD_CHECK(conv_shape(desc, &s));
    if (s.Bz == 0) return ok();
    const int64_t es = s.bf16 ? 2 : 4, nw = s.Bz * (s.W - 1) * s.C * es;
    if (!weight || !y || (!x && s.L > 0)) return fail(SSD_ERR_NULL, "x, weight and y are required");
    SSD_CHECK(check_aligned("x", x, es));
    SSD_CHECK(check_aligned("weight", weight, 4));
    SSD_CHECK(check_aligned("bias", bias, 4));
    SSD_CHECK(check_aligned("initial_window", initial_window, es));
    SSD_CHECK(check_aligned("final_window", final_window, es));
    SSD_CHECK(check_aligned("seqlens", seqlens, 4));
    Range out[4];
    SSD_CHECK(check_pieces(s, "y", y, out));
    out[3] = rng("final_window", final_window, nw);
    const Range in[] = {rng("x", x, span_bytes(s.Bz, s.L, s.C, s.xb, s.xr, es)), rng("weight", weight, s.C * s.W * 4),
                        rng("bias", bias, s.C * 4), rng("initial_window", initial_window, nw),
                        rng("seqlens", seqlens, s.Bz * 4)};
    SSD_CHECK(check_disjoint(out, 4, in, 5));
    if (s.L == 0 && !final_window) return ok();
    const hipError_t e = ssd::launch_conv_fwd(s, x, weight, bias, initial_window, seqlens, y, final_window,
                                              reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "convolution forward launch");
}

ssd_status ssd_short_conv_bwd_workspace_bytes(const ssd_conv_desc* desc, size_t* bytes) {
    if (!bytes) return fail(SSD_ERR_NULL, "bytes is NULL");
    ssd::ConvShape s;
    SSD_CHECK(conv_shape(desc, &s));
    *bytes = conv_bwd_bytes(s);
    return ok();
}

ssd_status ssd_short_conv_bwd(const ssd_conv_desc* desc, const void* x, const float* weight, const float* bias,
                              const void* initial_window, const int32_t* seqlens, const void* const* dy,
                              const void* dfinal_window, void* dx, float* dweight, float* dbias,
                              void* dinitial_window, void* workspace, size_t workspace_bytes, void* stream) {
    ssd::ConvShape s;
    SSD_CHECK(conv_shape(desc, &s));
    const int64_t es = s.bf16 ? 2 : 4, nw = s.Bz * (s.W - 1) * s.C * es;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    if (!weight || !dy || !dweight || (s.Bz > 0 && s.L > 0 && (!x || !dx)))
        return fail(SSD_ERR_NULL, "x, weight, dy, dx and dweight are required");
    if (!bias != !dbias) return fail(SSD_ERR_NULL, "dbias is required exactly when bias is given");
    SSD_CHECK(check_aligned("x", x, es));
    SSD_CHECK(check_aligned("weight", weight, 4));
    SSD_CHECK(check_aligned("bias", bias, 4));
    SSD_CHECK(check_aligned("initial_window", initial_window, es));
    SSD_CHECK(check_aligned("dfinal_window", dfinal_window, es));
    SSD_CHECK(check_aligned("seqlens", seqlens, 4));
    SSD_CHECK(check_aligned("dx", dx, es));
    SSD_CHECK(check_aligned("dweight", dweight, 4));
    SSD_CHECK(check_aligned("dbias", dbias, 4));
    SSD_CHECK(check_aligned("dinitial_window", dinitial_window, es));
    const size_t need = conv_bwd_bytes(s);
    SSD_CHECK(check_workspace(workspace, workspace_bytes, need));
    Range in[9];
    SSD_CHECK(check_pieces(s, "dy", dy, in));
    in[3] = rng("x", x, span_bytes(s.Bz, s.L, s.C, s.xb, s.xr, es));
    in[4] = rng("weight", weight, s.C * s.W * 4);
    in[5] = rng("bias", bias, s.C * 4);
    in[6] = rng("initial_window", initial_window, nw);
    in[7] = rng("dfinal_window", dfinal_window, nw);
    in[8] = rng("seqlens", seqlens, s.Bz * 4);
    const Range out[] = {rng("dx", dx, s.Bz * s.L * s.C * es), rng("dweight", dweight, s.C * s.W * 4),
                         rng("dbias", dbias, s.C * 4), rng("dinitial_window", dinitial_window, nw),
                         rng("workspace", workspace, (int64_t)need)};
    SSD_CHECK(check_disjoint(out, 5, in, 9));
    hipError_t e;
    if (s.Bz == 0) {   // no rows: the parameters' gradients are zero
        e = ssd::launch_fill_zero(dweight, s.C * s.W, hs);
        if (e == hipSuccess && dbias) e = ssd::launch_fill_zero(dbias, s.C, hs);
        return e == hipSuccess ? ok() : hip_fail(e, "empty convolution gradient");
    }
    e = ssd::launch_conv_bwd(s, x, weight, bias, initial_window, seqlens, dy, dfinal_window, dx, dweight, dbias,
                             dinitial_window, static_cast<float*>(workspace), hs);
    return e == hipSuccess ? ok() : hip_fail(e, "convolution backward launch");
}

ssd_status ssd_short_conv_step(const ssd_conv_desc* desc, void* window, const void* x, const float* weight,
                               const float* bias, void* const* y, void* stream) {
    ssd::ConvShape s;
    SSD_CHECK(conv_shape(desc, &s));
    if (s.L != 1) return fail(SSD_ERR_SHAPE, "seqlen must be 1 (got %lld)", (long long)s.L);
    if (s.Bz == 0) return ok();
    const int64_t es = s.bf16 ? 2 : 4;
    if (!window || !x || !weight || !y) return fail(SSD_ERR_NULL, "window, x, weight and y are required");
    SSD_CHECK(check_aligned("window", window, es));
    SSD_CHECK(check_aligned("x", x, es));
    SSD_CHECK(check_aligned("weight", weight, 4));
    SSD_CHECK(check_aligned("bias", bias, 4));
    Range out[4];
    SSD_CHECK(check_pieces(s, "y", y, out));
    out[3] = rng("window", window, s.Bz * (s.W - 1) * s.C * es);
    const Range in[] = {rng("x", x, span_bytes(s.Bz, 1, s.C, s.xb, 0, es)), rng("weight", weight, s.C * s.W * 4),
                        rng("bias", bias, s.C * 4)};
    SSD_CHECK(check_disjoint(out, 4, in, 3));
    const hipError_t e = ssd::launch_conv_step(s, window, x, weight, bias, y, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "convolution step launch");
}

ssd_status ssd_channel_scan_fwd_workspace_bytes(const ssd_channel_desc* desc, size_t* bytes) {
    if (!bytes) return fail(SSD_ERR_NULL, "bytes is NULL");
    ssd::ChanShape s;
    SSD_CHECK(chan_shape(desc, &s));
    *bytes = ssd::chan_fwd_bytes(s, ssd::chan_fwd_plan(s));
    return ok();
}

ssd_status ssd_channel_scan_fwd(const ssd_channel_desc* desc, const void* u, const void* delta, const float* A,
                                const void* B, const void* C, const float* skip, const void* gate,
                                const float* delta_bias, const float* initial_state, const int32_t* seqlens, void* y,
                                float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
    ssd::ChanShape s;
    SSD_CHECK(chan_shape(desc, &s));
    const ssd::ChanIn in{u, delta, B, C, gate, A, skip, delta_bias, initial_state, seqlens};
    Range r[kChanIn];
    SSD_CHECK(check_chan_in(s, in, r));
    const int64_t es = s.bf16 ? 2 : 4;
    if (!y && s.Bz > 0 && s.L > 0) return fail(SSD_ERR_NULL, "y is required");
    SSD_CHECK(check_aligned("y", y, es));
    SSD_CHECK(check_aligned("final_state", final_state, 4));
    const ssd::ChanPlan p = ssd::chan_fwd_plan(s);
    const size_t need = ssd::chan_fwd_bytes(s, p);
    SSD_CHECK(check_workspace(workspace, workspace_bytes, need));
    const Range out[] = {rng("y", y, s.Bz * s.L * s.D * es), rng("final_state", final_state, s.Bz * s.D * s.N * 4),
                         rng("workspace", workspace, (int64_t)need)};
    SSD_CHECK(check_disjoint(out, 3, r, kChanIn));
    if (s.Bz == 0 || (s.L == 0 && !final_state)) return ok();
    const hipError_t e = ssd::launch_chan_fwd(s, p, in, y, final_state, need > 0 ? static_cast<float*>(workspace) : nullptr,
                                              reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "per-channel scan launch");
}

ssd_status ssd_channel_scan_bwd_workspace_bytes(const ssd_channel_desc* desc, size_t* bytes) {
    if (!bytes) return fail(SSD_ERR_NULL, "bytes is NULL");
    ssd::ChanShape s;
    SSD_CHECK(chan_shape(desc, &s));
    SSD_CHECK(check_chan_bwd(s));
    *bytes = ssd::chan_bwd_plan(s).off[9];
    return ok();
}

ssd_status ssd_channel_scan_bwd(const ssd_channel_desc* desc, const void* u, const void* delta, const float* A,
                                const void* B, const void* C, const float* skip, const void* gate,
                                const float* delta_bias, const float* initial_state, const int32_t* seqlens,
                                const void* dy, const float* dfinal_state, const ssd_channel_grads* grads,
                                void* workspace, size_t workspace_bytes, void* stream) {
    ssd::ChanShape s;
    SSD_CHECK(chan_shape(desc, &s));
    SSD_CHECK(check_chan_bwd(s));
    if (!grads) return fail(SSD_ERR_NULL, "grads is NULL");
    const ssd_channel_grads& o = *grads;
    const ssd::ChanIn in{u, delta, B, C, gate, A, skip, delta_bias, initial_state, seqlens};
    Range r[kChanIn + 2];
    SSD_CHECK(check_chan_in(s, in, r));
    const int64_t es = s.bf16 ? 2 : 4, nx = s.Bz * s.L * s.D * es, nbc = s.Bz * s.L * s.G * s.N * es;
    const int64_t nh = s.Bz * s.D * s.N * 4;
    if (!o.dA || (s.Bz > 0 && s.L > 0 && (!dy || !o.du || !o.ddelta || !o.dB || !o.dC)))
        return fail(SSD_ERR_NULL, "dy, du, ddelta, dA, dB and dC are required");
    if ((s.Bz > 0 && s.L > 0 && !gate != !o.dgate) || !skip != !o.dskip || !delta_bias != !o.ddelta_bias)
        return fail(SSD_ERR_NULL, "dgate, dskip and ddelta_bias are required exactly when their input is given");
    struct { const char* name; const void* p; size_t n; int64_t bytes; } const outs[] = {
        {"du", o.du, (size_t)es, nx}, {"ddelta", o.ddelta, (size_t)es, nx}, {"dgate", o.dgate, (size_t)es, nx},
        {"dB", o.dB, (size_t)es, nbc}, {"dC", o.dC, (size_t)es, nbc}, {"dA", o.dA, 4, s.D * s.N * 4},
        {"dskip", o.dskip, 4, s.D * 4}, {"ddelta_bias", o.ddelta_bias, 4, s.D * 4},
        {"dinitial_state", o.dinitial_state, 4, nh}};
    Range out[10];
    for (int i = 0; i < 9; ++i) {
        SSD_CHECK(check_aligned(outs[i].name, outs[i].p, outs[i].n));
        out[i] = rng(outs[i].name, outs[i].p, outs[i].bytes);
    }
    SSD_CHECK(check_aligned("dy", dy, es));
    SSD_CHECK(check_aligned("dfinal_state", dfinal_state, 4));
    r[kChanIn] = rng("dy", dy, nx);
    r[kChanIn + 1] = rng("dfinal_state", dfinal_state, nh);
    const ssd::ChanBwdPlan p = ssd::chan_bwd_plan(s);
    SSD_CHECK(check_workspace(workspace, workspace_bytes, p.off[9]));
    out[9] = rng("workspace", workspace, (int64_t)p.off[9]);
    SSD_CHECK(check_disjoint(out, 10, r, kChanIn + 2));
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (s.Bz == 0) {   // no rows: the parameters' gradients are zero
        e = ssd::launch_fill_zero(o.dA, s.D * s.N, hs);
        if (e == hipSuccess && o.dskip) e = ssd::launch_fill_zero(o.dskip, s.D, hs);
        if (e == hipSuccess && o.ddelta_bias) e = ssd::launch_fill_zero(o.ddelta_bias, s.D, hs);
        return e == hipSuccess ? ok() : hip_fail(e, "empty scan gradient");
    }
    const ssd::ChanGrads gr{o.du, o.ddelta, o.dgate, o.dB, o.dC, o.dA, o.dskip, o.ddelta_bias, o.dinitial_state};
    e = ssd::launch_chan_bwd(s, p, in, dy, dfinal_state, gr, workspace, hs);
    return e == hipSuccess ? ok() : hip_fail(e, "per-channel scan backward launch");
}

ssd_status ssd_channel_step(const ssd_channel_desc* desc, float* state, const void* u, const void* delta,
                            const float* A, const void* B, const void* C, const float* skip, const void* gate,
                            const float* delta_bias, void* y, void* stream) {
    ssd::ChanShape s;
    SSD_CHECK(chan_shape(desc, &s));
    if (s.L != 1) return fail(SSD_ERR_SHAPE, "seqlen must be 1 (got %lld)", (long long)s.L);
    const ssd::ChanIn in{u, delta, B, C, gate, A, skip, delta_bias, nullptr, nullptr};
    Range r[kChanIn];
    SSD_CHECK(check_chan_in(s, in, r));
    if (s.Bz == 0) return ok();
    const int64_t es = s.bf16 ? 2 : 4;
    if (!state || !y) return fail(SSD_ERR_NULL, "state and y are required");
    SSD_CHECK(check_aligned("state", state, 4));
    SSD_CHECK(check_aligned("y", y, es));
    const Range out[] = {rng("y", y, s.Bz * s.D * es), rng("state", state, s.Bz * s.D * s.N * 4)};
    SSD_CHECK(check_disjoint(out, 2, r, kChanIn));
    const hipError_t e = ssd::launch_chan_step(s, state, in, y, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "per-channel step launch");
}

}  // extern "C"
