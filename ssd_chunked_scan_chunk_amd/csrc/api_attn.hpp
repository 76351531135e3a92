// api_attn.hpp -- the C ABI of linear attention with a decay per head and of the norm
// over groups of channels.  Included once, at the end of api.cpp, after
// api_layer.hpp, whose checks it shares.
#include "attn_launch.hpp"

namespace {

ssd_status attn_shape(const ssd_linear_attn_desc* d, ssd::AttnShape* s) {
    if (!d) return fail(SSD_ERR_NULL, "desc is NULL");
    if (d->batch < 0 || d->seqlen < 0 || d->nheads < 1 || d->kv_heads < 1 || d->key_dim < 1 || d->value_dim < 1)
        return fail(SSD_ERR_SHAPE,
                    "sizes must be batch>=0, seqlen>=0, nheads,kv_heads,key_dim,value_dim>=1 "
                    "(got %lld,%lld,%lld,%lld,%lld,%lld)",
                    (long long)d->batch, (long long)d->seqlen, (long long)d->nheads, (long long)d->kv_heads,
                    (long long)d->key_dim, (long long)d->value_dim);
    if (d->nheads % d->kv_heads != 0)
        return fail(SSD_ERR_SHAPE, "nheads (%lld) must be a multiple of kv_heads (%lld)", (long long)d->nheads,
                    (long long)d->kv_heads);
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16)
        return fail(SSD_ERR_DTYPE, "dtype %d is not SSD_F32 or SSD_BF16", (int)d->dtype);
    if (d->key_dim > 256 || d->value_dim > 256)
        return fail(SSD_ERR_UNSUPPORTED, "key_dim and value_dim must be at most 256 (got %lld, %lld)",
                    (long long)d->key_dim, (long long)d->value_dim);
    if (d->batch > 65535 || d->nheads > 65535 || d->seqlen > ((int64_t)1 << 30) ||
        d->batch * d->seqlen > kMaxSize / (d->nheads * 256))
        return fail(SSD_ERR_UNSUPPORTED, "sizes beyond the supported range");
    SSD_CHECK(check_stride("q", d->batch, d->q_bstride, d->seqlen, d->q_rstride));
    SSD_CHECK(check_stride("k", d->batch, d->k_bstride, d->seqlen, d->k_rstride));
    SSD_CHECK(check_stride("v", d->batch, d->v_bstride, d->seqlen, d->v_rstride));
    s->Bz = d->batch; s->L = d->seqlen; s->H = d->nheads; s->K = d->kv_heads; s->Dk = d->key_dim; s->Dv = d->value_dim;
    s->qb = d->q_bstride; s->qr = d->q_rstride; s->kb = d->k_bstride; s->kr = d->k_rstride;
    s->vb = d->v_bstride; s->vr = d->v_rstride;
    s->bf16 = d->dtype == SSD_BF16; s->scale = d->scale;
    // the kernels reach the rows of a chunk by 32-bit offsets
    int64_t* rows[] = {&s->qr, &s->kr, &s->vr};
    for (int64_t* r : rows) {
        if (s->L <= 1) *r = 0;
        if (*r > kMaxRow) return fail(SSD_ERR_UNSUPPORTED, "step strides must be at most 2^24 elements");
    }
    if (s->H * 256 > kMaxRow) return fail(SSD_ERR_UNSUPPORTED, "nheads too large");
    // grids: up to 512 threads for each of two slices of columns of the backward's three walks
    // of every (batch, head); a plan keeps what it cuts into segments below this as well
    if (s->Bz * s->H > ssd::kAttnGroups / 6)
        return fail(SSD_ERR_UNSUPPORTED, "batch*nheads too large for one launch");
    return SSD_OK;
}

constexpr int kAttnIn = 6;
ssd_status check_attn_in(const ssd::AttnShape& s, const void* q, const void* k, const void* v, const float* log_decay,
                         const float* first, const int32_t* lens, Range* r) {
    const int64_t es = s.bf16 ? 2 : 4;
    if (!log_decay || (s.Bz > 0 && s.L > 0 && (!q || !k || !v)))
        return fail(SSD_ERR_NULL, "q, k, v and log_decay are required");
    SSD_CHECK(check_aligned("q", q, es));
    SSD_CHECK(check_aligned("k", k, es));
    SSD_CHECK(check_aligned("v", v, es));
    SSD_CHECK(check_aligned("log_decay", log_decay, 4));
    SSD_CHECK(check_aligned("initial_state", first, 4));
    SSD_CHECK(check_aligned("seqlens", lens, 4));
    r[0] = rng("q", q, span_bytes(s.Bz, s.L, s.H * s.Dk, s.qb, s.qr, es));
    r[1] = rng("k", k, span_bytes(s.Bz, s.L, s.K * s.Dk, s.kb, s.kr, es));
    r[2] = rng("v", v, span_bytes(s.Bz, s.L, s.K * s.Dv, s.vb, s.vr, es));
    r[3] = rng("log_decay", log_decay, s.H * 4);
    r[4] = rng("initial_state", first, s.Bz * s.H * s.Dk * s.Dv * 4);
    r[5] = rng("seqlens", lens, s.Bz * 4);
    return SSD_OK;
}

// The forward's walk: queries, keys, values, states as they lie.
ssd::AttnPass attn_forward(const ssd::AttnShape& s, const void* q, const void* k, const void* v, const float* first) {
    ssd::AttnPass p = {};
    p.a = q; p.c = k; p.x = v;
    p.ab = s.qb; p.cb = s.kb; p.xb = s.vb;
    p.ar = (uint32_t)s.qr; p.cr = (uint32_t)s.kr; p.xr = (uint32_t)s.vr;
    p.ag = 1; p.cg = p.xg = (int)(s.H / s.K);
    p.cd = (int)s.Dk; p.xd = (int)s.Dv;
    p.first = first;
    p.sc = 1; p.sx = (int)s.Dk;
    p.scale_p = p.scale_in = s.scale;
    p.scale_w = 1.f;
    p.exact = 1;
    return p;
}

ssd_status norm_shape(const ssd_group_norm_desc* d, bool gated, ssd::NormShape* s) {
    if (!d) return fail(SSD_ERR_NULL, "desc is NULL");
    if (d->batch < 0 || d->seqlen < 0 || d->channels < 1 || d->groups < 1)
        return fail(SSD_ERR_SHAPE, "sizes must be batch>=0, seqlen>=0, channels,groups>=1 (got %lld,%lld,%lld,%lld)",
                    (long long)d->batch, (long long)d->seqlen, (long long)d->channels, (long long)d->groups);
    if (d->channels % d->groups != 0)
        return fail(SSD_ERR_SHAPE, "channels (%lld) must be a multiple of groups (%lld)", (long long)d->channels,
                    (long long)d->groups);
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16)
        return fail(SSD_ERR_DTYPE, "dtype %d is not SSD_F32 or SSD_BF16", (int)d->dtype);
    if ((d->center != 0 && d->center != 1) || (d->silu != 0 && d->silu != 1) || (d->gate_first != 0 && d->gate_first != 1))
        return fail(SSD_ERR_SHAPE, "center, silu and gate_first must be 0 or 1");
    if (d->reserved != 0) return fail(SSD_ERR_SHAPE, "reserved must be 0");
    if (d->gate_first && !gated) return fail(SSD_ERR_NULL, "gate_first needs a gate");
    if (!(d->eps >= 0.f) || d->eps > 3.402823466e38f)
        return fail(SSD_ERR_SHAPE, "eps must be finite and not negative");
    if (d->channels / d->groups > ssd::kNormMost)
        return fail(SSD_ERR_UNSUPPORTED, "groups must have at most %lld channels (got %lld)", (long long)ssd::kNormMost,
                    (long long)(d->channels / d->groups));
    if (d->batch > 65535 || d->channels > ((int64_t)1 << 24) || d->seqlen > ((int64_t)1 << 31) ||
        d->batch * d->seqlen >= ((int64_t)1 << 32) || d->batch * d->seqlen > kMaxSize / d->channels)
        return fail(SSD_ERR_UNSUPPORTED, "sizes beyond the supported range");
    SSD_CHECK(check_stride("x", d->batch, d->x_bstride, d->seqlen, d->x_rstride));
    SSD_CHECK(check_stride("gate", d->batch, d->gate_bstride, d->seqlen, d->gate_rstride));
    s->Bz = d->batch; s->L = d->seqlen; s->C = d->channels; s->G = d->groups;
    s->xb = d->x_bstride; s->xr = d->x_rstride; s->zb = d->gate_bstride; s->zr = d->gate_rstride;
    s->eps = d->eps; s->bf16 = d->dtype == SSD_BF16;
    s->center = d->center == 1; s->silu = d->silu == 1; s->gate_first = d->gate_first == 1;
    return SSD_OK;
}

constexpr int kNormIn = 5;
ssd_status check_norm_in(const ssd::NormShape& s, const ssd::NormIn& in, Range* r) {
    const int64_t es = s.bf16 ? 2 : 4;
    if (!in.x && s.Bz > 0 && s.L > 0) return fail(SSD_ERR_NULL, "x is required");
    SSD_CHECK(check_aligned("x", in.x, es));
    SSD_CHECK(check_aligned("gate", in.gate, es));
    SSD_CHECK(check_aligned("weight", in.weight, 4));
    SSD_CHECK(check_aligned("bias", in.bias, 4));
    SSD_CHECK(check_aligned("seqlens", in.lens, 4));
    r[0] = rng("x", in.x, span_bytes(s.Bz, s.L, s.C, s.xb, s.xr, es));
    r[1] = rng("gate", in.gate, span_bytes(s.Bz, s.L, s.C, s.zb, s.zr, es));
    r[2] = rng("weight", in.weight, s.C * 4);
    r[3] = rng("bias", in.bias, s.C * 4);
    r[4] = rng("seqlens", in.lens, s.Bz * 4);
    return SSD_OK;
}
size_t norm_bwd_bytes(const ssd::NormShape& s) {
    return s.Bz > 0 && s.L > 0 ? (size_t)ssd::norm_bwd_parts(s) * 2 * s.C * sizeof(float) : 0;
}

}  // namespace

extern "C" {

ssd_status ssd_linear_attn_fwd_workspace_bytes(const ssd_linear_attn_desc* desc, size_t* bytes) {
    if (!bytes) return fail(SSD_ERR_NULL, "bytes is NULL");
    ssd::AttnShape s;
    SSD_CHECK(attn_shape(desc, &s));
    *bytes = ssd::attn_plan(s, false).bytes;
    return ok();
}

ssd_status ssd_linear_attn_fwd(const ssd_linear_attn_desc* desc, const void* q, const void* k, const void* v,
                               const float* log_decay, const float* initial_state, const int32_t* seqlens, void* y,
                               float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
    ssd::AttnShape s;
    SSD_CHECK(attn_shape(desc, &s));
    Range r[kAttnIn];
    SSD_CHECK(check_attn_in(s, q, k, v, log_decay, initial_state, seqlens, r));
    const int64_t es = s.bf16 ? 2 : 4;
    if (!y && s.Bz > 0 && s.L > 0) return fail(SSD_ERR_NULL, "y is required");
    SSD_CHECK(check_aligned("y", y, es));
    SSD_CHECK(check_aligned("final_state", final_state, 4));
    const ssd::AttnPlan pl = ssd::attn_plan(s, false);
    SSD_CHECK(check_workspace(workspace, workspace_bytes, pl.bytes));
    const Range out[] = {rng("y", y, s.Bz * s.L * s.H * s.Dv * es),
                         rng("final_state", final_state, s.Bz * s.H * s.Dk * s.Dv * 4),
                         rng("workspace", workspace, (int64_t)pl.bytes)};
    SSD_CHECK(check_disjoint(out, 3, r, kAttnIn));
    if (s.Bz == 0 || (s.L == 0 && !final_state)) return ok();
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    float* states = static_cast<float*>(workspace);
    ssd::AttnPass p = attn_forward(s, q, k, v, initial_state);
    p.y = y;
    p.last = final_state;
    hipError_t e = ssd::launch_attn_states(s, pl, &p, &states, 1, log_decay, seqlens, hs);
    if (e == hipSuccess) e = ssd::launch_attn_walks(s, pl, &p, &states, 1, log_decay, seqlens, hs);
    return e == hipSuccess ? ok() : hip_fail(e, "linear attention launch");
}

ssd_status ssd_linear_attn_bwd_workspace_bytes(const ssd_linear_attn_desc* desc, size_t* bytes) {
    if (!bytes) return fail(SSD_ERR_NULL, "bytes is NULL");
    ssd::AttnShape s;
    SSD_CHECK(attn_shape(desc, &s));
    *bytes = ssd::attn_plan(s, true).bytes;
    return ok();
}

ssd_status ssd_linear_attn_bwd(const ssd_linear_attn_desc* desc, const void* q, const void* k, const void* v,
                               const float* log_decay, const float* initial_state, const int32_t* seqlens,
                               const void* dy, const float* dfinal_state, void* dq, void* dk, void* dv,
                               float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream) {
    ssd::AttnShape s;
    SSD_CHECK(attn_shape(desc, &s));
    Range r[kAttnIn + 2];
    SSD_CHECK(check_attn_in(s, q, k, v, log_decay, initial_state, seqlens, r));
    const int64_t es = s.bf16 ? 2 : 4, rows = s.Bz * s.L, nstate = s.Bz * s.H * s.Dk * s.Dv * 4;
    if (s.Bz > 0 && s.L > 0 && (!dy || !dq || !dk || !dv)) return fail(SSD_ERR_NULL, "dy, dq, dk and dv are required");
    SSD_CHECK(check_aligned("dy", dy, es));
    SSD_CHECK(check_aligned("dfinal_state", dfinal_state, 4));
    SSD_CHECK(check_aligned("dq", dq, es));
    SSD_CHECK(check_aligned("dk", dk, es));
    SSD_CHECK(check_aligned("dv", dv, es));
    SSD_CHECK(check_aligned("dinitial_state", dinitial_state, 4));
    r[kAttnIn] = rng("dy", dy, rows * s.H * s.Dv * es);
    r[kAttnIn + 1] = rng("dfinal_state", dfinal_state, nstate);
    const ssd::AttnPlan pl = ssd::attn_plan(s, true);
    SSD_CHECK(check_workspace(workspace, workspace_bytes, pl.bytes));
    const Range out[] = {rng("dq", dq, rows * s.H * s.Dk * es), rng("dk", dk, rows * s.K * s.Dk * es),
                         rng("dv", dv, rows * s.K * s.Dv * es), rng("dinitial_state", dinitial_state, nstate),
                         rng("workspace", workspace, (int64_t)pl.bytes)};
    SSD_CHECK(check_disjoint(out, 5, r, kAttnIn + 2));
    if (s.Bz == 0 || (s.L == 0 && !dinitial_state)) return ok();
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    float *states = reinterpret_cast<float*>(ws + pl.states), *adjoint = reinterpret_cast<float*>(ws + pl.adjoint);
    const bool shared = s.K != s.H;

    // dq = scale S^T dy: the forward with values for keys, dy for queries, states transposed
    const ssd::AttnPass f = attn_forward(s, q, k, v, initial_state);
    ssd::AttnPass pq = f;
    pq.a = dy; pq.ab = s.L * s.H * s.Dv; pq.ar = (uint32_t)(s.H * s.Dv); pq.ag = 1;
    pq.c = v; pq.cb = f.xb; pq.cr = f.xr; pq.cg = f.xg;
    pq.x = k; pq.xb = f.cb; pq.xr = f.cr; pq.xg = f.cg;
    pq.cd = f.xd; pq.xd = f.cd; pq.sc = f.sx; pq.sx = f.sc;
    pq.y = dq;
    pq.exact = 0;                    // its states are no results
    // against time, G[t] = scale dy[t] q[t]^T + gamma G[t+1]: dk = G^T v and dv = G k
    ssd::AttnPass pv = f;
    pv.rev = 1;
    pv.a = k; pv.ab = f.cb; pv.ar = f.cr; pv.ag = f.cg;
    pv.c = q; pv.cb = f.ab; pv.cr = f.ar; pv.cg = 1;
    pv.x = dy; pv.xb = pq.ab; pv.xr = pq.ar; pv.xg = 1;
    pv.first = dfinal_state;
    pv.scale_p = pv.scale_w = s.scale;
    pv.scale_in = 1.f;
    ssd::AttnPass pk = pv;
    pk.a = v; pk.ab = f.xb; pk.ar = f.xr; pk.ag = f.xg;
    pk.c = dy; pk.cb = pq.ab; pk.cr = pq.ar; pk.cg = 1;
    pk.x = q; pk.xb = f.ab; pk.xr = f.ar; pk.xg = 1;
    pk.cd = f.xd; pk.xd = f.cd; pk.sc = f.sx; pk.sx = f.sc;
    pk.exact = 0;
    pv.last = dinitial_state;
    pk.y = shared ? static_cast<void*>(ws + pl.dk) : dk;
    pv.y = shared ? static_cast<void*>(ws + pl.dv) : dv;
    pk.y_f32 = pv.y_f32 = shared;

    const ssd::AttnPass ends[] = {pq, pv}, walks[] = {pq, pk, pv};
    float* const slots[] = {states, adjoint, adjoint};
    hipError_t e = ssd::launch_attn_states(s, pl, ends, slots, 2, log_decay, seqlens, hs);
    if (e == hipSuccess) e = ssd::launch_attn_walks(s, pl, walks, slots, 3, log_decay, seqlens, hs);
    if (e == hipSuccess && shared && rows > 0)
        e = ssd::launch_attn_share(s, static_cast<const float*>(pk.y), static_cast<const float*>(pv.y), dk, dv, hs);
    return e == hipSuccess ? ok() : hip_fail(e, "linear attention backward launch");
}

ssd_status ssd_linear_attn_step(const ssd_linear_attn_desc* desc, float* state, const void* q, const void* k,
                                const void* v, const float* log_decay, void* y, void* stream) {
    ssd::AttnShape s;
    SSD_CHECK(attn_shape(desc, &s));
    if (s.L != 1) return fail(SSD_ERR_SHAPE, "seqlen must be 1 (got %lld)", (long long)s.L);
    Range r[kAttnIn];
    SSD_CHECK(check_attn_in(s, q, k, v, log_decay, nullptr, nullptr, r));
    if (s.Bz == 0) return ok();
    const int64_t es = s.bf16 ? 2 : 4;
    if (!state || !y) return fail(SSD_ERR_NULL, "state and y are required");
    SSD_CHECK(check_aligned("state", state, 4));
    SSD_CHECK(check_aligned("y", y, es));
    const Range out[] = {rng("y", y, s.Bz * s.H * s.Dv * es), rng("state", state, s.Bz * s.H * s.Dk * s.Dv * 4)};
    SSD_CHECK(check_disjoint(out, 2, r, kAttnIn));
    const hipError_t e = ssd::launch_attn_step(s, state, q, k, v, log_decay, y, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "linear attention step launch");
}

ssd_status ssd_group_norm_fwd(const ssd_group_norm_desc* desc, const void* x, const float* weight, const float* bias,
                              const void* gate, const int32_t* seqlens, void* y, void* stream) {
    ssd::NormShape s;
    SSD_CHECK(norm_shape(desc, gate != nullptr || (desc && (desc->batch == 0 || desc->seqlen == 0)), &s));
    const ssd::NormIn in{x, gate, weight, bias, seqlens};
    Range r[kNormIn];
    SSD_CHECK(check_norm_in(s, in, r));
    const int64_t es = s.bf16 ? 2 : 4;
    if (s.Bz == 0 || s.L == 0) return ok();
    if (!y) return fail(SSD_ERR_NULL, "y is required");
    SSD_CHECK(check_aligned("y", y, es));
    const Range out[] = {rng("y", y, s.Bz * s.L * s.C * es)};
    SSD_CHECK(check_disjoint(out, 1, r, kNormIn));
    const hipError_t e = ssd::launch_norm_fwd(s, in, y, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "group norm launch");
}

ssd_status ssd_group_norm_bwd_workspace_bytes(const ssd_group_norm_desc* desc, size_t* bytes) {
    if (!bytes) return fail(SSD_ERR_NULL, "bytes is NULL");
    ssd::NormShape s;
    SSD_CHECK(norm_shape(desc, true, &s));
    *bytes = norm_bwd_bytes(s);
    return ok();
}

ssd_status ssd_group_norm_bwd(const ssd_group_norm_desc* desc, const void* x, const float* weight, const float* bias,
                              const void* gate, const int32_t* seqlens, const void* dy, void* dx, void* dgate,
                              float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    ssd::NormShape s;
    SSD_CHECK(norm_shape(desc, gate != nullptr || (desc && (desc->batch == 0 || desc->seqlen == 0)), &s));
    const ssd::NormIn in{x, gate, weight, bias, seqlens};
    Range r[kNormIn + 1];
    SSD_CHECK(check_norm_in(s, in, r));
    const int64_t es = s.bf16 ? 2 : 4, n = s.Bz * s.L * s.C * es;
    const bool empty = s.Bz == 0 || s.L == 0;
    if (!empty && (!dy || !dx)) return fail(SSD_ERR_NULL, "dy and dx are required");
    if ((!empty && !gate != !dgate) || !weight != !dweight || !bias != !dbias)
        return fail(SSD_ERR_NULL, "dgate, dweight and dbias are required exactly when their input is given");
    SSD_CHECK(check_aligned("dy", dy, es));
    SSD_CHECK(check_aligned("dx", dx, es));
    SSD_CHECK(check_aligned("dgate", dgate, es));
    SSD_CHECK(check_aligned("dweight", dweight, 4));
    SSD_CHECK(check_aligned("dbias", dbias, 4));
    const size_t need = dweight || dbias ? norm_bwd_bytes(s) : 0;
    SSD_CHECK(check_workspace(workspace, workspace_bytes, need));
    r[kNormIn] = rng("dy", dy, n);
    const Range out[] = {rng("dx", dx, n), rng("dgate", dgate, n), rng("dweight", dweight, s.C * 4),
                         rng("dbias", dbias, s.C * 4), rng("workspace", workspace, (int64_t)need)};
    SSD_CHECK(check_disjoint(out, 5, r, kNormIn + 1));
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (empty) {   // no rows: the parameters' gradients are zero
        if (dweight) e = ssd::launch_fill_zero(dweight, s.C, hs);
        if (e == hipSuccess && dbias) e = ssd::launch_fill_zero(dbias, s.C, hs);
        return e == hipSuccess ? ok() : hip_fail(e, "empty group norm gradient");
    }
    e = ssd::launch_norm_bwd(s, in, dy, dx, dgate, dweight, dbias, static_cast<float*>(workspace), hs);
    return e == hipSuccess ? ok() : hip_fail(e, "group norm backward launch");
}

}  // extern "C"
