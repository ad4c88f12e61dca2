// block_host.cpp -- host side of the operators between a Transformer's linear
// layers and of its loss: norms around a block, dropout, cross attention, log
// probabilities.  As in ops_host.cpp, every argument is checked before any
// device work is enqueued, and nothing is allocated on the device.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "ops_check.h"
#include "ops_internal.h"

using namespace rar;

struct rar_norm_s {
    int64_t D = 0;
    rar_dtype dtype = RAR_F32;
    rar_norm_kind post = RAR_NORM_NONE, pre = RAR_NORM_NONE;
    float eps = 0;
};

struct rar_attn_s {
    int64_t H = 0, Hkv = 0, dh = 0;
    rar_dtype dtype = RAR_F32;
    float scale = 0;
};

namespace {

bool valid_kind(int k) { return k == RAR_NORM_NONE || k == RAR_NORM_LAYER || k == RAR_NORM_RMS; }

bool all_aligned(std::initializer_list<const void *> ps, int to)
{
    for (const void *p : ps)
        if (!aligned(p, to))
            return false;
    return true;
}

// (enough for every call of fewer rows too)
int64_t norm_ws_bytes(int64_t T, int64_t D) { return T ? norm_chunks_up_to(T, D) * 4 * up(D, 8) * 4 : 0; }

}  // namespace

// =============================================================================
// Norms around a block
// =============================================================================

extern "C" rar_status rar_norm_plan(int64_t D, rar_dtype dtype, rar_norm_kind post, rar_norm_kind pre, float eps,
                                    rar_norm_t *out)
{
    if (!out)
        return RAR_EINVAL;
    *out = nullptr;
    if (!valid_width(D) || !valid_dtype(dtype) || !valid_kind(post) || !valid_kind(pre) || !(eps > 0) ||
        !std::isfinite(eps))
        return RAR_EINVAL;
    rar_norm_s *p = new (std::nothrow) rar_norm_s;
    if (!p)
        return RAR_ENOMEM;
    p->D = D;
    p->dtype = dtype;
    p->post = post;
    p->pre = pre;
    p->eps = eps;
    *out = p;
    return RAR_OK;
}

extern "C" rar_status rar_norm_destroy(rar_norm_t plan)
{
    delete plan;
    return RAR_OK;
}

extern "C" rar_status rar_norm_workspace(rar_norm_t plan, int64_t T, int64_t *bytes)
{
    if (!plan || !bytes || !valid_rows(T))
        return RAR_EINVAL;
    *bytes = norm_ws_bytes(T, plan->D);
    return RAR_OK;
}

extern "C" rar_status rar_norm_forward(rar_norm_t plan, int64_t T, const void *x, int64_t ldx, const void *o,
                                       int64_t ldo, const void *post_w, const void *post_b, const void *gate, float a,
                                       float s, const void *pre_w, const void *pre_b, void *h, int64_t ldh, void *u,
                                       int64_t ldu, void *stream)
{
    if (!plan || !valid_rows(T))
        return RAR_EINVAL;
    if (T == 0)
        return RAR_OK;
    const int64_t D = plan->D;
    const int es = esize(plan->dtype);
    if (!x || (!h && !u))
        return RAR_EINVAL;
    if (!valid_ld(ldx, D) || (o && !valid_ld(ldo, D)) || (h && !valid_ld(ldh, D)) || (u && !valid_ld(ldu, D)))
        return RAR_EINVAL;
    if (!o || plan->post == RAR_NORM_NONE)
        post_w = post_b = nullptr;
    if (!o)
        gate = nullptr;
    if (plan->pre == RAR_NORM_NONE || !u)
        pre_w = pre_b = nullptr;
    if (!all_aligned({x, o, post_w, post_b, gate, pre_w, pre_b, h, u}, es))
        return RAR_EALIGN;
    const Mat mx{x, T, D, ldx, es}, mo{o, T, D, ldo, es}, mh{h, T, D, ldh, es}, mu{u, T, D, ldu, es};
    if (!apart({mh, mu}, {mo, vec(post_w, D, es), vec(post_b, D, es), vec(gate, D, es), vec(pre_w, D, es),
                          vec(pre_b, D, es)}) ||
        overlap(mu, mx) || (!same(mh, mx) && overlap(mh, mx)))
        return RAR_EINVAL;
    NormParams p{};
    p.x = x;
    p.ldx = ldx;
    p.o = o;
    p.ldo = ldo;
    p.post_w = post_w;
    p.post_b = post_b;
    p.gate = gate;
    p.pre_w = pre_w;
    p.pre_b = pre_b;
    p.h = h;
    p.ldh = ldh;
    p.u = u;
    p.ldu = ldu;
    p.rows = T;
    p.cols = D;
    p.a = a;
    p.s = s;
    p.eps = plan->eps;
    p.post = plan->post;
    p.pre = plan->pre;
    return launched(launch_norm(plan->dtype, p, static_cast<hipStream_t>(stream)));
}

extern "C" rar_status rar_norm_backward(rar_norm_t plan, int64_t T, const void *dh, int64_t lddh, const void *du,
                                        int64_t lddu, const void *o, int64_t ldo, const void *h, int64_t ldh,
                                        const void *post_w, const void *post_b, const void *gate, float a, float s,
                                        const void *pre_w, void *dx, int64_t lddx, void *d_o, int64_t lddo,
                                        void *dpost_w, void *dpost_b, void *dgate, void *dpre_w, void *dpre_b,
                                        int accumulate, void *ws, int64_t ws_bytes, void *stream)
{
    if (!plan || !valid_rows(T))
        return RAR_EINVAL;
    const int64_t D = plan->D;
    const int es = esize(plan->dtype);
    const bool post = plan->post != RAR_NORM_NONE, pre = plan->pre != RAR_NORM_NONE;
    const bool sum_post = dpost_w || dpost_b || dgate, sum_pre = dpre_w || dpre_b;
    if (((dpost_w || dpost_b) && !post) || (sum_pre && !pre))
        return RAR_EINVAL;
    const int64_t need = sum_post || sum_pre ? norm_ws_bytes(T, D) : 0;
    if (T > 0) {
        if (!o && (d_o || sum_post))
            return RAR_EINVAL;
        const bool use_h = pre && du;
        if (!use_h)
            h = nullptr;
        if ((use_h && !h) || (need && !ws))
            return RAR_EINVAL;
        if ((dh && !valid_ld(lddh, D)) || (du && !valid_ld(lddu, D)) || (o && !valid_ld(ldo, D)) ||
            (h && !valid_ld(ldh, D)) || (dx && !valid_ld(lddx, D)) || (d_o && !valid_ld(lddo, D)))
            return RAR_EINVAL;
    } else {
        dh = du = o = h = nullptr;
        dx = d_o = nullptr;
    }
    if (!post || !o)
        post_w = post_b = nullptr;
    if (!o)
        gate = nullptr;
    if (!pre || !du)
        pre_w = nullptr;
    if (!all_aligned({dh, du, o, h, post_w, post_b, gate, pre_w, dx, d_o, dpost_w, dpost_b, dgate, dpre_w, dpre_b},
                     es) ||
        (need && !aligned(ws, 16)))
        return RAR_EALIGN;
    if (need && ws_bytes < need)
        return RAR_EINVAL;
    const Mat mdh{dh, T, D, lddh, es}, mdu{du, T, D, lddu, es}, mo{o, T, D, ldo, es}, mh{h, T, D, ldh, es};
    const Mat mdx{dx, T, D, lddx, es}, mdo{d_o, T, D, lddo, es}, mws{need ? ws : nullptr, 1, need, need, 1};
    const Mat v1 = vec(dpost_w, D, es), v2 = vec(dpost_b, D, es), v3 = vec(dgate, D, es), v4 = vec(dpre_w, D, es),
              v5 = vec(dpre_b, D, es);
    if (!apart({mdx, mdo, v1, v2, v3, v4, v5, mws},
               {mdu, mh, vec(post_w, D, es), vec(post_b, D, es), vec(gate, D, es), vec(pre_w, D, es)}) ||
        !apart({v1, v2, v3, v4, v5, mws}, {mdh, mo}) || overlap(mdx, mo) || overlap(mdo, mdh) ||
        (!same(mdx, mdh) && overlap(mdx, mdh)) || (!same(mdo, mo) && overlap(mdo, mo)))
        return RAR_EINVAL;
    NormGradParams p{};
    p.dh = dh;
    p.lddh = lddh;
    p.du = du;
    p.lddu = lddu;
    p.o = o;
    p.ldo = ldo;
    p.h = h;
    p.ldh = ldh;
    p.post_w = post_w;
    p.post_b = post_b;
    p.gate = gate;
    p.pre_w = pre_w;
    p.dx = dx;
    p.lddx = lddx;
    p.d_o = d_o;
    p.lddo = lddo;
    p.dpost_w = dpost_w;
    p.dpost_b = dpost_b;
    p.dgate = dgate;
    p.dpre_w = dpre_w;
    p.dpre_b = dpre_b;
    p.accumulate = accumulate;
    p.part = (float *)ws;
    p.chunks = T ? norm_chunks(T, D) : 0;
    p.pitch = up(D, 8);
    p.sum_post = sum_post;
    p.sum_pre = sum_pre;
    p.rows = T;
    p.cols = D;
    p.a = a;
    p.s = s;
    p.eps = plan->eps;
    p.post = plan->post;
    p.pre = plan->pre;
    hipStream_t st = static_cast<hipStream_t>(stream);
    rar_status rc = RAR_OK;
    if (T > 0 && (dx || d_o || sum_post || sum_pre))
        rc = launched(launch_norm_grad(plan->dtype, p, st));
    if (rc == RAR_OK && (sum_post || sum_pre))
        rc = launched(launch_norm_sums(plan->dtype, p, st));
    return rc;
}

// =============================================================================
// Dropout
// =============================================================================

extern "C" rar_status rar_dropout(int64_t T, int64_t D, rar_dtype dtype, float p, uint64_t seed, const int64_t *step,
                                  const void *x, int64_t ldx, const void *r, int64_t ldr, void *y, int64_t ldy,
                                  void *stream)
{
    if (!valid_rows(T) || !valid_width(D) || !valid_dtype(dtype) || !(p >= 0) || !(p <= 1))
        return RAR_EINVAL;
    if (T == 0)
        return RAR_OK;
    if (!x || !y || !valid_ld(ldx, D) || !valid_ld(ldy, D) || (r && !valid_ld(ldr, D)))
        return RAR_EINVAL;
    const int es = esize(dtype);
    if (!all_aligned({x, r, y}, es) || !aligned(step, 8))
        return RAR_EALIGN;
    if (div_up(T * div_up(D, 8), 1024) * 256 > kMaxLanes)
        return RAR_EINVAL;
    const Mat mx{x, T, D, ldx, es}, mr{r, T, D, ldr, es}, my{y, T, D, ldy, es};
    if ((!same(my, mx) && overlap(my, mx)) || (!same(my, mr) && overlap(my, mr)) || overlap(my, vec(step, 1, 8)))
        return RAR_EINVAL;
    DropoutParams q{};
    q.x = x;
    q.ldx = ldx;
    q.r = r;
    q.ldr = ldr;
    q.y = y;
    q.ldy = ldy;
    q.rows = T;
    q.cols = D;
    q.step = step;
    q.seed_lo = (uint32_t)seed;
    q.seed_hi = (uint32_t)(seed >> 32);
    q.threshold = (uint32_t)std::floor((double)p * 65536 + 0.5);
    q.scale = q.threshold < 65536 ? (float)(65536.0 / (65536 - q.threshold)) : 0.0f;
    return launched(launch_dropout(dtype, q, static_cast<hipStream_t>(stream)));
}

// =============================================================================
// Cross attention
// =============================================================================

namespace {

constexpr int64_t kMaxBatch = 65535;
// The bf16 gradients start from -lse / scale, every call takes scale log2 e: neither may overflow where scores do not.
constexpr float kAttnScale = 0x1p-100f;

AttnShape attn_shape(const rar_attn_s &a, int64_t B, int64_t Tq, int64_t Tk)
{
    return AttnShape(a.H, a.Hkv, a.dh, a.dtype, B, Tq, Tk);
}

bool valid_attn(const rar_attn_s *a, int64_t B, int64_t Tq, int64_t Tk)
{
    return a && B >= 0 && B <= kMaxBatch && Tq >= 0 && Tk >= 0 && Tq <= kMaxRows && Tk <= kMaxRows &&
           B * Tq <= kMaxRows && B * Tk <= kMaxRows && attn_shape(*a, B, Tq, Tk).fits();
}

struct AttnWs {
    void *q, *k, *v, *g;
    float *part, *stats, *lse, *delta, *q_part, *k_part;
    int64_t bytes;
};

AttnWs attn_ws(const AttnShape &s, bool backward, void *ws)
{
    Carve c{(char *)ws};
    AttnWs w{};
    const int es = esize(s.dt);
    const int64_t wide = s.B * s.Tq * s.H * s.cols * es, narrow = s.B * s.Tk * s.Hkv * s.cols * es;
    if (backward || !s.token()) {
        w.q = c.take(wide);
        w.k = c.take(narrow);
        w.v = c.take(narrow);
    }
    if (backward) {
        w.g = c.take(wide);
        w.lse = (float *)c.take(s.B * s.H * s.padded * 4);
        w.delta = (float *)c.take(s.B * s.H * s.padded * 4);
        w.q_part = (float *)c.take(s.q_room() * s.width * 4);
        w.k_part = (float *)c.take(s.k_room() * 2 * s.width * 4);
    } else {
        w.part = (float *)c.take(s.part_room() * s.width * 4);
        w.stats = (float *)c.take(s.part_room() * 8);
    }
    w.bytes = c.used;
    return w;
}

// Where the kernels read a matrix of heads: itself, or a packed copy.
AttnOperand operand(const AttnShape &s, const Mat &m, int64_t heads, void *copy, AttnPack &pack)
{
    const int64_t per = 16 / m.es;
    if (aligned(m.p, 16) && m.ld % per == 0 && s.dh % per == 0)
        return AttnOperand{m.p, m.ld, s.dh, (int)s.cols};
    if (!m.empty())
        pack.item[pack.count++] = AttnPack::Item{m.p, copy, m.ld, heads, m.rows * heads * (s.cols / per)};
    return AttnOperand{copy, heads * s.cols, s.cols, (int)s.cols};
}

AttnParams attn_params(const rar_attn_s &a, const AttnShape &s, const int64_t *qlen, const int64_t *klen)
{
    AttnParams p{};
    p.B = s.B;
    p.Tq = s.Tq;
    p.Tk = s.Tk;
    p.H = s.H;
    p.Hkv = s.Hkv;
    p.share = s.share;
    p.dh = (int)s.dh;
    p.scale = a.scale;
    p.qlen = qlen;
    p.klen = klen;
    p.tiles = s.tiles;
    p.splits = 1;
    p.padded = s.padded;
    return p;
}

}  // namespace

extern "C" rar_status rar_attn_plan(int64_t H, int64_t Hkv, int64_t dh, rar_dtype dtype, float scale, rar_attn_t *out)
{
    if (!out)
        return RAR_EINVAL;
    *out = nullptr;
    if (H < 1 || H > kMaxWidth || Hkv < 1 || Hkv > H || H % Hkv || dh < 1 || dh > RAR_ATTN_MAX_WIDTH ||
        H * dh > kMaxWidth || !valid_dtype(dtype) || !(scale >= kAttnScale) || !(scale <= 1 / kAttnScale))
        return RAR_EINVAL;
    rar_attn_s *p = new (std::nothrow) rar_attn_s;
    if (!p)
        return RAR_ENOMEM;
    p->H = H;
    p->Hkv = Hkv;
    p->dh = dh;
    p->dtype = dtype;
    p->scale = scale;
    *out = p;
    return RAR_OK;
}

extern "C" rar_status rar_attn_destroy(rar_attn_t plan)
{
    delete plan;
    return RAR_OK;
}

extern "C" rar_status rar_attn_workspace(rar_attn_t plan, int64_t B, int64_t Tq, int64_t Tk, int64_t *forward_bytes,
                                         int64_t *backward_bytes)
{
    if (!valid_attn(plan, B, Tq, Tk))
        return RAR_EINVAL;
    const AttnShape s = attn_shape(*plan, B, Tq, Tk);
    if (forward_bytes)
        *forward_bytes = attn_ws(s, false, nullptr).bytes;
    if (backward_bytes)
        *backward_bytes = attn_ws(s, true, nullptr).bytes;
    return RAR_OK;
}

extern "C" rar_status rar_attn_forward(rar_attn_t plan, int64_t B, int64_t Tq, int64_t Tk, const void *q, int64_t ldq,
                                       const void *k, int64_t ldk, const void *v, int64_t ldv, const int64_t *qlen,
                                       const int64_t *klen, void *o, int64_t ldo, float *lse, void *ws,
                                       int64_t ws_bytes, void *stream)
{
    if (!valid_attn(plan, B, Tq, Tk))
        return RAR_EINVAL;
    if (B * Tq == 0)
        return RAR_OK;
    const AttnShape s = attn_shape(*plan, B, Tq, Tk);
    const int es = esize(s.dt);
    const int64_t wide = s.H * s.dh, narrow = s.Hkv * s.dh;
    const AttnWs w = attn_ws(s, false, ws);
    if (!q || !o || (Tk > 0 && (!k || !v)) || (!ws && w.bytes))
        return RAR_EINVAL;
    if (Tk == 0)
        k = v = nullptr;
    if (!valid_ld(ldq, wide) || !valid_ld(ldo, wide) || (Tk > 0 && (!valid_ld(ldk, narrow) || !valid_ld(ldv, narrow))))
        return RAR_EINVAL;
    if (!all_aligned({q, k, v, o}, es) || !all_aligned({qlen, klen}, 8) || !aligned(lse, 4) || !aligned(ws, 16))
        return RAR_EALIGN;
    if (ws_bytes < w.bytes)
        return RAR_EINVAL;
    const Mat mq{q, B * Tq, wide, ldq, es}, mk{k, B * Tk, narrow, ldk, es}, mv{v, B * Tk, narrow, ldv, es};
    if (!apart({Mat{o, B * Tq, wide, ldo, es}, vec(lse, B * Tq * s.H, 4), vec(ws, w.bytes, 1)},
               {mq, mk, mv, vec(qlen, B, 8), vec(klen, B, 8)}))
        return RAR_EINVAL;
    hipStream_t st = static_cast<hipStream_t>(stream);
    AttnPack pack{};
    pack.dh = (int)s.dh;
    pack.cols = (int)s.cols;
    AttnParams p = attn_params(*plan, s, qlen, klen);
    if (s.token()) {
        p.q = AttnOperand{q, ldq, s.dh, (int)s.dh};
        p.k = AttnOperand{k, ldk, s.dh, (int)s.dh};
        p.v = AttnOperand{v, ldv, s.dh, (int)s.dh};
    } else {
        p.q = operand(s, mq, s.H, w.q, pack);
        p.k = operand(s, mk, s.Hkv, w.k, pack);
        p.v = operand(s, mv, s.Hkv, w.v, pack);
    }
    p.o = o;
    p.ldo = ldo;
    p.lse = lse;
    p.splits = (int)s.splits;
    p.stages = (int)s.stages;
    p.blocks = s.blocks();
    p.part = w.part;
    p.stats = w.stats;
    p.part_rows = s.part_rows();
    p.pitch = s.width;
    rar_status rc = pack.count ? launched(launch_attn_pack(s.dt, pack, st)) : RAR_OK;
    if (rc == RAR_OK)
        rc = launched(launch_attn_rows(s.dt, p, s.few, st));
    if (rc == RAR_OK && p.splits > 1)
        rc = launched(launch_attn_join(s.dt, p, st));
    return rc;
}

extern "C" rar_status rar_attn_backward(rar_attn_t plan, int64_t B, int64_t Tq, int64_t Tk, const void *d_o,
                                        int64_t lddo, const void *q, int64_t ldq, const void *k, int64_t ldk,
                                        const void *v, int64_t ldv, const int64_t *qlen, const int64_t *klen,
                                        const void *o, int64_t ldo, const float *lse, void *dq, int64_t lddq, void *dk,
                                        int64_t lddk, void *dv, int64_t lddv, void *ws, int64_t ws_bytes, void *stream)
{
    if (!valid_attn(plan, B, Tq, Tk))
        return RAR_EINVAL;
    const AttnShape s = attn_shape(*plan, B, Tq, Tk);
    const int es = esize(s.dt);
    const int64_t wide = s.H * s.dh, narrow = s.Hkv * s.dh;
    const AttnWs w = attn_ws(s, true, ws);
    const bool queries = B * Tq > 0, keys = B * Tk > 0;
    if (!queries) {
        d_o = q = o = nullptr;
        lse = nullptr;
        dq = nullptr;
    }
    if (!keys) {
        k = v = nullptr;
        dk = dv = nullptr;
    }
    if (!dq && !dk && !dv)
        return RAR_OK;
    if ((queries && (!d_o || !q || !o || !lse)) || (keys && (!k || !v)) || !ws)
        return RAR_EINVAL;
    if ((queries && (!valid_ld(lddo, wide) || !valid_ld(ldq, wide) || !valid_ld(ldo, wide))) ||
        (dq && !valid_ld(lddq, wide)) || (keys && (!valid_ld(ldk, narrow) || !valid_ld(ldv, narrow))) ||
        (dk && !valid_ld(lddk, narrow)) || (dv && !valid_ld(lddv, narrow)))
        return RAR_EINVAL;
    if (!all_aligned({d_o, q, k, v, o, dq, dk, dv}, es) || !all_aligned({qlen, klen}, 8) || !aligned(lse, 4) ||
        !aligned(ws, 16))
        return RAR_EALIGN;
    if (ws_bytes < w.bytes)
        return RAR_EINVAL;
    const Mat mq{q, B * Tq, wide, ldq, es}, mk{k, B * Tk, narrow, ldk, es}, mv{v, B * Tk, narrow, ldv, es};
    const Mat mg{d_o, B * Tq, wide, lddo, es}, mo{o, B * Tq, wide, ldo, es};
    if (!apart({Mat{dq, B * Tq, wide, lddq, es}, Mat{dk, B * Tk, narrow, lddk, es}, Mat{dv, B * Tk, narrow, lddv, es},
                vec(ws, w.bytes, 1)},
               {mq, mk, mv, mg, mo, vec(lse, B * Tq * s.H, 4), vec(qlen, B, 8), vec(klen, B, 8)}))
        return RAR_EINVAL;
    hipStream_t st = static_cast<hipStream_t>(stream);
    AttnPack pack{};
    pack.dh = (int)s.dh;
    pack.cols = (int)s.cols;
    AttnParams p = attn_params(*plan, s, qlen, klen);
    p.q = operand(s, mq, s.H, w.q, pack);
    p.k = operand(s, mk, s.Hkv, w.k, pack);
    p.v = operand(s, mv, s.Hkv, w.v, pack);
    p.g = operand(s, mg, s.H, w.g, pack);
    p.o = (void *)o;
    p.ldo = ldo;
    p.d_o = d_o;
    p.lddo = lddo;
    p.lse = (float *)lse;
    p.row_lse = w.lse;
    p.row_delta = w.delta;
    p.dq = dq;
    p.lddq = lddq;
    p.dk = dk;
    p.lddk = lddk;
    p.dv = dv;
    p.lddv = lddv;
    rar_status rc = pack.count ? launched(launch_attn_pack(s.dt, pack, st)) : RAR_OK;
    if (rc == RAR_OK && queries)
        rc = launched(launch_attn_delta(s.dt, p, st));
    AttnSum sum{};
    if (rc == RAR_OK && dq) {
        p.tiles = s.q_tiles;
        p.splits = (int)s.q_splits;
        p.blocks = B * s.Hkv * p.tiles * p.splits;
        p.part = w.q_part;
        p.part_rows = s.part_rows();
        rc = launched(launch_attn_dq(s.dt, p, st));
        if (p.splits > 1) {
            sum.q_part = w.q_part;
            sum.q_rows = s.part_rows();
        }
    }
    if (rc == RAR_OK && (dk || dv)) {
        p.tiles = s.key_tiles;
        p.splits = (int)s.k_splits;
        p.blocks = B * s.Hkv * p.tiles * p.splits;
        p.part = w.k_part;
        p.part_rows = B * s.Hkv * Tk;
        rc = launched(launch_attn_dkv(s.dt, p, st));
        if (p.splits > 1) {
            sum.k_part = w.k_part;
            sum.k_rows = B * s.Hkv * Tk;
        }
    }
    if (rc == RAR_OK && (sum.q_rows || sum.k_rows)) {
        sum.Tq = Tq;
        sum.Tk = Tk;
        sum.Hkv = s.Hkv;
        sum.share = s.share;
        sum.q_splits = (int)s.q_splits;
        sum.k_splits = (int)s.k_splits;
        sum.pitch = s.width;
        sum.dh = (int)s.dh;
        sum.dq = dq;
        sum.lddq = lddq;
        sum.dk = dk;
        sum.lddk = lddk;
        sum.dv = dv;
        sum.lddv = lddv;
        rc = launched(launch_attn_sum(s.dt, sum, st));
    }
    return rc;
}

// =============================================================================
// Log probabilities
// =============================================================================

namespace {

constexpr float kLogprobScale = 0x1p126f;  // scale log2 e is finite: times the maximum's distance, zero, it is zero

bool valid_logprob(int64_t T, int64_t V, rar_dtype dtype, float scale)
{
    return valid_rows(T) && valid_width(V) && valid_dtype(dtype) && scale > 0 && scale <= kLogprobScale;
}

}  // namespace

extern "C" rar_status rar_logprob(int64_t T, int64_t V, rar_dtype dtype, const void *logits, int64_t ldz, float scale,
                                  const int64_t *targets, float *logp, float *entropy, int K, int64_t *top_ids,
                                  float *top_logp, void *stream)
{
    if (!valid_logprob(T, V, dtype, scale) || K < 0 || K > RAR_LOGPROB_MAX_TOP)
        return RAR_EINVAL;
    if (T == 0)
        return RAR_OK;
    if (!logits || !valid_ld(ldz, V) || (logp && !targets) || (K > 0 && (!top_ids || !top_logp)))
        return RAR_EINVAL;
    if (K == 0)
        top_ids = nullptr, top_logp = nullptr;
    const int es = esize(dtype);
    if (!aligned(logits, es) || !all_aligned({targets, top_ids}, 8) || !all_aligned({logp, entropy, top_logp}, 4))
        return RAR_EALIGN;
    if (!apart({vec(logp, T, 4), vec(entropy, T, 4), vec(top_ids, T * K, 8), vec(top_logp, T * K, 4)},
               {Mat{logits, T, V, ldz, es}, vec(targets, T, 8)}))
        return RAR_EINVAL;
    LogprobParams p{};
    p.z = logits;
    p.ldz = ldz;
    p.scale = scale;
    p.targets = targets;
    p.logp = logp;
    p.entropy = entropy;
    p.top = K;
    p.top_ids = top_ids;
    p.top_logp = top_logp;
    p.rows = T;
    p.cols = V;
    return launched(launch_logprob(dtype, p, static_cast<hipStream_t>(stream)));
}

extern "C" rar_status rar_logprob_grad(int64_t T, int64_t V, rar_dtype dtype, const void *logits, int64_t ldz,
                                       float scale, const int64_t *targets, const float *dlogp, const float *dentropy,
                                       float *logp, float *entropy, void *dz, int64_t lddz, void *stream)
{
    if (!valid_logprob(T, V, dtype, scale))
        return RAR_EINVAL;
    if (T == 0)
        return RAR_OK;
    if (!logits || !dz || !valid_ld(ldz, V) || !valid_ld(lddz, V) || ((logp || dlogp) && !targets))
        return RAR_EINVAL;
    const int es = esize(dtype);
    if (!all_aligned({logits, dz}, es) || !aligned(targets, 8) || !all_aligned({dlogp, dentropy, logp, entropy}, 4))
        return RAR_EALIGN;
    const Mat mz{logits, T, V, ldz, es}, md{dz, T, V, lddz, es};
    const Mat ml = vec(logp, T, 4), me = vec(entropy, T, 4);
    if (!apart({md, ml, me}, {vec(targets, T, 8), vec(dlogp, T, 4), vec(dentropy, T, 4)}) || !apart({ml, me}, {mz}) ||
        (!same(md, mz) && overlap(md, mz)))
        return RAR_EINVAL;
    LogprobParams p{};
    p.z = logits;
    p.ldz = ldz;
    p.scale = scale;
    p.targets = targets;
    p.dlogp = dlogp;
    p.dentropy = dentropy;
    p.logp = logp;
    p.entropy = entropy;
    p.dz = dz;
    p.lddz = lddz;
    p.rows = T;
    p.cols = V;
    return launched(launch_logprob(dtype, p, static_cast<hipStream_t>(stream)));
}
