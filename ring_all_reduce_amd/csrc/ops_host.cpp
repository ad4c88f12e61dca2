// ops_host.cpp -- host side of the gradient-producing operators of librar.so:
// argument checks, workspace layout and the launch sequence of each call.  No
// device work is enqueued before every argument has been checked, and nothing
// is allocated on the device.
#include <algorithm>
#include <cstdint>
#include <new>

#include "linear_shape.h"
#include "ops_check.h"
#include "ops_internal.h"

using namespace rar;

struct rar_linear_s {
    int64_t K = 0;
    int64_t N = 0;
    rar_dtype dtype = RAR_F32;
    rar_act act = RAR_ACT_NONE;
};

namespace {

int64_t packed(int64_t cols, rar_dtype dt) { return up(cols, 16 / esize(dt)); }

struct Layer {
    int64_t T, K, N;
    rar_dtype dt;
};

// Chunks of rows whose column sums are kept apart: about 2048 workgroups of 512
// columns, at least 16 rows each.
int64_t sum_rows(int64_t T, int64_t N)
{
    const int64_t chunks = std::max<int64_t>(1, std::min(div_up(T, 16), 2048 / div_up(N, 512)));
    return std::max<int64_t>(1, div_up(T, chunks));
}

struct ForwardWs {
    void *x, *w;
    float *part;
    int64_t bytes;
};

ForwardWs forward_ws(const Layer &l, void *ws)
{
    Carve c{(char *)ws};
    ForwardWs f{};
    const int es = esize(l.dt);
    f.x = c.take(l.T * packed(l.K, l.dt) * es);
    f.w = c.take(l.K * packed(l.N, l.dt) * es);
    f.part = (float *)c.take(shape_of(l.dt, l.T, l.N, l.K).part_bytes);
    f.bytes = l.T > rar::kGemvRows ? c.used : 0;  // few rows need none
    return f;
}

struct BackwardWs {
    void *dz, *x, *w;
    float *sums, *part_x, *part_w;
    int64_t bytes;
};

BackwardWs backward_ws(const Layer &l, void *ws)
{
    Carve c{(char *)ws};
    BackwardWs b{};
    const int es = esize(l.dt);
    b.dz = c.take(l.T * packed(l.N, l.dt) * es);
    b.x = c.take(l.T * packed(l.K, l.dt) * es);
    b.w = c.take(l.K * packed(l.N, l.dt) * es);
    b.sums = (float *)c.take(div_up(l.T, sum_rows(l.T, l.N)) * l.N * 4);
    b.part_x = (float *)c.take(shape_of(l.dt, l.T, l.K, l.N).part_bytes);
    b.part_w = (float *)c.take(shape_of(l.dt, l.K, l.N, l.T).part_bytes);
    b.bytes = l.T ? c.used : 0;
    return b;
}

// Whether the layer's matrices are within the documented size: every product of
// such a layer has a tile whose grid fits a launch.
bool valid_layer(int64_t T, int64_t K, int64_t N)
{
    return T * K <= rar::kMaxOutputs && T * N <= rar::kMaxOutputs && K * N <= rar::kMaxOutputs;
}

// Fills in the shape of a product.
void shape_product(rar_dtype dt, GemmParams &p, float *part, int *tile)
{
    const Shape s = shape_of(dt, p.M, p.N, p.K);
    p.tiles_m = s.tiles_m;
    p.tiles_n = s.tiles_n;
    p.splits = (int)s.splits;
    p.steps_per_split = s.steps;
    p.pitch = s.pitch;
    p.part = part;
    *tile = s.tile;
}

// The product as its launch sees it: partial sums where the reduction is split.
GemmParams launched_form(GemmParams p)
{
    if (p.splits > 1)
        p.mode = rar::kModePartial;
    return p;
}

// Sends an operand whose rows cannot be read directly to a packed copy.
bool needs_pack(const Mat &m, rar_dtype dt, void *copy, const void **p, int64_t *ld, rar::PackParams *k)
{
    *p = m.p;
    *ld = m.ld;
    if (m.empty() || direct(m))
        return false;
    *k = rar::PackParams{m.p, copy, m.ld, packed(m.cols, dt), m.rows, m.cols};
    *p = copy;
    *ld = k->pitch;
    return true;
}

int64_t groups_of(int64_t cols) { return div_up(cols, rar::kCkptGroup); }

}  // namespace

// =============================================================================
// Embedding
// =============================================================================

extern "C" rar_status rar_embed_lookup(int64_t V, int64_t D, rar_dtype dtype, const void *table, int64_t T,
                                       const int64_t *ids, float scale, void *out, int64_t ldo, void *stream)
{
    if (V < 1 || V > kMaxVocab || !valid_width(D) || !valid_dtype(dtype) || !valid_rows(T) || !valid_ld(ldo, D))
        return RAR_EINVAL;
    if (T == 0)
        return RAR_OK;
    if (!table || !ids || !out)
        return RAR_EINVAL;
    const int es = esize(dtype);
    if (!aligned(table, es) || !aligned(out, es) || !aligned(ids, 8))
        return RAR_EALIGN;
    if (!apart({{out, T, D, ldo, es}}, {{table, V, D, D, es}, {ids, 1, T, T, 8}}))
        return RAR_EINVAL;
    rar::EmbedParams p{table, ids, out, T, V, D, ldo, scale};
    return launched(rar::launch_embed_lookup(dtype, p, static_cast<hipStream_t>(stream)));
}

extern "C" rar_status rar_embed_grad_workspace(int64_t V, int64_t D, int64_t T, int64_t *bytes)
{
    if (!bytes || V < 1 || V > kMaxVocab || !valid_width(D) || !valid_rows(T))
        return RAR_EINVAL;
    *bytes = rar::embed_grad_workspace(T, V, D);
    return RAR_OK;
}

extern "C" rar_status rar_embed_grad(int64_t V, int64_t D, rar_dtype dtype, int64_t T, const int64_t *ids,
                                     const void *dy, int64_t lddy, float scale, int accumulate, void *grad, void *ws,
                                     int64_t ws_bytes, void *stream)
{
    if (V < 1 || V > kMaxVocab || !valid_width(D) || !valid_dtype(dtype) || !valid_rows(T) || !valid_ld(lddy, D))
        return RAR_EINVAL;
    if (!grad || (T > 0 && (!ids || !dy || !ws)))
        return RAR_EINVAL;
    const int es = esize(dtype);
    if (!aligned(grad, es) || !aligned(dy, es) || !aligned(ids, 8) || !aligned(ws, 16))
        return RAR_EALIGN;
    const int64_t need = rar::embed_grad_workspace(T, V, D);
    if (ws_bytes < need || !rar::embed_grad_fits(T, D, V * D * es, kMaxLanes))
        return RAR_EINVAL;
    if (!apart({{grad, V, D, D, es}, {ws, 1, need, need, 1}}, {{dy, T, D, lddy, es}, {ids, 1, T, T, 8}}))
        return RAR_EINVAL;
    rar::EmbedGradParams p{ids, dy, lddy, grad, T, V, D, scale, accumulate, ws};
    return launched(rar::launch_embed_grad(dtype, p, static_cast<hipStream_t>(stream)));
}

// =============================================================================
// Linear layer
// =============================================================================

extern "C" rar_status rar_linear_plan(int64_t K, int64_t N, rar_dtype dtype, rar_act act, rar_linear_t *out)
{
    if (!out)
        return RAR_EINVAL;
    *out = nullptr;
    if (!valid_width(K) || !valid_width(N) || !valid_dtype(dtype) || !valid_act(act))
        return RAR_EINVAL;
    rar_linear_s *p = new (std::nothrow) rar_linear_s;
    if (!p)
        return RAR_ENOMEM;
    p->K = K;
    p->N = N;
    p->dtype = dtype;
    p->act = act;
    *out = p;
    return RAR_OK;
}

extern "C" rar_status rar_linear_destroy(rar_linear_t plan)
{
    delete plan;
    return RAR_OK;
}

extern "C" rar_status rar_linear_workspace(rar_linear_t plan, int64_t T, int64_t *forward_bytes,
                                           int64_t *backward_bytes)
{
    if (!plan || !valid_rows(T) || !valid_layer(T, plan->K, plan->N))
        return RAR_EINVAL;
    const Layer l{T, plan->K, plan->N, plan->dtype};
    if (forward_bytes)
        *forward_bytes = forward_ws(l, nullptr).bytes;
    if (backward_bytes)
        *backward_bytes = backward_ws(l, nullptr).bytes;
    return RAR_OK;
}

extern "C" rar_status rar_linear_forward(rar_linear_t plan, int64_t T, const void *x, int64_t ldx, const void *w,
                                         const void *bias, const void *residual, int64_t ldr, void *y, int64_t ldy,
                                         void *pre, int64_t ldp, uint8_t *pre_scales, void *ws, int64_t ws_bytes,
                                         void *stream)
{
    if (!plan || !valid_rows(T) || !valid_layer(T, plan->K, plan->N))
        return RAR_EINVAL;
    if (T == 0)
        return RAR_OK;
    const int64_t K = plan->K, N = plan->N;
    const rar_dtype dt = plan->dtype;
    const int es = esize(dt);
    if (!x || !w || !y || (!ws && T > rar::kGemvRows) || (pre_scales && !pre))
        return RAR_EINVAL;
    if (!valid_ld(ldx, K) || !valid_ld(ldy, N) || (residual && !valid_ld(ldr, N)) ||
        (pre && !pre_scales && !valid_ld(ldp, N)))
        return RAR_EINVAL;
    if (!aligned(x, es) || !aligned(w, es) || !aligned(bias, es) || !aligned(residual, es) || !aligned(y, es) ||
        !aligned(pre, pre_scales ? 16 : es) || !aligned(ws, 16))
        return RAR_EALIGN;
    const Layer l{T, K, N, dt};
    const ForwardWs f = forward_ws(l, ws);
    if (ws_bytes < f.bytes)
        return RAR_EINVAL;
    const int64_t groups = groups_of(N), pitch = groups * rar::kCkptGroup;
    const Mat mx{x, T, K, ldx, es}, mw{w, K, N, N, es}, my{y, T, N, ldy, es}, mb{bias, 1, N, N, es};
    const Mat mr{residual, T, N, ldr, es};
    const Mat mp = pre_scales ? Mat{pre, 1, T * pitch, T * pitch, 1} : Mat{pre, T, N, ldp, es};
    const Mat ms{pre_scales, 1, T * groups, T * groups, 1}, mws{ws, 1, f.bytes, f.bytes, 1};
    const bool in_place = residual == y && ldr == ldy;
    if (!apart({my, mp, ms, mws}, {mx, mw, mb}) || (residual && !in_place && !apart({my}, {mr})) ||
        (residual && !apart({mp, ms, mws}, {mr})))
        return RAR_EINVAL;
    hipStream_t st = static_cast<hipStream_t>(stream);
    GemmParams p{};
    p.M = T;
    p.N = N;
    p.K = K;
    p.out = y;
    p.ldo = ldy;
    p.pre = pre;
    p.ldp = ldp;
    p.pre_scales = pre_scales;
    p.bias = bias;
    p.res = residual;
    p.ldr = ldr;
    p.mode = rar::kModeForward;
    p.act = plan->act;
    if (T <= rar::kGemvRows) {
        p.a = x;
        p.lda = ldx;
        p.b = w;
        p.ldb = N;
        return launched(rar::launch_gemv(dt, p, N * es % 16 == 0, st));
    }
    rar::PackParams kx{}, kw{};
    int tile;
    const bool px = needs_pack(mx, dt, f.x, &p.a, &p.lda, &kx), pw = needs_pack(mw, dt, f.w, &p.b, &p.ldb, &kw);
    shape_product(dt, p, f.part, &tile);
    rar_status rc = px || pw ? launched(rar::launch_pack(dt, kx, kw, st)) : RAR_OK;
    if (rc == RAR_OK)
        rc = launched(rar::launch_forward(dt, launched_form(p), tile, st));
    if (rc == RAR_OK && p.splits > 1) {
        rar::FinishParams e{};
        e.a = p;
        e.a_blocks = rar::join_blocks(p);
        rc = launched(rar::launch_finish(dt, e, st));
    }
    return rc;
}

extern "C" rar_status rar_linear_backward(rar_linear_t plan, int64_t T, const void *dy, int64_t lddy, const void *x,
                                          int64_t ldx, const uint8_t *x_scales, const void *w, const void *pre,
                                          int64_t ldp, const uint8_t *pre_scales, void *dx, int64_t lddx, void *dw,
                                          void *db, int accumulate, void *ws, int64_t ws_bytes, void *stream)
{
    if (!plan || !valid_rows(T) || !valid_layer(T, plan->K, plan->N))
        return RAR_EINVAL;
    const int64_t K = plan->K, N = plan->N;
    const rar_dtype dt = plan->dtype;
    const int es = esize(dt);
    const bool act = plan->act != RAR_ACT_NONE;
    if (!act) {
        pre = nullptr;
        pre_scales = nullptr;
    }
    const Layer l{T, K, N, dt};
    const BackwardWs b = backward_ws(l, ws);
    if (T > 0) {
        if (!dy || !ws || (dx && !w) || (dw && !x) || (act && !pre))
            return RAR_EINVAL;
        if (!valid_ld(lddy, N) || (dx && !valid_ld(lddx, K)) || (dw && !x_scales && !valid_ld(ldx, K)) ||
            (act && !pre_scales && !valid_ld(ldp, N)))
            return RAR_EINVAL;
    } else {
        dx = nullptr;
    }
    if (!aligned(dy, es) || !aligned(x, x_scales ? 16 : es) || !aligned(w, es) || !aligned(pre, pre_scales ? 16 : es) ||
        !aligned(dx, es) || !aligned(dw, es) || !aligned(db, es) || !aligned(ws, 16))
        return RAR_EALIGN;
    if (ws_bytes < b.bytes)
        return RAR_EINVAL;
    const int64_t gk = groups_of(K), gn = groups_of(N);
    const Mat mdy{dy, T, N, lddy, es}, mw{dx ? w : nullptr, K, N, N, es};
    Mat mx{dw ? x : nullptr, T, K, ldx, es}, mp{pre, T, N, ldp, es};
    if (x_scales)
        mx = Mat{dw ? x : nullptr, 1, T * gk * rar::kCkptGroup, T * gk * rar::kCkptGroup, 1};
    if (pre_scales)
        mp = Mat{pre, 1, T * gn * rar::kCkptGroup, T * gn * rar::kCkptGroup, 1};
    const Mat mxs{dw ? x_scales : nullptr, 1, T * gk, T * gk, 1}, mps{pre_scales, 1, T * gn, T * gn, 1};
    const Mat mdx{dx, T, K, lddx, es}, mdw{dw, K, N, N, es}, mdb{db, 1, N, N, es}, mws{ws, 1, b.bytes, b.bytes, 1};
    if (!apart({mdx, mdw, mdb, mws}, {mdy, mx, mw, mp, mxs, mps}))
        return RAR_EINVAL;

    const bool need_dz = (dx || dw) && T > 0 && (act || !direct(mdy));
    const void *const dz = need_dz ? b.dz : dy;
    const int64_t lddz = need_dz ? packed(N, dt) : lddy;
    rar::PackParams kx{}, kw{};
    bool px = false, pw = false;
    GemmParams gx{}, gw{};
    int tile_x = 0, tile_w = 0;
    if (dx) {
        gx.a = dz;
        gx.lda = lddz;
        pw = needs_pack(mw, dt, b.w, &gx.b, &gx.ldb, &kw);
        gx.M = T;
        gx.N = K;
        gx.K = N;
        gx.out = dx;
        gx.ldo = lddx;
        gx.mode = rar::kModeStore;
        shape_product(dt, gx, b.part_x, &tile_x);
    }
    if (dw) {
        if (x_scales) {
            gw.a = b.x;
            gw.lda = packed(K, dt);
        } else {
            px = needs_pack(mx, dt, b.x, &gw.a, &gw.lda, &kx);
        }
        gw.b = dz;
        gw.ldb = lddz;
        gw.M = K;
        gw.N = N;
        gw.K = T;
        gw.out = dw;
        gw.ldo = N;
        gw.mode = rar::kModeStore;
        gw.accumulate = accumulate;
        shape_product(dt, gw, b.part_w, &tile_w);
    }

    hipStream_t st = static_cast<hipStream_t>(stream);
    rar_status rc = px || pw ? launched(rar::launch_pack(dt, kx, kw, st)) : RAR_OK;
    if (rc == RAR_OK && dw && x_scales && T > 0) {
        rar::CkptParams c{};
        c.codes = (uint8_t *)x;
        c.scales = (uint8_t *)x_scales;
        c.y = b.x;
        c.ldy = packed(K, dt);
        c.pitch_zero = c.ldy;
        c.rows = T;
        c.cols = K;
        c.act = RAR_ACT_NONE;
        rc = launched(rar::launch_ckpt_load(dt, c, st));
    }
    if (rc == RAR_OK && T > 0 && (need_dz || db)) {
        rar::DzParams d{};
        d.dy = dy;
        d.ldy = lddy;
        d.pre = pre;
        d.ldp = ldp;
        d.pre_scales = pre_scales;
        d.pitch = packed(N, dt);
        d.dz = need_dz ? b.dz : nullptr;
        d.part = db ? b.sums : nullptr;
        d.rows = T;
        d.cols = N;
        d.rows_per_chunk = sum_rows(T, N);
        d.act = plan->act;
        rc = launched(rar::launch_dz(dt, d, st));
    }
    // the two products together where they take the same kernel and fit one grid
    rar::GemmPair pair{launched_form(gx), launched_form(gw), dx ? rar::blocks_of(gx) : 0};
    const unsigned w_blocks = dw ? rar::blocks_of(gw) : 0;
    if (rc == RAR_OK && dx && dw && tile_x == tile_w &&
        (int64_t)pair.x_blocks + w_blocks <= most_blocks(dt, tile_x)) {
        rc = launched(rar::launch_backward(dt, pair, w_blocks, tile_x, st));
    } else {
        if (rc == RAR_OK && dx)
            rc = launched(rar::launch_backward(dt, pair, 0, tile_x, st));
        pair.x_blocks = 0;
        if (rc == RAR_OK && dw)
            rc = launched(rar::launch_backward(dt, pair, w_blocks, tile_w, st));
    }
    rar::FinishParams e{};
    if (dx) {
        e.a = gx;
        e.a_blocks = rar::join_blocks(gx);
    }
    if (dw) {
        e.b = gw;
        e.b_blocks = rar::join_blocks(gw);
    }
    if (db)
        e.sum = rar::SumParams{b.sums, T > 0 ? div_up(T, sum_rows(T, N)) : 0, N, db, accumulate};
    if (rc == RAR_OK && (e.a_blocks || e.b_blocks || db))
        rc = launched(rar::launch_finish(dt, e, st));
    return rc;
}

// =============================================================================
// 8-bit checkpoints
// =============================================================================

extern "C" rar_status rar_ckpt_size(int64_t D, int64_t *pitch, int64_t *groups)
{
    if (!valid_width(D))
        return RAR_EINVAL;
    if (pitch)
        *pitch = groups_of(D) * rar::kCkptGroup;
    if (groups)
        *groups = groups_of(D);
    return RAR_OK;
}

namespace {

rar_status check_ckpt(int64_t T, int64_t D, rar_dtype dt, const void *m, int64_t ld, const uint8_t *codes,
                      const uint8_t *scales, bool store)
{
    if (!valid_rows(T) || !valid_width(D) || !valid_dtype(dt) || !valid_ld(ld, D))
        return RAR_EINVAL;
    if (T == 0)
        return RAR_OK;
    if (!m || !codes || !scales)
        return RAR_EINVAL;
    const int es = esize(dt);
    if (!aligned(m, es) || !aligned(codes, 16))
        return RAR_EALIGN;
    const int64_t g = groups_of(D) * T, c = g * rar::kCkptGroup;
    if (g > kMaxLanes - 256)  // four lanes move four groups each
        return RAR_EINVAL;
    const Mat mm{m, T, D, ld, es}, mc{codes, 1, c, c, 1}, ms{scales, 1, g, g, 1};
    if (store ? !apart({mc, ms}, {mm}) : !apart({mm}, {mc, ms}))
        return RAR_EINVAL;
    return RAR_OK;
}

}  // namespace

extern "C" rar_status rar_ckpt_store(int64_t T, int64_t D, rar_dtype dtype, const void *x, int64_t ldx, uint8_t *codes,
                                     uint8_t *scales, void *stream)
{
    const rar_status rc = check_ckpt(T, D, dtype, x, ldx, codes, scales, true);
    if (rc != RAR_OK || T == 0)
        return rc;
    rar::CkptParams p{};
    p.x = x;
    p.ldx = ldx;
    p.codes = codes;
    p.scales = scales;
    p.rows = T;
    p.cols = D;
    return launched(rar::launch_ckpt_store(dtype, p, static_cast<hipStream_t>(stream)));
}

extern "C" rar_status rar_ckpt_load(int64_t T, int64_t D, rar_dtype dtype, const uint8_t *codes, const uint8_t *scales,
                                    rar_act act, void *y, int64_t ldy, void *stream)
{
    if (!valid_act(act))
        return RAR_EINVAL;
    const rar_status rc = check_ckpt(T, D, dtype, y, ldy, codes, scales, false);
    if (rc != RAR_OK || T == 0)
        return rc;
    rar::CkptParams p{};
    p.codes = (uint8_t *)codes;
    p.scales = (uint8_t *)scales;
    p.y = y;
    p.ldy = ldy;
    p.rows = T;
    p.cols = D;
    p.act = act;
    return launched(rar::launch_ckpt_load(dtype, p, static_cast<hipStream_t>(stream)));
}
