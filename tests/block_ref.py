"""Plain 64-bit forms of the norms around a block, dropout, cross attention and
log probabilities, with error bounds that count roundings (see ops_ref.py).

`U` is half a step of the type relative to the value, `E` that of binary32.  A
row's sum is taken eight elements a lane (more where a row has over 8192), then
over the 64 lanes of a wave, then over at most 16 waves, so a term passes
through at most `depth` additions.  exp2, the square root, the division and the
logarithm are good to two steps of binary32; exp2 gives zero for a result under
2^-126, the smallest normal number, so a weight may be off by that (`TINY`) times
what it multiplies.  Bounds of products of small errors are covered by a factor of
1.1.
"""
import math

import numpy as np
import torch

from ops_ref import DT, U, check  # noqa: F401

E = 2.0 ** -24
TINY = 2.0 ** -126
KINDS = {"none": 0, "layer": 1, "rms": 2}
INF = math.inf


def depth(D):
    return 8 * -(-D // 8192) + 6 + 16


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------

def _stats(v, ev, kind, eps):
    """(v^, its error, r) of rows v known to ev."""
    D, n = v.shape[1], depth(v.shape[1])
    if kind == "none":
        return v, ev, torch.ones_like(v[:, :1])
    d, ed = v, ev
    if kind == "layer":
        mean = v.mean(1, keepdim=True)
        em = ev.mean(1, keepdim=True) + (n + 2) * E * v.abs().mean(1, keepdim=True)
        d = v - mean
        ed = ev + em + E * d.abs()
    var = (d * d).mean(1, keepdim=True)
    evar = 2 * (d.abs() * ed).mean(1, keepdim=True) + (ed * ed).mean(1, keepdim=True) + (n + 3) * E * var
    r = (var + eps) ** -0.5
    rel = evar / (var + eps) / 2 + 4 * E
    return d * r, 1.1 * (ed * r + d.abs() * r * (rel + E)), r


def _affine(v, ev, w, b):
    if w is not None:
        v, ev = v * w.double(), ev * w.double().abs()
    if b is not None:
        v = v + b.double()
        ev = ev + E * v.abs()
    return v, ev + E * v.abs()


def norm_forward(x, o, post_w, post_b, gate, pre_w, pre_b, post, pre, eps, a, s, dtype):
    """((h, bound), (u, bound)); x, o ... as the call reads them."""
    u = U[dtype]
    h = a * x.double()
    eh = E * h.abs()
    if o is not None:
        n, en, _ = _stats(o.double(), torch.zeros_like(h), post, eps)
        if post != "none":
            n, en = _affine(n, en, post_w, post_b)
        g = torch.ones(x.shape[1], dtype=torch.float64) if gate is None else gate.double()
        t = s * g * n
        h = h + t
        eh = eh + (s * g).abs() * en + 3 * E * t.abs() + E * h.abs()
    y, ey, _ = _stats(h, eh, pre, eps)
    if pre != "none":
        y, ey = _affine(y, ey, pre_w, pre_b)
    return (h, eh * (1 + u) + u * h.abs()), (y, ey * (1 + u) + u * y.abs())


def _norm_back(q, eq, vh, evh, r, rel, kind):
    """r (q - mean(q) - v^ mean(q v^)) and its error."""
    if kind == "none":
        return q, eq
    n = depth(q.shape[1])
    m2 = (q * vh).mean(1, keepdim=True)
    em2 = (eq * vh.abs() + q.abs() * evh).mean(1, keepdim=True) + (n + 3) * E * (q * vh).abs().mean(1, keepdim=True)
    t = q - vh * m2
    et = eq + evh * m2.abs() + vh.abs() * em2 + 2 * E * (q.abs() + (vh * m2).abs())
    if kind == "layer":
        m1 = q.mean(1, keepdim=True)
        t = t - m1
        et = et + eq.mean(1, keepdim=True) + (n + 2) * E * q.abs().mean(1, keepdim=True) + 2 * E * (m1.abs() + t.abs())
    return t * r, 1.1 * r * (et + t.abs() * (rel + 2 * E))


def norm_backward(dh, du, o, h, post_w, post_b, gate, pre_w, post, pre, eps, a, s, dtype, before=None):
    """{name: (value, bound)} of every gradient; before: vectors that are added to."""
    u = U[dtype]
    some = next(t for t in (dh, du, o, h) if t is not None)
    T, D = some.shape
    z = torch.zeros(T, D, dtype=torch.float64)
    one = torch.ones(D, dtype=torch.float64)
    n = depth(D)
    dh = z if dh is None else dh.double()
    du = None if du is None else du.double()
    w1 = one if post_w is None or post == "none" else post_w.double()
    b1 = 0 * one if post_b is None or post == "none" else post_b.double()
    w2 = one if pre_w is None or pre == "none" else pre_w.double()
    gt = one if gate is None else gate.double()

    def rel(v, kind):
        if kind == "none":
            return 0.0
        d = v - v.mean(1, keepdim=True) if kind == "layer" else v
        var = (d * d).mean(1, keepdim=True)
        em = (n + 2) * E * v.abs().mean(1, keepdim=True) if kind == "layer" else 0.0
        return (2 * d.abs().mean(1, keepdim=True) * em + em * em + (n + 3) * E * var) / (var + eps) / 2 + 4 * E

    out = {}
    g, eg = dh, z
    if du is not None:
        if pre == "none":
            g = g + du
            eg = E * g.abs()
        else:
            hd = h.double()
            hh, ehh, r = _stats(hd, z, pre, eps)
            q = du * w2
            t, et = _norm_back(q, E * q.abs(), hh, ehh, r, rel(hd, pre), pre)
            g = g + t
            eg = et + E * g.abs()
            out["dpre_w"] = ((du * hh).sum(0), (du.abs() * ehh + T * 2 * E * (du * hh).abs()).sum(0))
            out["dpre_b"] = (du.sum(0), T * 2 * E * du.abs().sum(0))
    elif pre != "none":
        out["dpre_w"] = out["dpre_b"] = (torch.zeros(D, dtype=torch.float64),) * 2
    out["dx"] = (a * g, abs(a) * eg + E * (a * g).abs())
    if o is not None:
        od = o.double()
        oh, eoh, r = _stats(od, z, post, eps)
        q = s * gt * w1 * g
        eq = (s * gt * w1).abs() * eg + 3 * E * q.abs()
        t, et = _norm_back(q, eq, oh, eoh, r, rel(od, post), post)
        out["do"] = (t, et)
        A, eA = (g * oh).sum(0), (eg * oh.abs() + g.abs() * eoh + T * 2 * E * (g * oh).abs()).sum(0)
        B, eB = g.sum(0), (eg + T * 2 * E * g.abs()).sum(0)
        n_ = w1 * A + b1 * B
        out["dgate"] = (s * n_, abs(s) * (w1.abs() * eA + b1.abs() * eB + 4 * E * ((w1 * A).abs() + (b1 * B).abs())))
        if post != "none":
            out["dpost_w"] = (s * gt * A, (s * gt).abs() * (eA + 3 * E * A.abs()))
            out["dpost_b"] = (s * gt * B, (s * gt).abs() * (eB + 3 * E * B.abs()))
    done = {}
    for k, (v, e) in out.items():
        if before is not None and k in before:
            v = v + before[k].double()
            e = e + 2 * E * (v.abs() + before[k].double().abs())
        done[k] = (v, 1.1 * e * (1 + u) + u * v.abs())
    return done


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------

def philox(counter, key):
    """Philox4x32-10 of [n, 4] counters, in numpy."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k0, k1 = key
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k0), b & low, (a >> sh) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1)


def keep_mask(T, D, p, seed, step, first=0):
    G = -(-D // 8)
    g = np.arange(first, first + T * G, dtype=np.uint64)
    step &= (1 << 64) - 1
    counter = np.stack([g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), np.full(T * G, step & 0xFFFFFFFF, np.uint64),
                        np.full(T * G, step >> 32, np.uint64)], 1)
    w = philox(counter, (seed & 0xFFFFFFFF, seed >> 32)).astype("<u4").view("<u2")
    thr = math.floor(float(np.float32(p)) * 65536 + 0.5)
    return torch.from_numpy((w.reshape(T, G * 8)[:, :D] >= thr).copy()), (65536 / (65536 - thr) if thr < 65536 else 0.0)


def dropout(x, r, p, seed, step, dtype):
    keep, scale = keep_mask(*x.shape, p, seed, step)
    y = torch.where(keep, x.double() * scale, 0.0)
    e = 2 * E * y.abs()
    if r is not None:
        y = y + r.double()
        e = e + E * y.abs()
    return y, e * (1 + U[dtype]) + U[dtype] * y.abs()


# ---------------------------------------------------------------------------
# Cross attention
# ---------------------------------------------------------------------------

def heads(m, B, n):
    """[B n_rows, n dh] as [B, n, n_rows, dh]."""
    return m.double().view(B, -1, n, m.shape[1] // n).transpose(1, 2)


def rows(x):
    B, H, n, d = x.shape
    return x.transpose(1, 2).reshape(B * n, H * d)


def _scores(q, k, scale, klen):
    """(S, |error|, live) [B, H, Tq, Tk]; keys behind klen are -infinity."""
    dh, Tk = q.shape[3], k.shape[2]
    S = scale * (q @ k.transpose(2, 3))
    eS = (dh + 3) * 2 * E * abs(scale) * (q.abs() @ k.abs().transpose(2, 3))
    live = (torch.arange(Tk) < klen.view(-1, 1)).view(-1, 1, 1, Tk)
    return torch.where(live, S, -INF), torch.where(live, eS, 0.0), live


def _lens(lens, B, most):
    return torch.full((B,), most) if lens is None else lens.clamp(0, most)


def _clean(m, lens, B, n):
    """Rows behind the lengths as zeros: what they hold does not count."""
    on = (torch.arange(n) < lens.view(-1, 1)).reshape(B * n, 1)
    return torch.where(on, m.double(), 0.0)


def attn_forward(q, k, v, B, H, Hkv, scale, qlen, klen, dtype):
    """((o, bound), (lse, bound)): [B Tq, H dh] and [B Tq, H]."""
    u, low = U[dtype], (0.0 if dtype == "f32" else U[dtype])
    Tq, Tk = q.shape[0] // B, k.shape[0] // B
    ql, kl = _lens(qlen, B, Tq), _lens(klen, B, Tk)
    q, k, v = _clean(q, ql, B, Tq), _clean(k, kl, B, Tk), _clean(v, kl, B, Tk)
    q, k, v = heads(q, B, H), heads(k, B, Hkv), heads(v, B, Hkv)
    k, v = (t.repeat_interleave(H // Hkv, 1) for t in (k, v))
    S, eS, live = _scores(q, k, scale, kl)
    m = S.amax(3, keepdim=True) if Tk else torch.full((*S.shape[:3], 1), -INF, dtype=torch.float64)
    base = torch.where(m == -INF, 0.0, m)
    P = torch.exp(S - base)
    l = P.sum(3, keepdim=True)
    # a weight's relative error: of its score (and of the maximum, the same in every weight and in the sum), of
    # the exponent's argument, which is formed from numbers as large as score and maximum, and of exp2
    rel = eS + torch.where(live, 4 * E * (S.abs().nan_to_num(0, 0, 0) + base.abs()), 0.0) + 6 * E
    n = Tk + 64
    el = (P * rel).sum(3, keepdim=True) + n * 2 * E * l
    safe = torch.where(l == 0, 1.0, l)
    o = (P @ v) / safe
    mag = (P @ v.abs()) / safe
    eo = ((P * (rel + low) + torch.where(live, TINY, 0.0)) @ v.abs()) / safe
    eo = eo + mag * (el / safe + n * 2 * E) + 4 * E * mag
    on = (torch.arange(Tq) < ql.view(-1, 1)).view(B, 1, Tq, 1)
    o, eo = torch.where(on, o, 0.0), torch.where(on, eo, 0.0)
    lse = torch.where(on & (l > 0), base + torch.log(safe), -INF)
    el = torch.where(on & (l > 0), el / safe + 4 * E * (base.abs() + torch.log(safe).abs()) + eS.amax(3, keepdim=True)
                     if Tk else 0.0, 0.0)
    flat = lambda t: t.squeeze(3).transpose(1, 2).reshape(B * Tq, H)  # noqa: E731
    return (rows(o), rows(1.1 * eo * (1 + u) + u * o.abs())), (flat(lse), flat(1.1 * el) + 0)


def attn_backward(do, q, k, v, o, lse, B, H, Hkv, scale, qlen, klen, dtype):
    """((dq, bound), (dk, bound), (dv, bound)) for the o and lse that the call reads."""
    u, low = U[dtype], (0.0 if dtype == "f32" else U[dtype])
    Tq, Tk, share = q.shape[0] // B, k.shape[0] // B, H // Hkv
    ql, kl = _lens(qlen, B, Tq), _lens(klen, B, Tk)
    q, o, do = (heads(_clean(t, ql, B, Tq), B, H) for t in (q, o, do))
    k, v = (heads(_clean(t, kl, B, Tk), B, Hkv).repeat_interleave(share, 1) for t in (k, v))
    S, eS, live = _scores(q, k, scale, kl)
    on = (torch.arange(Tq) < ql.view(-1, 1)).view(B, 1, Tq, 1)
    L = lse.double().view(B, Tq, H).transpose(1, 2).unsqueeze(3)
    counts = on & (L > -INF) & live
    L0 = torch.where(torch.isfinite(L), L, 0.0)
    S0 = torch.where(live, S, 0.0)
    P = torch.where(counts, torch.exp(S0 - L0), 0.0)
    rel = eS + 4 * E * (S0.abs() + L0.abs()) + 6 * E
    dh = q.shape[3]
    X, eX = do @ v.transpose(2, 3), (dh + 2) * 2 * E * (do.abs() @ v.abs().transpose(2, 3))
    d, ed = (do * o).sum(3, keepdim=True), (dh + 2) * 2 * E * (do * o).abs().sum(3, keepdim=True)
    dS = P * (X - d)
    eP = P * rel + torch.where(counts, TINY, 0.0)
    eS_ = eP * (X - d).abs() + P * (eX + ed + 2 * E * (X.abs() + d.abs())) + 2 * E * dS.abs()
    eP, eS_ = eP * (1 + low) + low * P, eS_ * (1 + low) + low * dS.abs()

    def total(a, ea, b, n):
        return a @ b, ea @ b.abs() + n * 2 * E * (a.abs() @ b.abs())

    def close(t, e, f):
        t, e = t * f, e * abs(f) + E * (t * f).abs()
        return rows(t), rows(1.1 * e * (1 + u) + u * t.abs())

    def shared(t):
        return t.view(B, Hkv, share, Tk, dh).sum(2)

    dq = total(dS, eS_, k, Tk + 64)
    dk = total(dS.transpose(2, 3), eS_.transpose(2, 3), q, Tq * share + 64)
    dv = total(P.transpose(2, 3), eP.transpose(2, 3), do, Tq * share + 64)
    return close(*dq, scale), close(*(shared(t) for t in dk), scale), close(*(shared(t) for t in dv), 1.0)


# ---------------------------------------------------------------------------
# Log probabilities
# ---------------------------------------------------------------------------

def _log_softmax(z, scale):
    """(log p, its error, p, its relative error, entropy, its error) for rows with something left."""
    V = z.shape[1]
    n = depth(V) + 8 * -(-V // 8192)
    s = z.double() * scale
    m = s.amax(1, keepdim=True)
    base = torch.where(m == -INF, 0.0, m)
    d = base - s
    fd = torch.where(torch.isfinite(d), d, 0.0)
    e = torch.exp(-d)
    re = 4 * E * fd + 4 * E                       # argument and exp2
    S = e.sum(1, keepdim=True)
    rs = ((e * re).sum(1, keepdim=True) + n * E * S) / S
    ls = torch.log(S)
    els = rs + 4 * E * ls.abs() + 2 * E
    lp = -d - ls
    elp = 3 * E * fd + els + E * lp.abs().nan_to_num(0, 0, 0)
    p = e / S
    w = (e * fd).sum(1, keepdim=True) / S
    ew = ((e * fd * (re + 3 * E)).sum(1, keepdim=True)) / S + w * (rs + (n + 3) * E)
    return lp, elp, p, re + rs + 3 * E, ls + w, els + ew + E * (ls + w)


def logprob(z, targets, scale):
    """((logp, bound), (entropy, bound)): [T]."""
    lp, elp, _, _, H, eH = _log_softmax(z, scale)
    T, V = z.shape
    ok = (targets >= 0) & (targets < V)
    at = torch.where(ok, targets, 0).unsqueeze(1)
    lp, elp = lp.gather(1, at).squeeze(1), elp.gather(1, at).squeeze(1)
    return (torch.where(ok, lp, 0.0), 1.1 * torch.where(ok, elp, 0.0)), (H.squeeze(1), 1.1 * eH.squeeze(1))


def top(z, scale, K):
    """(ids, logp, bound) [T, K]: by value, then by the lower index; -1 where nothing is left."""
    lp, elp, *_ = _log_softmax(z, scale)
    T, V = z.shape
    ids = torch.full((T, K), -1, dtype=torch.int64)
    out, e = torch.full((T, K), -INF, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        row = z[t].double().numpy()
        order = np.lexsort((np.arange(V), -row))
        order = [int(i) for i in order if row[i] > -INF][:K]
        for k, i in enumerate(order):
            ids[t, k], out[t, k], e[t, k] = i, lp[t, i], 1.1 * elp[t, i]
    return ids, out, e


def logprob_grad(z, targets, dlogp, dent, scale, dtype):
    """(dz, bound)."""
    T, V = z.shape
    lp, elp, p, rp, H, eH = _log_softmax(z, scale)
    ok = (targets >= 0) & (targets < V) if targets is not None else torch.zeros(T, dtype=torch.bool)
    dl = torch.where(ok, dlogp.double(), 0.0).unsqueeze(1) if dlogp is not None else torch.zeros(T, 1).double()
    de = dent.double().unsqueeze(1) if dent is not None else torch.zeros(T, 1).double()
    flp = torch.where(torch.isfinite(lp), lp, 0.0)
    w = dl + de * (flp + H)
    ew = de.abs() * (elp + eH + 2 * E * (flp.abs() + H)) + 2 * E * (dl.abs() + w.abs())
    g = -p * w
    eg = p * ew + g.abs() * (rp + 3 * E) + TINY * w.abs()
    if targets is not None:
        hot = torch.zeros_like(g).scatter_(1, torch.where(ok, targets, 0).unsqueeze(1), dl)
        g = g + hot
        eg = eg + 2 * E * (g.abs() + hot.abs())
    g, eg = g * scale, eg * scale + 2 * E * (g * scale).abs()
    u = U[dtype]
    return g, 1.1 * eg * (1 + u) + u * g.abs()
