"""Plain 64-bit forms of the gradient-producing operators, and error bounds.

Bounds: `U` is half a step of the type relative to the value.  A binary32 sum
of n products is off by at most n * 2^-23 times the sum of the products'
magnitudes (each addition rounds once; one bit is left for the order and the
internal rounding of the matrix instructions).  The activation functions are
evaluated in binary32 with an error of at most 2^-20 (1 + |z|).
"""
import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
SUM = 2.0 ** -23
ACT_ERR = 2.0 ** -20
ACTS = {"none": 0, "relu": 1, "gelu": 2}


def phi(z):
    return 0.5 * torch.special.erfc(-z / 2 ** 0.5)


def act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * phi(z)
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return phi(z) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    return torch.ones_like(z)


def forward(x, w, b, r, name, dtype):
    """((y, bound), (z, bound)) in 64 bits."""
    K = x.shape[1]
    x, w = x.double(), w.double()
    z = x @ w
    mag = x.abs() @ w.abs()
    if b is not None:
        z = z + b.double()
        mag = mag + b.double().abs()
    ez = (K + 2) * SUM * mag
    a = act(z, name)
    # |act'| < 1.13
    ey = 1.13 * ez + (ACT_ERR * (1 + z.abs()) if name == "gelu" else 0)
    y = a
    if r is not None:
        y = y + r.double()
        ey = ey + 2 ** -24 * y.abs() + 2 ** -24 * a.abs()
    u = U[dtype]
    return (y, ey * (1 + u) + u * y.abs()), (z, ez * (1 + u) + u * z.abs())


def backward(dy, x, w, z, name, dtype, dw0=None, db0=None):
    """((dx, bound), (dw, bound), (db, bound)) in 64 bits; z and x are what the call reads."""
    T, N = dy.shape
    u = U[dtype]
    dy, x, w, z = dy.double(), x.double(), w.double(), z.double()
    g = act_grad(z, name)
    dz = dy * g
    edz = 2 ** -23 * dz.abs() + (ACT_ERR * (1 + z.abs()) * dy.abs() if name == "gelu" else 0)
    er = edz * (1 + u) + (0 if name == "none" else u) * dz.abs()   # after rounding to the layer's type
    out = []
    dx = dz @ w.T
    e = er @ w.abs().T + N * SUM * (dz.abs() @ w.abs().T)
    out.append((dx, e * (1 + u) + u * dx.abs()))
    dw = x.T @ dz
    e = x.abs().T @ er + T * SUM * (x.abs().T @ dz.abs())
    if dw0 is not None:
        dw = dw + dw0.double()
        e = e + 2 ** -23 * (dw.abs() + dw0.double().abs())
    out.append((dw, e * (1 + u) + u * dw.abs()))
    db = dz.sum(0)
    e = edz.sum(0) + T * SUM * dz.abs().sum(0)
    if db0 is not None:
        db = db + db0.double()
        e = e + 2 ** -23 * (db.abs() + db0.double().abs())
    out.append((db, e * (1 + u) + u * db.abs()))
    return out


def quantise(x):
    """(codes uint8 [T, pitch], scales uint8 [T, groups], values float64 [T, D]) of an 8-bit checkpoint, from the
    definition, in numpy.  x: a 2-D torch tensor on the CPU."""
    v = x.double().numpy()
    T, D = v.shape
    G = -(-D // 32)
    p = np.zeros((T, G * 32))
    p[:, :D] = v
    p = p.reshape(T, G, 32)
    fin = np.isfinite(p)
    amax = np.abs(np.where(fin, p, 0)).max(-1)
    e = np.full(amax.shape, -126)
    for k in range(-125, 122):                       # the smallest e with amax <= 448 * 2^e
        e = np.where(amax > 448 * 2.0 ** (k - 1), k, e)
    scaled = np.where(fin, p, 0) / (2.0 ** e)[..., None]
    # every e4m3 value of a sign bit of 0, in order
    grid = np.array([(m / 8 * 2.0 ** -6) if ex == 0 else (1 + m / 8) * 2.0 ** (ex - 7)
                     for ex in range(16) for m in range(8)][:127])
    a = np.abs(scaled)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(a == grid[hi], hi, pick)
    vals = np.where(np.signbit(p), -grid[pick], grid[pick]) * (2.0 ** e)[..., None]
    vals = np.where(fin, vals, np.nan)
    codes = np.where(fin, pick, 127).astype(np.uint8) | (np.signbit(p).astype(np.uint8) << 7)
    return codes.reshape(T, G * 32), (e + 127).astype(np.uint8), vals.reshape(T, G * 32)[:, :D]


def values(codes, scales, D):
    """What a checkpoint stands for, float64 torch [T, D], from numpy arrays."""
    c = codes.astype(np.int64)
    ex, m = (c >> 3) & 15, c & 7
    mag = np.where(ex == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (ex - 7.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    v = np.where(c >= 128, -mag, mag)
    s = 2.0 ** (scales.astype(np.float64) - 127)
    return torch.from_numpy((v * np.repeat(s, 32, 1))[:, :D].copy())


def embed_grad(V, ids, dy, scale, dtype, grad0=None):
    """(grad, bound) in 64 bits."""
    D = dy.shape[1]
    ok = (ids >= 0) & (ids < V)
    g = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids[ok], dy[ok].double())
    mag = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids[ok], dy[ok].double().abs())
    n = torch.bincount(ids[ok], minlength=V).double()[:, None]
    scale = float(np.float32(scale))
    g, e = g * scale, (n + 1) * SUM * mag * abs(scale)
    if grad0 is not None:
        g = g + grad0.double()
        e = e + 2 ** -23 * (g.abs() + grad0.double().abs())
    u = U[dtype]
    return g, e * (1 + u) + u * g.abs()


def check(got, want, bound, what):
    got = got.detach().double().cpu()
    bad = (got - want).abs() > bound + 1e-37
    bad |= ~torch.isfinite(got) & torch.isfinite(want)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {got[i].item()!r}, "
                             f"want {want[i].item()!r} +- {bound[i].item():.3g}")
