"""Timed cases of the operators that produce a training step's gradients: the
embedding (lookup with scaling, gradient by tokens), the linear layer (bias,
activation and residual, with its backward pass) and activation checkpoints in
8 bits (stored, loaded, and read by the linear layer's backward pass).

`run` computes an operator in elementary torch operations in binary32, or,
with `own` set, through ring_all_reduce_amd.api.  `exact` gives the same
outputs from the definitions in binary64.

Shapes: T tokens, K features in, N features out, V vocabulary rows of D
features.  The sizes come from the Transformer whose gradient tensors the
bucketed workload reduces (d = 2048, h = 8192, V = 32000).
"""
import functools
import math

import torch

own = False

GROUP = 32       # values of a row that share one scale in an 8-bit checkpoint
E4M3_MAX = 448.0
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the tokens of one decoding step of a few requests: latency
        dict(name="lookup_decode", op="lookup", T=8, V=32000, D=2048, dtype="f32"),
        # the tokens of one rank's batch: 32 sequences of 2048
        dict(name="lookup_batch", op="lookup", T=65536, V=32000, D=2048, dtype="bf16"),
        # a short ragged batch on an odd table
        dict(name="embed_grad_ragged", op="embed_grad", T=4097, V=5003, D=509, dtype="f32"),
        # one rank's batch; the most frequent tokens take several percent of it
        dict(name="embed_grad_batch", op="embed_grad", T=65536, V=32000, D=2048, dtype="bf16"),
        # one token through the first feed-forward product: bound by reading the weights
        dict(name="forward_one_token", op="forward", T=1, K=2048, N=8192, dtype="bf16", act="gelu", residual=False),
        # the output projection with its residual for a few sequences, in binary32
        dict(name="forward_f32_residual", op="forward", T=515, K=2048, N=2048, dtype="f32", act="none", residual=True),
        # the first feed-forward product of one rank's micro-batch, with z kept for the backward pass
        dict(name="forward_ffn", op="forward", T=8192, K=2048, N=8192, dtype="bf16", act="gelu", residual=False),
        # odd sizes in binary32
        dict(name="backward_ragged", op="backward", T=333, K=501, N=259, dtype="f32", act="relu"),
        # the first feed-forward product's backward pass
        dict(name="backward_ffn", op="backward", T=8192, K=2048, N=8192, dtype="bf16", act="gelu"),
        # an odd batch stored in 8 bits and read back
        dict(name="ckpt_ragged", op="ckpt", T=1027, D=1001, dtype="f32", act="none"),
        # the feed-forward layer's z stored in 8 bits, and gelu(z) made again from it
        dict(name="ckpt_ffn", op="ckpt", T=8192, D=8192, dtype="bf16", act="gelu"),
        # the backward pass whose x and z are 8-bit checkpoints
        dict(name="backward_ckpt_ffn", op="backward_ckpt", T=8192, K=2048, N=8192, dtype="bf16", act="gelu"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; half of them whole eights."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 16 and rng.random() < 0.5:
        n -= n % 8
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["lookup", "embed_grad", "forward", "forward", "backward", "backward", "ckpt", "backward_ckpt"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("lookup", "embed_grad"):
        return dict(op=op, T=_size(rng, 1, 32768), V=_size(rng, 100, 32000), D=_size(rng, 64, 2048), dtype=dtype)
    act = rng.choice(["none", "relu", "gelu"])
    if op == "ckpt":
        return dict(op=op, T=_size(rng, 1, 8192), D=_size(rng, 64, 8192), dtype=dtype, act=act)
    K, N = _size(rng, 64, 4096), _size(rng, 64, 4096)
    # binary32 products run at a sixteenth of the bfloat16 rate
    T = _size(rng, 1, 8192 if dtype == "bf16" else 2048)
    case = dict(op=op, T=T, K=K, N=N, dtype=dtype, act=act)
    if op == "forward":
        case["residual"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _exp2(e):
    """2^e for integer tensors e in -126..127, in binary32."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _groups(x):
    """x [T, D] in binary32, zero-padded to whole groups, as [T, G, GROUP]."""
    T, D = x.shape
    G = (D + GROUP - 1) // GROUP
    return torch.nn.functional.pad(x.float(), (0, G * GROUP - D)).view(T, G, GROUP)


def _quantise(x):
    """The 8-bit checkpoint of x: e4m3 codes [T, 32 G] and exponent bytes [T, G].
    The exponent is the smallest e with max|x| <= 448 * 2^e."""
    g = _groups(x)
    amax = g.abs().amax(-1)
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    e = e.clamp(-126, 120)
    codes = (g * _exp2(-e).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.view(x.shape[0], -1).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales, D):
    """What a checkpoint stands for, in binary32."""
    v = codes.view(torch.float8_e4m3fn).float().view(*scales.shape, GROUP)
    return (v * _exp2(scales.to(torch.int32) - 127).unsqueeze(-1)).view(codes.shape)[:, :D]


def prepare(case, seed):
    """What the program has in hand: activations of unit scale, weights of
    scale 1/sqrt(K), gradients of scale 1e-2, tokens of a 1/k distribution
    with some rows of padding (-1)."""
    dev = torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    s = dict(case)
    T = case["T"]
    if op in ("lookup", "embed_grad"):
        V, D = case["V"], case["D"]
        u = torch.rand(T, generator=gen, device=dev, dtype=torch.float64)
        rank = torch.exp(u * math.log(V)).long().clamp(1, V) - 1
        ids = torch.randperm(V, generator=gen, device=dev)[rank]
        ids[torch.rand(T, generator=gen, device=dev) < 0.01] = -1
        s["ids"] = ids
        s["scale"] = math.sqrt(D)
        if op == "lookup":
            s["table"] = normal(V, D, scale=D ** -0.5)
        else:
            s["dy"] = normal(T, D, scale=1e-2)
        return s
    if op == "ckpt":
        s["x"] = normal(T, case["D"])
        return s
    K, N = case["K"], case["N"]
    s["w"] = normal(K, N, scale=K ** -0.5)
    if op == "forward":
        s["x"] = normal(T, K)
        s["b"] = normal(N, scale=0.1)
        s["r"] = normal(T, N) if case["residual"] else None
        return s
    s["dy"] = normal(T, N, scale=1e-2)
    if op == "backward":
        s["x"], s["z"] = normal(T, K), normal(T, N)
    else:
        s["x"], s["xs"] = _quantise(normal(T, K))
        s["z"], s["zs"] = _quantise(normal(T, N))
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain(s):
    op, dt = s["op"], _DT[s["dtype"]]
    if op == "lookup":
        ok = (s["ids"] >= 0) & (s["ids"] < s["V"])
        rows = s["table"][torch.where(ok, s["ids"], 0)].float() * s["scale"]
        return torch.where(ok.unsqueeze(-1), rows, 0.0).to(dt)
    if op == "embed_grad":
        ok = (s["ids"] >= 0) & (s["ids"] < s["V"])
        grad = torch.zeros(s["V"] + 1, s["D"], device=s["dy"].device)
        grad.index_add_(0, torch.where(ok, s["ids"], s["V"]), s["dy"].float())
        return (grad[:s["V"]] * s["scale"]).to(dt)
    if op == "forward":
        z = s["x"].float() @ s["w"].float() + s["b"].float()
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return y.to(dt), z.to(dt)
    if op == "ckpt":
        return _act(_values(*_quantise(s["x"]), s["D"]), s["act"]).to(dt)
    if op == "backward_ckpt":
        x, z = _values(s["x"], s["xs"], s["K"]), _values(s["z"], s["zs"], s["N"])
    else:
        x, z = s["x"].float(), s["z"].float()
    dz = s["dy"].float() * _act_grad(z, s["act"])
    return (dz @ s["w"].float().T).to(dt), (x.T @ dz).to(dt), dz.sum(0).to(dt)


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _layer(K, N, dtype, act):
    """The layer's plan, made once as a program that keeps its layers would."""
    from ring_all_reduce_amd import api
    return api.rar_linear_plan(K, N, {"f32": api.F32, "bf16": api.BF16}[dtype],
                               {"none": api.ACT_NONE, "relu": api.ACT_RELU, "gelu": api.ACT_GELU}[act])


def _framework(s):
    from ring_all_reduce_amd import api
    op, T, dt = s["op"], s["T"], _DT[s["dtype"]]
    code = api.F32 if s["dtype"] == "f32" else api.BF16

    def new(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "lookup":
        out = new(T, s["D"])
        api.rar_embed_lookup(s["V"], s["D"], code, s["table"], T, s["ids"], out, s["scale"])
        return out
    if op == "embed_grad":
        grad = new(s["V"], s["D"])
        api.rar_embed_grad(s["V"], s["D"], code, T, s["ids"], s["dy"], grad, s["scale"])
        return grad
    if op == "ckpt":
        D = s["D"]
        pitch, groups = api.rar_ckpt_size(D)
        codes, scales = new(T, pitch, dtype=torch.uint8), new(T, groups, dtype=torch.uint8)
        out = new(T, D)
        api.rar_ckpt_store(T, D, code, s["x"], codes, scales)
        api.rar_ckpt_load(T, D, code, codes, scales, out,
                          act={"none": api.ACT_NONE, "relu": api.ACT_RELU, "gelu": api.ACT_GELU}[s["act"]])
        return out
    K, N = s["K"], s["N"]
    plan = _layer(K, N, s["dtype"], s["act"])
    if op == "forward":
        y, z = new(T, N), new(T, N)
        api.rar_linear_forward(plan, T, s["x"], s["w"], s["b"], s["r"], y, pre=z)
        return y, z
    dx, dw, db = new(T, K), new(K, N), new(N)
    api.rar_linear_backward(plan, T, s["dy"], s["x"], s["w"], s["z"], dx, dw, db,
                            x_scales=s.get("xs"), pre_scales=s.get("zs"))
    return dx, dw, db


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------

def work(case):
    T, es = case["T"], 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "lookup":
        # at most min(T, V) distinct rows are read
        rows = min(T, case["V"])
        return {"bytes": 8 * T + (rows + T) * case["D"] * es, "flops": T * case["D"]}
    if op == "embed_grad":
        return {"bytes": 8 * T + (T + case["V"]) * case["D"] * es, "flops": T * case["D"]}
    if op == "ckpt":
        n = T * case["D"]
        return {"bytes": 2 * n * es + 2 * (n + n // GROUP), "flops": 8 * n}
    K, N = case["K"], case["N"]
    if op == "forward":
        n_out = 2 + (1 if case["residual"] else 0)
        return {"bytes": es * (T * K + K * N + N + n_out * T * N), "flops": 2 * T * K * N}
    kept = (T * K + T * N) * (es if op == "backward" else 1 + 1 / GROUP)
    return {"bytes": es * (T * N + K * N + T * K + K * N + N) + kept, "flops": 4 * T * K * N}


def _round_e4m3(v):
    """binary64 values of magnitude <= 448 rounded to the nearest e4m3 value, ties to even."""
    _, ex = torch.frexp(v)                       # |v| in [2^(ex-1), 2^ex)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(ex - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_ckpt(x):
    """The values an 8-bit checkpoint of x stands for, in binary64."""
    T, D = x.shape
    out = torch.empty(T, D, dtype=torch.float64, device=x.device)
    for d in range(0, D, GROUP):
        v = x[:, d:d + GROUP].double()
        frac, ex = torch.frexp(v.abs().amax(1, keepdim=True))   # amax = frac * 2^ex, frac in [0.5, 1)
        # 448 = 0.875 * 2^9
        e = torch.clamp(ex - 9 + (frac > E4M3_MAX / 512).to(ex.dtype), -126, 120)
        one = torch.ones_like(frac)
        out[:, d:d + GROUP] = _round_e4m3(v * torch.ldexp(one, -e)) * torch.ldexp(one, e)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "lookup":
        out = torch.zeros(s["T"], s["D"], dtype=torch.float64, device=s["ids"].device)
        live = torch.nonzero(s["ids"] >= 0).squeeze(-1)
        out[live] = s["scale"] * s["table"].double()[s["ids"][live]]
        return out
    if op == "embed_grad":
        live = torch.nonzero(s["ids"] >= 0).squeeze(-1)
        ids, order = torch.sort(s["ids"][live], stable=True)
        sums = torch.cumsum(s["dy"][live[order]].double(), 0)
        last = torch.nonzero(torch.cat([ids[1:] != ids[:-1], ids.new_ones(min(1, ids.numel())).bool()])).squeeze(-1)
        out = torch.zeros(s["V"], s["D"], dtype=torch.float64, device=ids.device)
        if last.numel():
            ends = sums[last]
            out[ids[last]] = s["scale"] * torch.cat([ends[:1], ends[1:] - ends[:-1]])
        return out
    root = math.sqrt(0.5)

    def phi(v):  # the normal distribution function
        return 0.5 * torch.special.erfc(-v * root)

    def f(v):
        return {"none": lambda: v, "relu": lambda: torch.maximum(v, torch.zeros_like(v)), "gelu": lambda: v * phi(v)}[s["act"]]()

    def df(v):
        return {"none": lambda: torch.ones_like(v), "relu": lambda: torch.heaviside(v, torch.zeros_like(v)),
                "gelu": lambda: phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)}[s["act"]]()

    if op == "ckpt":
        return f(_exact_ckpt(s["x"]))
    w = s["w"].double()
    if op == "forward":
        z = torch.addmm(s["b"].double(), s["x"].double(), w)
        y = f(z)
        return (y if s["r"] is None else y + s["r"].double()), z
    if op == "backward_ckpt":
        def value(codes, scales, n):
            c = codes.to(torch.int64)
            ex, m = (c >> 3) & 15, (c & 7).double()
            mag = torch.where(ex == 0, m * 2.0 ** -9, torch.ldexp(1 + m / 8, ex - 7))
            v = torch.where(c >= 128, -mag, mag)
            sc = torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.to(torch.int64) - 127)
            return (v * sc.repeat_interleave(GROUP, dim=1))[:, :n]
        x, z = value(s["x"], s["xs"], s["K"]), value(s["z"], s["zs"], s["N"])
    else:
        x, z = s["x"].double(), s["z"].double()
    dz = s["dy"].double() * df(z)
    return dz @ w.t(), x.t() @ dz, dz.sum(dim=0)
