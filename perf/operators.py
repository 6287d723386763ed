"""Operators for training and serving a bf16 mixture-of-experts layer, in their plain form
and through this package, with the cases they are timed on.

Four operators with their gradients, by the ``kind`` of a case:

* ``grouped``: products of the rows of each expert with that expert's weights
  (``dir`` fwd, dx or dw; ``out`` bf16 or fp32);
* ``linear``: one dense layer with bias, activation and residual, and ``linear_dz``: the
  gradient through its activation, with the bias's (its products' gradients are ``grouped``
  with one group);
* ``swiglu``: silu(g) * u of rows [g | u] (``dir`` fwd or bwd);
* ``combine``: expert rows summed back to their tokens by gate (``dir`` fwd or bwd), and
  ``permute``: tokens copied to their expert rows (without gates, combine is its gradient).
"""
import math

import torch

own = False

BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "fp32": FP32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one decode step of a 16-expert layer with 16 tokens, both up-projections side by side:
        # a token or two for each expert, so the time goes into reading weights
        dict(name="grouped_fwd_decode", kind="grouped", dir="fwd", P=16, E=16, N=16384, K=5120, skew=0.0, out="bf16"),
        # the same layer over a prompt or a training batch of 8192 tokens, each direction
        dict(name="grouped_fwd_batch", kind="grouped", dir="fwd", P=8192, E=16, N=16384, K=5120, skew=0.5, out="bf16"),
        dict(name="grouped_dx_batch", kind="grouped", dir="dx", P=8192, E=16, N=16384, K=5120, skew=0.5, out="bf16"),
        dict(name="grouped_dw_batch", kind="grouped", dir="dw", P=8192, E=16, N=5120, K=8192, skew=0.5, out="bf16"),
        # many small experts of odd widths, about twenty rows each, some with none; gradients kept in 32 bits
        dict(name="grouped_dw_ragged", kind="grouped", dir="dw", P=2571, E=128, N=1000, K=712, skew=1.0, out="fp32"),
        # one token through the shared expert's gate projection: the call where latency counts
        dict(name="linear_token", kind="linear", T=1, N=8192, K=5120, act="silu", bias=True, residual=False),
        # the shared expert's down projection over a batch, with the layer's residual added
        dict(name="linear_batch", kind="linear", T=8192, N=5120, K=8192, act="none", bias=False, residual=True),
        # through an activation in a training step, with the bias's gradient
        dict(name="linear_dz_batch", kind="linear_dz", T=8192, N=8192, act="gelu"),
        # a decode step's rows, and a training batch's gradient
        dict(name="swiglu_decode", kind="swiglu", dir="fwd", rows=16, h=8192),
        dict(name="swiglu_bwd_batch", kind="swiglu", dir="bwd", rows=8192, h=8192),
        # eight experts for each token: the widest routing; and its gradient at an odd size
        dict(name="combine_wide", kind="combine", dir="fwd", T=8192, k=8, d=5120, gates=True, residual=True, o="bf16"),
        dict(name="combine_bwd_odd", kind="combine", dir="bwd", T=1511, k=3, d=1416, gates=True, residual=False, o="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["grouped", "grouped", "grouped", "linear", "linear_dz", "swiglu", "permute", "combine"])
    if kind == "grouped":
        while True:
            c = dict(kind=kind, dir=rng.choice(["fwd", "dx", "dw"]), P=_log(rng, 1, 16384),
                     E=rng.choice([1, 2, 4, 8, 16, 16, 32, 64, 128]), N=_log(rng, 64, 16384, 8), K=_log(rng, 64, 8192, 8),
                     skew=rng.choice([0.0, 0.5, 1.0]), out=rng.choice(["bf16", "bf16", "fp32"]))
            if c["P"] * c["N"] * c["K"] <= 8192 * 5120 * 8192 and c["E"] * c["N"] * c["K"] <= 8 * 16384 * 5120:
                return c
    if kind == "linear":
        while True:
            c = dict(kind=kind, T=_log(rng, 1, 16384), N=_log(rng, 64, 16384, 8), K=_log(rng, 64, 8192, 8),
                     act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5)
            if c["T"] * c["N"] * c["K"] <= 8192 * 5120 * 8192:
                return c
    if kind == "linear_dz":
        return dict(kind=kind, T=_log(rng, 1, 8192), N=_log(rng, 64, 8192, 8), act=rng.choice(ACTS[1:]))
    if kind == "swiglu":
        return dict(kind=kind, dir=rng.choice(["fwd", "bwd"]), rows=_log(rng, 1, 8192), h=_log(rng, 64, 8192, 8))
    k = rng.choice([1, 1, 2, 3, 4, 6, 8])
    T, d = _log(rng, 1, 8192), _log(rng, 64, 5120, 8)
    if kind == "permute":
        return dict(kind=kind, T=T, k=k, d=d)
    way = rng.choice(["fwd", "bwd"])
    return dict(kind=kind, dir=way, T=T, k=k, d=d, gates=way == "bwd" or rng.random() < 0.7,
                residual=way == "fwd" and rng.random() < 0.5, o=rng.choice(["bf16", "bf16", "fp32"]))


def _normal(gen, *shape, scale=1.0, dtype=BF16):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, scale, generator=gen)


def _routing(gen, T, k):
    """Stable dispatch order of k pairs for each of T tokens over random experts: perm and inv."""
    key = torch.rand(T * k, generator=gen, device="cuda")
    perm = torch.argsort(key)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device="cuda")
    return perm.to(torch.int32), inv.view(T, k).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    s = dict(case=case)
    kind = case["kind"]
    if kind == "grouped":
        P, E, N, K = case["P"], case["E"], case["N"], case["K"]
        # each row's expert, popular ones more often where the routing is skewed
        share = (torch.arange(E, dtype=FP32, device="cuda") + 1.0) ** -case["skew"]
        ids = torch.multinomial(share[torch.randperm(E, generator=gen, device="cuda")], P, True, generator=gen)
        counts = torch.bincount(ids, minlength=E)
        s["counts"] = counts.tolist()
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        if case["dir"] != "dx":
            s["x"] = _normal(gen, P, K)
        if case["dir"] != "fwd":
            s["dy"] = _normal(gen, P, N)
        if case["dir"] != "dw":
            s["w"] = _normal(gen, E, N, K, scale=0.02)
    elif kind == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"], s["w"] = _normal(gen, T, K), _normal(gen, N, K, scale=0.02)
        s["bias"] = _normal(gen, N, scale=0.5, dtype=FP32) if case["bias"] else None
        s["residual"] = _normal(gen, T, N) if case["residual"] else None
    elif kind == "linear_dz":
        s["dy"], s["z"] = _normal(gen, case["T"], case["N"]), _normal(gen, case["T"], case["N"], scale=1.5)
    elif kind == "swiglu":
        s["z"] = _normal(gen, case["rows"], 2 * case["h"], scale=1.5)
        if case["dir"] == "bwd":
            s["dy"] = _normal(gen, case["rows"], case["h"])
    else:
        T, k, d = case["T"], case["k"], case["d"]
        s["perm"], s["inv"] = _routing(gen, T, k)
        if kind == "permute":
            s["x"] = _normal(gen, T, d)
        else:
            s["o"] = _normal(gen, T * k, d, dtype=DTYPES[case["o"]])
            s["gates"] = torch.rand(T, k, generator=gen, device="cuda") if case["gates"] else None
            s["residual"] = _normal(gen, T, d) if case["residual"] else None
            if case["dir"] == "bwd":
                s["dy"] = _normal(gen, T, d)
    return s


# ------------------------------------------------------------- plain forms

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "silu":
        g = 1.0 / (1.0 + torch.exp(-z))
        return g * (1.0 + z * (1.0 - g))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_grouped(s, way, out):
    counts = s["counts"]
    a = s["x"] if way == "fwd" else s["dy"]
    if way == "dw":
        dw = torch.zeros(len(counts), s["dy"].shape[1], s["x"].shape[1], dtype=out, device=a.device)
        rows = zip(torch.split(s["dy"], counts), torch.split(s["x"], counts))
        # the groups are ragged: one product for each that has rows does less than padding them to one length
        for e, (dy, x) in enumerate(rows):
            if counts[e]:
                dw[e] = torch.mm(dy.float().t(), x.float())
        return dw
    y = torch.empty(a.shape[0], s["w"].shape[1 if way == "fwd" else 2], dtype=out, device=a.device)
    for e, (rows, to) in enumerate(zip(torch.split(a, counts), torch.split(y, counts))):
        if counts[e]:
            w = s["w"][e].float()
            to.copy_(torch.mm(rows.float(), w.t() if way == "fwd" else w))
    return y


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "grouped":
        return _plain_grouped(s, c["dir"], DTYPES[c["out"]])
    if kind == "linear":
        z = torch.mm(s["x"].float(), s["w"].float().t())
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(BF16)
    if kind == "linear_dz":
        dz = s["dy"].float() * _act_grad(s["z"].float(), c["act"])
        return dz.to(BF16), dz.sum(0)
    if kind == "swiglu":
        g, u = s["z"].float().chunk(2, dim=1)
        sig = 1.0 / (1.0 + torch.exp(-g))
        if c["dir"] == "fwd":
            return (g * sig * u).to(BF16)
        dy = s["dy"].float()
        return torch.cat([dy * u * sig * (1.0 + g * (1.0 - sig)), dy * g * sig], dim=1).to(BF16)
    if kind == "permute":
        return s["x"][torch.div(s["perm"].long(), c["k"], rounding_mode="floor")]
    if c["dir"] == "fwd":
        o = s["o"][s["inv"].long()].float()
        y = (o * s["gates"].unsqueeze(2) if s["gates"] is not None else o).sum(1)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(BF16)
    dy = s["dy"].float()
    pairs = s["perm"].long()
    token = torch.div(pairs, c["k"], rounding_mode="floor")
    do = (dy[token] * s["gates"].reshape(-1)[pairs].unsqueeze(1)).to(BF16)
    dg = (dy.unsqueeze(1) * s["o"][s["inv"].long()].float()).sum(2)
    return do, dg


def _own(s):
    import moe_ffn_int4_amd as moe

    c = s["case"]
    kind = c["kind"]
    if kind == "grouped":
        out = DTYPES[c["out"]]
        if c["dir"] == "fwd":
            return moe.grouped_matmul(s["x"], s["w"], s["offsets"], out_dtype=out)
        if c["dir"] == "dx":
            return moe.grouped_matmul_dx(s["dy"], s["w"], s["offsets"], out_dtype=out)
        return moe.grouped_matmul_dw(s["dy"], s["x"], s["offsets"], out_dtype=out)
    if kind == "linear":
        return moe.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"])
    if kind == "linear_dz":
        return moe.linear_dz(s["dy"], s["z"], c["act"])
    if kind == "swiglu":
        return moe.swiglu(s["z"]) if c["dir"] == "fwd" else moe.swiglu_backward(s["dy"], s["z"])
    if kind == "permute":
        return moe.permute_rows(s["x"], s["perm"], c["k"])
    if c["dir"] == "fwd":
        return moe.combine(s["o"], s["inv"], gates=s["gates"], residual=s["residual"])
    return moe.combine_backward(s["dy"], s["o"], s["inv"], s["gates"])


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once. A group
    without rows needs no weights read; how many have some is what a uniform draw expects."""
    kind = case["kind"]
    if kind == "grouped":
        P, E, N, K = case["P"], case["E"], case["N"], case["K"]
        size = 2 if case["out"] == "bf16" else 4
        touched = E * (1.0 - (1.0 - 1.0 / E) ** P)
        if case["dir"] == "dw":
            moved = 2 * P * (N + K) + size * E * N * K
        else:
            k, n = (K, N) if case["dir"] == "fwd" else (N, K)
            moved = 2 * P * k + size * P * n + 2 * touched * N * K
        return {"bytes": moved, "flops": 2.0 * P * N * K}
    if kind == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        moved = 2 * T * K + 2 * N * K + 2 * T * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        return {"bytes": moved, "flops": 2.0 * T * N * K}
    if kind == "linear_dz":
        n = case["T"] * case["N"]
        return {"bytes": 6 * n + 4 * case["N"], "flops": 12.0 * n}
    if kind == "swiglu":
        n = case["rows"] * case["h"]
        return {"bytes": (6 if case["dir"] == "fwd" else 10) * n, "flops": (6.0 if case["dir"] == "fwd" else 14.0) * n}
    T, k, d = case["T"], case["k"], case["d"]
    if kind == "permute":
        return {"bytes": 2 * T * d + 2 * T * k * d + 4 * T * k, "flops": 0.0}
    size = 2 if case["o"] == "bf16" else 4
    index = 4 * T * k * (2 if case["gates"] else 1)
    if case["dir"] == "fwd":
        return {"bytes": size * T * k * d + 2 * T * d * (2 if case["residual"] else 1) + index, "flops": 2.0 * T * k * d}
    return {"bytes": (size + 2) * T * k * d + 2 * T * d + index + 4 * T * k, "flops": 3.0 * T * k * d}


# ------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    wide = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point() and n != "w"}
    if kind == "grouped":
        at = s["offsets"].tolist()
        parts = []
        for e in range(case["E"]):
            rows = slice(at[e], at[e + 1])
            if case["dir"] == "fwd":
                parts.append(wide["x"][rows].matmul(s["w"][e].double().t()))
            elif case["dir"] == "dx":
                parts.append(wide["dy"][rows].matmul(s["w"][e].double()))
            else:
                parts.append(wide["dy"][rows].t().matmul(wide["x"][rows]))
        return torch.stack(parts) if case["dir"] == "dw" else torch.cat(parts)
    if kind in ("linear", "linear_dz"):
        act = case["act"]
        z = wide["z"] if kind == "linear_dz" else wide["x"].matmul(s["w"].double().t()) + wide.get("bias", 0.0)
        gate = torch.sigmoid(z)
        cdf = torch.special.ndtr(z)
        inner = math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)  # gelu_tanh is z * sigmoid of it
        if kind == "linear":
            y = {"none": z, "relu": torch.where(z > 0, z, torch.zeros_like(z)), "silu": z * gate, "gelu": z * cdf,
                 "gelu_tanh": z * torch.sigmoid(inner)}[act]
            return y + wide.get("residual", 0.0)
        soft = torch.sigmoid(inner)
        slope = {"none": torch.ones_like(z), "relu": (z > 0).double(), "silu": gate + z * gate * (1 - gate),
                 "gelu": cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                 "gelu_tanh": soft + z * soft * (1 - soft) * math.sqrt(8.0 / math.pi) * (1 + 0.134145 * z * z)}[act]
        dz = wide["dy"] * slope
        return dz, dz.sum(dim=0)
    if kind == "swiglu":
        h = case["h"]
        g, u = wide["z"][:, :h], wide["z"][:, h:]
        gate = torch.sigmoid(g)
        if case["dir"] == "fwd":
            return u * g * gate
        dz = torch.empty_like(wide["z"])
        dz[:, :h] = wide["dy"] * u * (gate + g * gate * (1 - gate))
        dz[:, h:] = wide["dy"] * g * gate
        return dz
    T, k, d = case["T"], case["k"], case["d"]
    if kind == "permute":
        return wide["x"].repeat_interleave(k, dim=0).index_select(0, s["perm"].long())
    to = s["perm"].long()
    if case["dir"] == "fwd":
        # scattered from the expert rows, where the plain form gathers by token
        y = wide["residual"] if case["residual"] else torch.zeros(T, d, dtype=torch.float64, device="cuda")
        rows = wide["o"] * wide["gates"].reshape(-1, 1)[to] if case["gates"] else wide["o"]
        return y.index_add_(0, to // k, rows)
    do, dg = torch.empty(T * k, d, dtype=torch.float64, device="cuda"), torch.empty(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        slot = s["inv"][:, j].long()
        do[slot] = wide["gates"][:, j:j + 1] * wide["dy"]
        dg[:, j] = (wide["dy"] * wide["o"].index_select(0, slot)).sum(dim=1)
    return do, dg
