"""More operators for training and serving a mixture-of-experts layer, in their plain form and
through this package, with the cases they are timed on.

Three operators, by the ``kind`` of a case:

* ``gated``: both up-projections of a gated feed-forward block with the activation and the product,
  y = act(x Wg^T) * (x Wu^T), for the rows of each expert or (``E`` 0) one dense layer; and
  ``gated_dz``: back from the down-projection's output to the two projections', which also gives y again;
* ``int4``: products with 4-bit weights that have one scale for each group of a row, dense
  (``E`` 0, with bias, activation and residual) or by expert;
* ``adamw``: a step over many tensors at once, its two moments in 32 or in 8 bits.
"""
import math

import torch

own = False

BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "fp32": FP32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
BLOCK = 128       # elements that share a scale of an 8-bit moment
TINY = 2.0 ** -100  # the least maximum of a block


def listed():
    return [
        # one token through a dense gated block: the call where latency counts, two matrices read once
        dict(name="gated_token", kind="gated", E=0, P=1, h=8192, d=5120, act="silu", bias=False, z=False, skew=0.0),
        # a decode step of a 16-expert layer with 16 tokens
        dict(name="gated_decode", kind="gated", E=16, P=16, h=8192, d=5120, act="silu", bias=False, z=False, skew=0.0),
        # a training batch of the same layer, the projections kept for the way back; and that way
        dict(name="gated_batch", kind="gated", E=16, P=8192, h=8192, d=5120, act="silu", bias=False, z=True, skew=0.5),
        dict(name="gated_dz_batch", kind="gated_dz", E=16, P=8192, h=8192, d=5120, act="silu", skew=0.5),
        # many small experts of odd widths, some without rows, gelu in place of silu
        dict(name="gated_dz_ragged", kind="gated_dz", E=128, P=2571, h=1000, d=712, act="gelu", skew=1.0),
        # one token through a dense layer held in 4 bits
        dict(name="int4_token", kind="int4", E=0, T=1, N=8192, K=5120, group=128, act="silu", bias=True, residual=False, out="bf16", skew=0.0),
        # a decode step over 16 experts in 4 bits, both up-projections side by side
        dict(name="int4_decode", kind="int4", E=16, T=16, N=16384, K=5120, group=128, act="none", bias=False, residual=False, out="bf16", skew=0.0),
        # a speculative or small batch at the smallest group, into a residual
        dict(name="int4_odd", kind="int4", E=0, T=37, N=5120, K=8192, group=32, act="none", bias=False, residual=True, out="bf16", skew=0.0),
        # a prompt through the same layer
        dict(name="int4_prompt", kind="int4", E=0, T=4096, N=5120, K=8192, group=128, act="none", bias=False, residual=True, out="bf16", skew=0.0),
        # biases and a router: small tensors in 32 bits, where the launch is what it costs
        dict(name="adamw_small", kind="adamw", tensors=12, size=81920, param="fp32", grad="fp32", master=False, bits=32, step=100, clip=False),
        # bf16 weights of a few experts with 32-bit copies, moments in 32 bits, clipped gradients
        dict(name="adamw_layer", kind="adamw", tensors=6, size=41943040, param="bf16", grad="bf16", master=True, bits=32, step=1000, clip=True),
        # the same with moments in 8 bits and many tensors
        dict(name="adamw_layer8", kind="adamw", tensors=40, size=8388608, param="bf16", grad="fp32", master=True, bits=8, step=1000, clip=False),
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["gated", "gated", "gated_dz", "int4", "int4", "adamw"])
    if kind in ("gated", "gated_dz"):
        while True:
            c = dict(kind=kind, E=rng.choice([0, 0, 1, 2, 4, 8, 16, 16, 32, 64, 128]), P=_log(rng, 1, 16384),
                     h=_log(rng, 64, 8192, 8), d=_log(rng, 64, 8192, 8), act=rng.choice(ACTS), skew=rng.choice([0.0, 0.5, 1.0]))
            c["skew"] = c["skew"] if c["E"] else 0.0
            if kind == "gated":
                c.update(bias=c["E"] == 0 and rng.random() < 0.4, z=rng.random() < 0.5)
            if c["P"] * c["h"] * c["d"] <= 8192 * 8192 * 5120 and max(c["E"], 1) * c["h"] * c["d"] <= 16 * 8192 * 5120:
                return c
    if kind == "int4":
        while True:
            c = dict(kind=kind, E=rng.choice([0, 0, 0, 1, 4, 16, 32, 128]), T=_log(rng, 1, 8192), N=_log(rng, 64, 16384, 16),
                     K=_log(rng, 128, 8192, 128), group=rng.choice([128, 128, 64, 32]), out=rng.choice(["bf16", "bf16", "fp32"]),
                     skew=rng.choice([0.0, 0.5, 1.0]))
            dense = c["E"] == 0
            c.update(skew=0.0 if dense else c["skew"], act=rng.choice(ACTS) if dense else "none", bias=dense and rng.random() < 0.5, residual=dense and rng.random() < 0.5)
            if c["T"] * c["N"] * c["K"] <= 4096 * 5120 * 8192 and max(c["E"], 1) * c["N"] * c["K"] <= 16 * 16384 * 5120:
                return c
    while True:
        c = dict(kind=kind, tensors=_log(rng, 1, 56), size=_log(rng, 1, 40000000), param=rng.choice(["bf16", "fp32"]),
                 grad=rng.choice(["bf16", "fp32"]), bits=rng.choice([8, 32]), step=_log(rng, 1, 100000), clip=rng.random() < 0.5)
        c["master"] = c["param"] == "bf16" and rng.random() < 0.7
        if sum(_sizes(c)) <= 120000000:
            return c


def _normal(gen, *shape, scale=1.0, dtype=BF16):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, scale, generator=gen)


def _groups(gen, s, E, P, skew):
    """Each row's expert, popular ones more often where the routing is skewed."""
    share = (torch.arange(E, dtype=FP32, device="cuda") + 1.0) ** -skew
    ids = torch.multinomial(share[torch.randperm(E, generator=gen, device="cuda")], P, True, generator=gen)
    counts = torch.bincount(ids, minlength=E)
    s["counts"] = counts.tolist()
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _tile(q, scales, group):
    """Codes [.., N, K/2] and scales of row-major 4-bit weights in tiles of 16 rows and 128 columns:
    code bytes by step of 32 columns, row, byte; scales by row, group."""
    N, half = q.shape[-2:]
    lead = q.shape[:-2]
    n, per = len(lead), 128 // group
    t = q.reshape(*lead, N // 16, 16, half // 64, 4, 16)
    t = t.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).contiguous().reshape(q.shape)
    u = scales.reshape(*lead, N // 16, 16, half // 64, per)
    return t, u.permute(*range(n), n, n + 2, n + 1, n + 3).contiguous().reshape(scales.shape)


def _sizes(c):
    """Elements of each tensor: large ones, some of a fraction of that, and small odd ones."""
    share = (1.0, 0.4, 0.002, 0.0003)
    return [max(1, int(c["size"] * share[i % 4]) + (7 * i) % 11 - 5) if i else c["size"] for i in range(c["tensors"])]


def _starts(sizes):
    """Where each tensor's elements begin in the flat moments: on whole blocks; and the end."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + (n + BLOCK - 1) // BLOCK * BLOCK)
    return at


def _prepare_adamw(gen, c, s):
    sizes = _sizes(c)
    starts = _starts(sizes)
    total = starts[-1]
    s["lr"], s["betas"], s["eps"], s["decay"] = 3e-4, (0.9, 0.95), 1e-8, 0.1
    s["sizes"], s["starts"] = sizes, starts
    wide = _normal(gen, total, scale=0.02, dtype=FP32)
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for o, n in zip(starts, sizes):
        inside[o:o + n] = True
    wide *= inside
    s["params"] = [wide[o:o + n].to(DTYPES[c["param"]]) for o, n in zip(starts, sizes)]
    s["master"] = wide if c["master"] else None
    s["grads"] = [_normal(gen, n, scale=1e-3, dtype=DTYPES[c["grad"]]) for n in sizes]
    s["clip"] = torch.rand(1, generator=gen, device="cuda") if c["clip"] else None
    m = _normal(gen, total, scale=3e-4, dtype=FP32) * inside
    r = (_normal(gen, total, scale=1e-3, dtype=FP32).abs() + 1e-5) * inside  # the second moment's root
    if c["bits"] == 8:
        for name, t in (("m", m), ("v", r)):
            most = t.abs().reshape(-1, BLOCK).amax(1).clamp(min=TINY)
            s[name + "_scale"] = most / 448.0
            codes = (t.reshape(-1, BLOCK) * (448.0 / most).unsqueeze(1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            s[name] = codes.view(torch.uint8).reshape(-1)
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, r * r, None, None
    if own:
        import moe_ffn_int4_amd as moe

        s["state"] = moe.AdamWState(s["params"], s["m"], s["v"], s["m_scale"], s["v_scale"], s["master"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    s = dict(case=case)
    kind = case["kind"]
    if kind == "adamw":
        _prepare_adamw(gen, case, s)
        return s
    E = case["E"]
    lead = (E,) if E else ()
    if E:
        _groups(gen, s, E, case["T" if kind == "int4" else "P"], case["skew"])
    if kind == "int4":
        T, N, K, group = case["T"], case["N"], case["K"], case["group"]
        s["x"] = _normal(gen, T, K)
        s["q"] = torch.randint(0, 256, lead + (N, K // 2), dtype=torch.uint8, generator=gen, device="cuda")
        s["scales"] = torch.rand(lead + (N, K // group), generator=gen, device="cuda") * 0.006 + 0.002
        s["tiled"] = _tile(s["q"], s["scales"], group)
        s["bias"] = _normal(gen, N, scale=0.5, dtype=FP32) if case["bias"] else None
        s["residual"] = _normal(gen, T, N) if case["residual"] else None
        return s
    P, h, d = case["P"], case["h"], case["d"]
    if kind == "gated":
        s["x"] = _normal(gen, P, d)
        s["w"] = _normal(gen, *lead, 2 * h, d, scale=0.02)
        s["bias"] = _normal(gen, 2 * h, scale=0.5, dtype=FP32) if case["bias"] else None
    else:
        s["dy"] = _normal(gen, P, d)
        s["w"] = _normal(gen, *lead, d, h, scale=0.02)
        s["z"] = _normal(gen, P, 2 * h, scale=1.5)
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


def _each_group(s, rows, P):
    """(expert or None, its rows' slice) of the groups that have rows."""
    if "counts" not in s:
        return [(None, slice(0, P))]
    parts, at = [], 0
    for e, n in enumerate(s["counts"]):
        if n:
            parts.append((e, slice(at, at + n)))
        at += n
    return parts


def _plain_gated(s):
    c = s["case"]
    P, h, act = c["P"], c["h"], c["act"]
    if c["kind"] == "gated":
        y = torch.empty(P, h, dtype=BF16, device="cuda")
        z = torch.empty(P, 2 * h, dtype=BF16, device="cuda") if c["z"] else None
        for e, rows in _each_group(s, s["x"], P):
            w = s["w"] if e is None else s["w"][e]
            wide = torch.mm(s["x"][rows].float(), w.float().t())
            if s["bias"] is not None:
                wide = wide + s["bias"]
            if z is not None:
                z[rows] = wide.to(BF16)
            y[rows] = (_act(wide[:, :h], act) * wide[:, h:]).to(BF16)
        return (y, z) if c["z"] else y
    dh = torch.empty(P, h, dtype=FP32, device="cuda")
    for e, rows in _each_group(s, s["dy"], P):
        dh[rows] = torch.mm(s["dy"][rows].float(), (s["w"] if e is None else s["w"][e]).float())
    g, u = s["z"].float().chunk(2, dim=1)
    a = _act(g, act)
    dz = torch.cat([dh * u * _act_grad(g, act), dh * a], dim=1).to(BF16)
    return dz, (a * u).to(BF16)


def _codes(q):
    """The signed 4-bit numbers of each byte, low half first."""
    low, high = q & 15, q >> 4
    n = torch.stack([low, high], dim=-1).flatten(-2).to(torch.int8)
    return torch.where(n > 7, n - 16, n)


def _plain_int4(s):
    c = s["case"]
    T, N, K = c["T"], c["N"], c["K"]
    y = torch.empty(T, N, dtype=FP32, device="cuda")
    for e, rows in _each_group(s, s["x"], T):
        q, scales = (s["q"], s["scales"]) if e is None else (s["q"][e], s["scales"][e])
        w = (_codes(q).float().reshape(N, -1, c["group"]) * scales.unsqueeze(2)).reshape(N, K)
        y[rows] = torch.mm(s["x"][rows].float(), w.t())
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


def _results_adamw(s):
    # 8-bit moments as the numbers their codes are, and the scales beside them
    if s["case"]["bits"] == 8:
        moments = [s["m"].view(torch.float8_e4m3fn), s["m_scale"], s["v"].view(torch.float8_e4m3fn), s["v_scale"]]
    else:
        moments = [s["m"], s["v"]]
    return s["params"] + moments + ([s["master"]] if s["master"] is not None else [])


def _plain_adamw(s):
    c = s["case"]
    (b1, b2), t, lr = s["betas"], c["step"], s["lr"]
    fix1, fix2 = 1.0 - b1 ** t, 1.0 - b2 ** t
    for i, (n, o) in enumerate(zip(s["sizes"], s["starts"])):
        end = s["starts"][i + 1]
        g = s["grads"][i].float()
        if s["clip"] is not None:
            g = g * s["clip"]
        if c["bits"] == 8:
            blocks = slice(o // BLOCK, end // BLOCK)
            m = (s["m"][o:end].view(torch.float8_e4m3fn).float().reshape(-1, BLOCK) * s["m_scale"][blocks].unsqueeze(1)).reshape(-1)[:n]
            r = (s["v"][o:end].view(torch.float8_e4m3fn).float().reshape(-1, BLOCK) * s["v_scale"][blocks].unsqueeze(1)).reshape(-1)[:n]
            v = r * r
        else:
            m, v = s["m"][o:o + n], s["v"][o:o + n]
        # each product and sum rounded by itself: an 8-bit code depends on the last bit next to a border
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + (g * g) * (1.0 - b2)
        root = torch.sqrt(v)
        p = s["master"][o:o + n] if s["master"] is not None else s["params"][i].float()
        p = p * (1.0 - lr * s["decay"]) - (lr / fix1) * (m / (root / math.sqrt(fix2) + s["eps"]))
        if s["master"] is not None:
            s["master"][o:o + n] = p
        s["params"][i].copy_(p)
        if c["bits"] == 8:
            for name, x in (("m", m), ("v", root)):
                x = torch.nn.functional.pad(x, (0, end - o - n)).reshape(-1, BLOCK)
                most = x.abs().amax(1).clamp(min=TINY)
                s[name + "_scale"][blocks] = most / 448.0
                codes = (x * (448.0 / most).unsqueeze(1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
                s[name][o:end] = codes.view(torch.uint8).reshape(-1)
        else:
            s["m"][o:o + n] = m
            s["v"][o:o + n] = v
    return _results_adamw(s)


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "int4":
        return _plain_int4(s)
    return _plain_adamw(s) if kind == "adamw" else _plain_gated(s)


def _own(s):
    import moe_ffn_int4_amd as moe

    c = s["case"]
    kind = c["kind"]
    if kind == "gated":
        z = torch.empty(c["P"], 2 * c["h"], dtype=BF16, device="cuda") if c["z"] else None
        if c["E"]:
            y = moe.grouped_gated(s["x"], s["w"], s["offsets"], c["act"], z=z)
        else:
            y = moe.gated_linear(s["x"], s["w"], s["bias"], c["act"], z=z)
        return (y, z) if c["z"] else y
    if kind == "gated_dz":
        y = torch.empty(c["P"], c["h"], dtype=BF16, device="cuda")
        if c["E"]:
            return moe.grouped_gated_dz(s["dy"], s["w"], s["z"], s["offsets"], c["act"], y=y), y
        return moe.gated_linear_dz(s["dy"], s["w"], s["z"], c["act"], y=y), y
    if kind == "int4":
        q, scales = s["tiled"]
        if c["E"]:
            return moe.grouped_matmul_int4(s["x"], q, scales, s["offsets"], out_dtype=DTYPES[c["out"]])
        return moe.linear_int4(s["x"], q, scales, bias=s["bias"], act=c["act"], residual=s["residual"], out_dtype=DTYPES[c["out"]])
    moe.adamw(s["state"], s["grads"], c["step"], lr=s["lr"], betas=s["betas"], eps=s["eps"], weight_decay=s["decay"], grad_scale=s["clip"])
    return _results_adamw(s)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once. An expert
    without rows needs no weights read; how many have some is what a uniform draw expects."""
    kind = case["kind"]
    if kind == "adamw":
        n = float(sum(_sizes(case)))
        p, g = (2 if case["param"] == "bf16" else 4), (2 if case["grad"] == "bf16" else 4)
        moments = 4 + 16.0 / BLOCK if case["bits"] == 8 else 16
        return {"bytes": n * (g + moments + (8 + p if case["master"] else 2 * p)), "flops": 15.0 * n}
    E, rows = case["E"], case["T" if kind == "int4" else "P"]
    touched = E * (1.0 - (1.0 - 1.0 / E) ** rows) if E else 1.0
    if kind == "int4":
        N, K = case["N"], case["K"]
        size = 2 if case["out"] == "bf16" else 4
        weights = touched * N * K * (0.5 + 4.0 / case["group"])
        moved = 2 * rows * K + weights + rows * N * (size + (2 if case["residual"] else 0)) + (4 * N if case["bias"] else 0)
        return {"bytes": moved, "flops": 2.0 * rows * N * K}
    h, d = case["h"], case["d"]
    if kind == "gated":
        moved = 2 * rows * d + 4 * touched * h * d + 2 * rows * h * (3 if case["z"] else 1) + (8 * h if case["bias"] else 0)
        return {"bytes": moved, "flops": 4.0 * rows * h * d}
    return {"bytes": 2 * rows * d + 2 * touched * h * d + 10 * rows * h, "flops": 2.0 * rows * h * d}


# ------------------------------------------------------- definitions in 64 bits

def _act_exact(z, act):
    """(act(z), act'(z)) in 64 bits."""
    gate = torch.sigmoid(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).double()
    if act == "silu":
        return z * gate, gate + z * gate * (1 - gate)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        soft = torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
        return z * soft, soft + z * soft * (1 - soft) * math.sqrt(8.0 / math.pi) * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)


def _weights_exact(s, e):
    c = s["case"]
    q, scales = (s["q"], s["scales"]) if e is None else (s["q"][e], s["scales"][e])
    w = torch.empty(c["N"], c["K"], dtype=torch.float64, device="cuda")
    w[:, 0::2] = (q & 15).double()
    w[:, 1::2] = (q >> 4).double()
    w -= 16.0 * (w >= 8)
    return w.mul_(scales.double().repeat_interleave(c["group"], dim=1))


def _exact_adamw(s):
    c = s["case"]
    b1, b2 = s["betas"]
    t = c["step"]
    params, flat = [], {"m": [], "v": [], "m_scale": [], "v_scale": [], "master": []}
    for i, n in enumerate(s["sizes"]):
        o, end = s["starts"][i], s["starts"][i + 1]
        g = torch.zeros(end - o, dtype=torch.float64, device="cuda")
        g[:n] = s["grads"][i].double()
        if s["clip"] is not None:
            g *= s["clip"].double()
        old = {}
        for name in ("m", "v"):
            old[name] = s[name][o:end]
            if c["bits"] == 8:
                per = s[name + "_scale"][o // BLOCK:end // BLOCK].double().repeat_interleave(BLOCK)
                old[name] = old[name].view(torch.float8_e4m3fn).double() * per
            old[name] = old[name].double()
        m = b1 * old["m"] + (1 - b1) * g
        v = b2 * (old["v"] ** 2 if c["bits"] == 8 else old["v"]) + (1 - b2) * g ** 2
        p = torch.zeros_like(g)
        p[:n] = s["master"][o:o + n].double() if s["master"] is not None else s["params"][i].double()
        step = m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + s["eps"])
        p = p - s["lr"] * s["decay"] * p - s["lr"] * step
        params.append(p[:n])
        flat["master"].append(torch.cat([p[:n], torch.zeros(end - o - n, dtype=torch.float64, device="cuda")]))
        for name, x in (("m", m), ("v", v)):
            if c["bits"] == 8:
                x = x if name == "m" else torch.sqrt(x)
                most = torch.clamp(x.reshape(-1, BLOCK).abs().max(dim=1).values, min=TINY)
                flat[name + "_scale"].append(most / 448)
                x = (x.reshape(-1, BLOCK) / most.unsqueeze(1) * 448).float().to(torch.float8_e4m3fn).double().reshape(-1)
            flat[name].append(x)
    names = ["m", "m_scale", "v", "v_scale"] if c["bits"] == 8 else ["m", "v"]
    return params + [torch.cat(flat[n]) for n in names + (["master"] if s["master"] is not None else [])]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "adamw":
        return _exact_adamw(s)
    E = case["E"]
    at = s["offsets"].tolist() if E else [0, case["T" if kind == "int4" else "P"]]
    out = []
    for e in range(max(E, 1)):
        rows = slice(at[e], at[e + 1])
        if kind == "int4":
            out.append(s["x"][rows].double().matmul(_weights_exact(s, e if E else None).t()) if at[e + 1] > at[e]
                       else torch.zeros(0, case["N"], dtype=torch.float64, device="cuda"))
        else:
            w = (s["w"][e] if E else s["w"]).double()
            out.append((s["x"][rows].double().matmul(w.t()) if kind == "gated" else s["dy"][rows].double().matmul(w)))
    y = torch.cat(out)
    if kind == "int4":
        if case["bias"]:
            y = y + s["bias"].double()
        y = _act_exact(y, case["act"])[0]
        return y + s["residual"].double() if case["residual"] else y
    h = case["h"]
    if kind == "gated":
        if case["bias"]:
            y = y + s["bias"].double()
        v = _act_exact(y[:, :h], case["act"])[0] * y[:, h:]
        return (v, y) if case["z"] else v
    z = s["z"].double()
    a, slope = _act_exact(z[:, :h], case["act"])
    dz = torch.empty_like(z)
    dz[:, :h] = y * z[:, h:] * slope
    dz[:, h:] = y * a
    return dz, a * z[:, h:]
