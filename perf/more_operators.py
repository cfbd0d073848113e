"""The measured cases of the low-rank adapters and the 8-bit activation checkpoints, with their plain forms.

Five operators of a layer whose projections are frozen and carry low-rank adapters, many of them at once:

* ``group``: sorts a batch's rows by adapter (rows without one last), once for all its projections;
* ``checkpoint``: an activation kept in 8 bits (E4M3 codes, one E8M0 scale per 32 elements) and restored;
* ``forward``: ``t = scale[g] x down[g]^T`` and ``out = base + t up[g]``, beside the projection's result ``base``;
* ``grad_input``: ``dt = scale[g] dy up[g]^T`` and ``dx = base + dt down[g]``;
* ``grad_weight``: ``dw[g] = t_g^T z_g``, z the layer's input (bf16, or its 8-bit checkpoint) or its output's gradient.

Plain forms are elementary torch operations in 32 bits. ``own`` selects the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # serving: a decode batch of 64 requests, each with one of 256 adapters, some with none
        {"name": "group 64 rows of 256", "op": "group", "m": 64, "g": 256, "skew": 0.5, "none": 0.1},
        # a fine-tuning batch of many tenants
        {"name": "group 16384 rows of 64", "op": "group", "m": 16384, "g": 64, "skew": 1.1, "none": 0.0},
        # an expert layer's input kept for the backward pass: 8192 tokens, two copies each
        {"name": "checkpoint 16384x4096", "op": "checkpoint", "m": 16384, "k": 4096, "dtype": "bf16"},
        # a small odd batch in fp32
        {"name": "checkpoint 61x7168 f32", "op": "checkpoint", "m": 61, "k": 7168, "dtype": "f32"},
        # serving, one token: latency
        {"name": "forward 1 row rank 16", "op": "forward", "m": 1, "k": 4096, "n": 4096, "g": 64, "rank": 16,
         "skew": 0.0, "none": 0.0, "order": True},
        # serving, a decode batch of 64 requests over 256 adapters of the up projection
        {"name": "forward 64 rows of 256 rank 16", "op": "forward", "m": 64, "k": 4096, "n": 14336, "g": 256,
         "rank": 16, "skew": 0.5, "none": 0.1, "order": True},
        # serving, prompts of many requests together, an odd number of rows, larger adapters
        {"name": "forward 2061 rows of 40 rank 64", "op": "forward", "m": 2061, "k": 7168, "n": 2048, "g": 40,
         "rank": 64, "skew": 1.1, "none": 0.1, "order": True},
        # fine-tuning: an adapter for each of 8 experts, rows sorted by expert as they come from the router
        {"name": "forward 16384 rows of 8 rank 16", "op": "forward", "m": 16384, "k": 4096, "n": 14336, "g": 8,
         "rank": 16, "skew": 0.0, "none": 0.0, "order": False},
        # its backward pass: the gradient of the rows
        {"name": "grad input 16384 rows of 8 rank 16", "op": "grad_input", "m": 16384, "k": 4096, "n": 14336, "g": 8,
         "rank": 16, "skew": 0.0, "none": 0.0, "order": False},
        # the same for a small odd batch of several tenants
        {"name": "grad input 515 rows of 5 rank 40", "op": "grad_input", "m": 515, "k": 1408, "n": 2048, "g": 5,
         "rank": 40, "skew": 0.5, "none": 0.1, "order": True},
        # the gradient of the down matrices from the 8-bit checkpoint of the layer's input
        {"name": "grad weight 16384x4096 rank 16 8-bit", "op": "grad_weight", "m": 16384, "c": 4096, "g": 8, "rank": 16,
         "skew": 0.0, "none": 0.0, "order": False, "z": "mxfp8", "out": "f32"},
        # the gradient of the up matrices of several tenants
        {"name": "grad weight 4099x7168 rank 64", "op": "grad_weight", "m": 4099, "c": 7168, "g": 24, "rank": 64,
         "skew": 0.5, "none": 0.1, "order": True, "z": "bf16", "out": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["group", "checkpoint", "forward", "forward", "grad_input", "grad_weight", "grad_weight"])
    routing = {"skew": rng.choice([0.0, 0.5, 1.1]), "none": rng.choice([0.0, 0.1])}
    if op == "group":
        return {"op": op, "m": _log(rng, 1, 65536), "g": _log(rng, 1, 1024), **routing}
    if op == "checkpoint":
        k = _log(rng, 32, 16384, 32)
        return {"op": op, "m": _log(rng, 1, min(65536, (1 << 26) // k)), "k": k, "dtype": rng.choice(["bf16", "f32"])}
    g = _log(rng, 1, 256)
    case = {"op": op, "g": g, "rank": rng.choice([8, 16, 16, 24, 32, 40, 64, 64, 96, 128]), "order": rng.random() < 0.5,
            **routing}
    if op == "grad_weight":
        c = _log(rng, 64, 14336, 32)
        case["m"] = _log(rng, 1, max(1, min(32768, (1 << 26) // c, (1 << 32) // (c * g))))
        case["c"], case["z"], case["out"] = c, rng.choice(["bf16", "mxfp8"]), rng.choice(["bf16", "f32"])
        return case
    case["k"], case["n"] = _log(rng, 64, 14336, 8), _log(rng, 64, 14336, 8)
    widest = max(case["k"], case["n"])
    case["m"] = _log(rng, 1, max(1, min(32768, (1 << 28) // (case["k"] + case["n"]), (1 << 32) // (widest * g))))
    return case


# ------------------------------------------------------------------------------ inputs
def _randn(gen, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _ids(case, gen):
    """Each row's adapter, popularity rank^-skew, a share `none` of the rows without one (-1): int32 [M]."""
    m, g = case["m"], case["g"]
    ranks = torch.randperm(g, generator=gen, device=DEV) + 1
    ends = torch.cumsum(ranks.double() ** -case["skew"], 0)
    ids = torch.searchsorted(ends / ends[-1], torch.rand(m, generator=gen, device=DEV, dtype=torch.float64))
    ids = ids.clamp(max=g - 1)
    ids[torch.rand(m, generator=gen, device=DEV) < case["none"]] = -1
    return ids.int()


def _route(case, gen, st):
    """Group sizes, and the order of the rows unless they already stand sorted."""
    ids = _ids(case, gen)
    key = torch.where(ids < 0, case["g"], ids).long()
    sizes = torch.bincount(key, minlength=case["g"] + 1)[:case["g"]]
    st["sizes"], st["capacity"] = sizes.int(), max(1, int(sizes.max()))
    st["order"] = torch.argsort(key, stable=True).int() if case["order"] else None


def _activation(gen, m, k):
    """Rows of an activation: a few channels carry outliers, one row in 16 is an empty slot of zeros."""
    x = _randn(gen, (m, k)) * (1 + 15 * (torch.rand(k, generator=gen, device=DEV) < 0.01))
    x[torch.rand(m, generator=gen, device=DEV) < 1 / 16] = 0
    return x


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    st = dict(case)
    op = case["op"]
    empty = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)
    if op == "group":
        st["ids"] = _ids(case, gen)
        st["sizes"], st["order"] = empty(case["g"], torch.int32), empty(case["m"], torch.int32)
    elif op == "checkpoint":
        m, k = case["m"], case["k"]
        st["x"] = _activation(gen, m, k).to({"bf16": torch.bfloat16, "f32": torch.float32}[case["dtype"]])
        st["codes"], st["scales"] = empty((m, k), torch.uint8), empty((m, k // 32), torch.uint8)
        st["restored"] = empty((m, k), st["x"].dtype)
    elif op == "grad_weight":
        m, c, g, r = case["m"], case["c"], case["g"], case["rank"]
        _route(case, gen, st)
        st["t"] = _randn(gen, (m, r), torch.bfloat16)
        z = _activation(gen, m, c)
        if case["z"] == "mxfp8":
            s, q = _quantize(z)
            st["z"] = q.to(torch.float8_e4m3fn).view(torch.uint8).view(m, c)
            st["zs"] = s.to(torch.uint8)
        else:
            st["z"], st["zs"] = z.to(torch.bfloat16), None
        st["dw"] = empty((g, r, c), {"bf16": torch.bfloat16, "f32": torch.float32}[case["out"]])
    else:
        m, k, n, g, r = (case[f] for f in ("m", "k", "n", "g", "rank"))
        _route(case, gen, st)
        st["scale"] = torch.rand(g, generator=gen, device=DEV) + 0.5
        st["down"] = _randn(gen, (g, r, k), torch.bfloat16, k ** -0.5)
        st["up"] = _randn(gen, (g, r, n), torch.bfloat16, 0.05)
        width_in, width_out = (k, n) if op == "forward" else (n, k)
        st["x"] = _activation(gen, m, width_in).to(torch.bfloat16)
        st["base"] = _randn(gen, (m, width_out), torch.bfloat16)
        st["out"], st["t"] = empty((m, width_out), torch.bfloat16), empty((m, r), torch.bfloat16)
    return st


# ------------------------------------------------------------------------------ plain forms
def _quantize(x):
    """fp32 x [..., K] -> scale bytes [..., K/32] and the blocks' E4M3 values before scaling [..., K/32, 32]."""
    b = x.float().unflatten(-1, (-1, 32))
    bits = b.abs().amax(-1).view(torch.int32)
    # amax / 2^(s - 127) <= 448 = 1.75 x 2^8: the exponent less 8, and one more where the mantissa is above 1.75
    s = ((bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000).int()).clamp(min=0)
    v = b * ((254 - s) << 23).view(torch.float32).unsqueeze(-1)
    # 3 bits behind the leading one, steps of 2^-9 below 2^-6; torch.round takes halves to even
    e = ((v.abs().view(torch.int32) >> 23) - 127).clamp(min=-6) - 3
    step = ((e + 127) << 23).view(torch.float32)
    return s, torch.round(v / step) * step


def _power(s):
    """2^(s - 127) in fp32 from scale bytes (its lowest a subnormal)."""
    s = s.int()
    return torch.where(s > 0, s << 23, torch.full_like(s, 0x400000)).view(torch.float32)


def _decode(codes, s):
    """fp32 values [..., K] of E4M3 codes [..., K] with scale bytes [..., K/32]."""
    c = torch.arange(256, device=codes.device)
    e, mant = (c >> 3) & 15, (c & 7).float()
    mag = torch.where(e > 0, (8 + mant) * ((e.int() + 117) << 23).view(torch.float32), mant / 512)
    table = torch.where(c >= 128, -mag, mag)
    v = table[codes.int()].unflatten(-1, (-1, 32)) * _power(s).unsqueeze(-1)
    return v.flatten(-2)


def _plain_group(st):
    g = st["g"]
    key = torch.where((st["ids"] < 0) | (st["ids"] >= g), g, st["ids"]).long()
    sizes = torch.zeros(g + 1, dtype=torch.int32, device=DEV)
    sizes.scatter_add_(0, key, torch.ones_like(st["ids"]))
    return sizes[:g], torch.argsort(key, stable=True).int()


def _plain_checkpoint(st):
    s, q = _quantize(st["x"])
    return (q * _power(s).unsqueeze(-1)).flatten(-2).to(st["x"].dtype)


def _groups(st):
    """Each sorted position's group (g past the last) and place within it."""
    m = st["m"]
    ends = torch.cumsum(st["sizes"], 0)
    p = torch.arange(m, device=DEV)
    group = torch.searchsorted(ends, p, right=True)
    start = torch.cat((ends - st["sizes"], ends[-1:]))
    return group, (p - start[group]).clamp(max=st["capacity"] - 1)


def _sorted(st, x):
    return x if st["order"] is None else x[st["order"].long()]


def _pad(st, x, group, pos):
    """Sorted rows [M, W] -> fp32 [G, capacity, W], zeros where a group has no row."""
    out = torch.zeros((st["g"] + 1, st["capacity"], x.shape[1]), device=DEV)
    out[group, pos] = x.float()
    return out[:st["g"]]


def _plain_apply(st, first, second):
    """(out, t): t = scale x first^T by group, out = base + t second."""
    g = st["g"]
    group, pos = _groups(st)
    xp = _pad(st, _sorted(st, st["x"]), group, pos)
    tp = torch.bmm(xp, first.float().transpose(1, 2)) * st["scale"].view(g, 1, 1)
    yp = torch.bmm(tp, second.float())
    live, at = (group < g).unsqueeze(1), group.clamp(max=g - 1)
    t = torch.where(live, tp[at, pos], 0.0).to(torch.bfloat16)
    y = torch.where(live, yp[at, pos], 0.0)
    rows = slice(None) if st["order"] is None else st["order"].long()
    out = st["base"].float()
    out[rows] += y
    return out.to(torch.bfloat16), t


def _plain_grad_weight(st):
    group, pos = _groups(st)
    z = st["z"] if st["zs"] is None else _decode(st["z"], st["zs"])
    tp, zp = _pad(st, st["t"], group, pos), _pad(st, _sorted(st, z), group, pos)
    return torch.bmm(tp.transpose(1, 2), zp).to(st["dw"].dtype)


# ------------------------------------------------------------------------------ the framework's calls
def _own(st):
    import group_gemm_gb300 as gg

    op = st["op"]
    if op == "group":
        gg.rdot_lora_group(st["ids"], st["g"], st["sizes"], st["order"])
        return st["sizes"], st["order"]
    if op == "checkpoint":
        gg.rdot_quantize_mxfp8(st["x"], st["codes"], st["scales"])
        gg.rdot_dequantize_mxfp8(st["codes"], st["scales"], st["restored"])
        return st["restored"]
    if op == "grad_weight":
        gg.rdot_lora_grad_weight(st["t"], st["z"], st["sizes"], st["dw"], order=st["order"], z_scale=st["zs"])
        return st["dw"]
    call = gg.rdot_lora_forward if op == "forward" else gg.rdot_lora_grad_input
    call(st["x"], st["down"], st["up"], st["sizes"], st["out"], st["t"], order=st["order"], scale=st["scale"],
         base=st["base"])
    return st["out"], st["t"]


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "forward":
        return _plain_apply(state, state["down"], state["up"])
    if op == "grad_input":
        return _plain_apply(state, state["up"], state["down"])
    return {"group": _plain_group, "checkpoint": _plain_checkpoint, "grad_weight": _plain_grad_weight}[op](state)


# ------------------------------------------------------------------------------ work and exact values
def _used(case):
    """How many adapters have a row, on average."""
    p = [r ** -case["skew"] for r in range(1, case["g"] + 1)]
    rows = case["m"] * (1 - case["none"])
    return min(case["g"], rows, sum(1 - (1 - q / sum(p)) ** rows for q in p))


def work(case):
    op, m = case["op"], case["m"]
    if op == "group":
        return {"bytes": 8 * m + 4 * case["g"], "flops": m}
    if op == "checkpoint":
        n, esize = m * case["k"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * (esize + 1 + 1 / 32), "flops": 3 * n}
    rows, r = m * (1 - case["none"]), case["rank"]
    if op == "grad_weight":
        c = case["c"]
        zsize = 1 + 1 / 32 if case["z"] == "mxfp8" else 2
        return {"bytes": rows * c * zsize + 2 * rows * r + (4 if case["out"] == "f32" else 2) * case["g"] * r * c,
                "flops": 2 * rows * r * c}
    k, n = (case["k"], case["n"]) if op == "forward" else (case["n"], case["k"])
    return {"bytes": 2 * rows * k + 4 * m * n + 2 * m * r + 2 * _used(case) * r * (k + n),
            "flops": 2 * rows * r * (k + n)}


def _e4m3_64(v):
    """v in float64 to the nearest E4M3 value, ties to even; |v| <= 448."""
    e = (torch.frexp(v).exponent - 1).clamp(min=-6)
    step = torch.exp2(torch.zeros_like(v)) / 8 * ((e.long() + 1023) << 52).view(torch.float64)
    return torch.round(v / step) * step


def exact(case, seed):
    op = case["op"]
    if op == "group":
        return None
    st = prepare(case, seed)
    if op == "checkpoint":
        b = st["x"].double().unflatten(-1, (-1, 32))
        amax = b.abs().amax(-1, keepdim=True)
        mant, e = torch.frexp(torch.where(amax > 0, amax, torch.full_like(amax, 2.0 ** -140)))
        e = (e - 9 + (mant > 0.875).int()).clamp(min=-127)
        scale = ((e.long() + 1023) << 52).view(torch.float64)
        return (_e4m3_64(b / scale) * scale).flatten(-2)
    sizes = st["sizes"].tolist()
    rows = torch.arange(case["m"], device=DEV) if st["order"] is None else st["order"].long()
    if op == "grad_weight":
        if st["zs"] is None:
            z = st["z"].double()
        else:
            scale = ((st["zs"].long() + 896) << 52).view(torch.float64)
            z = st["z"].view(torch.float8_e4m3fn).double() * scale.repeat_interleave(32, 1)
        dw = torch.zeros(st["dw"].shape, dtype=torch.float64, device=DEV)
        at = 0
        for i, s in enumerate(sizes):
            dw[i] = st["t"][at:at + s].double().t() @ z[rows[at:at + s]]
            at += s
        return dw
    first, second = ("down", "up") if op == "forward" else ("up", "down")
    out = st["base"].double()
    t = torch.zeros(st["t"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for i, s in enumerate(sizes):
        if s:
            part = slice(at, at + s)
            t[part] = (st["x"][rows[part]].double() @ st[first][i].double().t()) * st["scale"][i].double()
            out[rows[part]] += t[part] @ st[second][i].double()
            at += s
    return out, t
