"""The measured cases of the 4-bit expert and routing-gradient operators, with their plain forms.

Five operators of a mixture-of-experts layer:

* ``quantize``: MXFP4 quantisation (E2M1 codes, one E8M0 scale per 32 elements of the contraction) of
  activation rows ``[M, K]`` or of a layer's weights ``[G, K, N]``, with the values the codes stand for;
* ``experts``: bf16 activation rows sorted by expert, quantised and multiplied by 4-bit expert weights;
* ``unpermute_grad``: the gradient of the router-weighted un-permute (of the expert outputs and the weights);
* ``permute_grad``: the gradient of the permute (of the token rows);
* ``router_grad``: the gradient of the top-k router (of the gate logits).

Plain forms are elementary torch operations in 32 bits. ``own`` selects the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
MODES = {"values": 0, "softmax": 1, "softmax_topk": 2}


def listed():
    return [
        # one training step's activations of the Mixtral-like layer: 8192 tokens, two copies each
        {"name": "quantize rows 16384x4096", "op": "quantize", "what": "rows", "m": 16384, "k": 4096, "dtype": "bf16"},
        # a small batch with an odd number of rows and a width of 44 blocks, fp32 activations: latency
        {"name": "quantize rows 37x1408 f32", "op": "quantize", "what": "rows", "m": 37, "k": 1408, "dtype": "f32"},
        # the fp32 master weights of one projection of the Mixtral-like layer, once per training step
        {"name": "quantize weights 8x4096x14336", "op": "quantize", "what": "weights", "g": 8, "k": 4096, "n": 14336,
         "dtype": "f32"},
        # serving, one token: the Mixtral-like up projection, top-2 of 8
        {"name": "experts 1 token top-2 of 8", "op": "experts", "tokens": 1, "topk": 2, "g": 8, "k": 4096, "n": 14336,
         "skew": 0.0, "spare": 0},
        # serving, a batch of 64: the DeepSeek-like layer, top-8 of 256, skewed routing, many experts without a row
        {"name": "experts 64 tokens top-8 of 256", "op": "experts", "tokens": 64, "topk": 8, "g": 256, "k": 7168,
         "n": 4096, "skew": 1.1, "spare": 0},
        # a prompt or a training step: 8192 tokens top-2 of 8, the Mixtral-like up projection
        {"name": "experts 8192 tokens top-2 of 8", "op": "experts", "tokens": 8192, "topk": 2, "g": 8, "k": 4096,
         "n": 14336, "skew": 0.0, "spare": 0},
        # backward of the layer's last step, Mixtral-like
        {"name": "unpermute grad 8192x2x4096", "op": "unpermute_grad", "tokens": 8192, "topk": 2, "g": 8, "n": 4096,
         "drop": 0.0},
        # a small odd batch of the DeepSeek-like layer in which one copy in ten was dropped
        {"name": "unpermute grad 61x8x7168", "op": "unpermute_grad", "tokens": 61, "topk": 8, "g": 256, "n": 7168,
         "drop": 0.1},
        # backward of the layer's first step: 8192 tokens top-8 of 128
        {"name": "permute grad 8192x8x4096", "op": "permute_grad", "tokens": 8192, "topk": 8, "g": 128, "n": 4096,
         "drop": 0.0, "dtype": "bf16"},
        # the same on a small odd batch in fp32, with dropped copies
        {"name": "permute grad 129x4x2048 f32", "op": "permute_grad", "tokens": 129, "topk": 4, "g": 64, "n": 2048,
         "drop": 0.1, "dtype": "f32"},
        # backward of the router: softmax over all 256 experts, top-8
        {"name": "router grad 4096x256 softmax", "op": "router_grad", "tokens": 4096, "g": 256, "topk": 8,
         "mode": "softmax", "dtype": "f32"},
        # backward of the router: softmax over the two selected of 8 experts, bf16 logits
        {"name": "router grad 8192x8 softmax_topk", "op": "router_grad", "tokens": 8192, "g": 8, "topk": 2,
         "mode": "softmax_topk", "dtype": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "experts", "experts", "unpermute_grad", "permute_grad", "router_grad"])
    if op == "quantize":
        dtype = rng.choice(["bf16", "f32"])
        if rng.random() < 0.5:
            k = _log(rng, 32, 16384, 32)
            return {"op": op, "what": "rows", "m": _log(rng, 1, min(65536, (1 << 27) // k)), "k": k, "dtype": dtype}
        k, n = _log(rng, 32, 8192, 32), _log(rng, 8, 16384, 8)
        return {"op": op, "what": "weights", "g": _log(rng, 1, max(1, min(128, (1 << 28) // (k * n)))), "k": k, "n": n,
                "dtype": dtype}
    g = _log(rng, 2, 256)
    topk = rng.randint(1, min(8, g))
    if op == "experts":
        k, n = _log(rng, 64, 8192, 32), _log(rng, 64, 14336, 8)
        g = max(topk, min(g, (1 << 31) // (k * n)))
        tokens = _log(rng, 1, max(1, min(65536 // topk, (1 << 39) // (topk * k * n))))
        return {"op": op, "tokens": tokens, "topk": topk, "g": g, "k": k, "n": n,
                "skew": rng.choice([0.0, 0.5, 1.1]), "spare": rng.choice([0, 0, rng.randint(1, 200)])}
    if op == "router_grad":
        return {"op": op, "tokens": _log(rng, 1, 32768), "g": g, "topk": topk, "mode": rng.choice(sorted(MODES)),
                "dtype": rng.choice(["bf16", "f32"])}
    n = _log(rng, 64, 8192, 8)
    tokens = _log(rng, 1, min(16384, (1 << 27) // (n * topk)))
    case = {"op": op, "tokens": tokens, "topk": topk, "g": g, "n": n, "drop": rng.choice([0.0, 0.1])}
    if op == "permute_grad":
        case["dtype"] = rng.choice(["bf16", "f32"])
    return case


# ------------------------------------------------------------------------------ inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _randn(gen, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _route(tokens, topk, g, skew, gen):
    """Each token's topk distinct experts, popularity rank^-skew (Gumbel top-k): int64 [T, k]."""
    ranks = torch.randperm(g, generator=gen, device=DEV) + 1
    gumbel = -torch.log(-torch.log(torch.rand((tokens, g), generator=gen, device=DEV).clamp(1e-9, 1 - 1e-7)))
    return torch.topk(gumbel - skew * torch.log(ranks.float()), topk, dim=1).indices


def _sort(ids, g, drop, gen):
    """The permute's index outputs for these ids, a share `drop` of the copies dropped (id -1)."""
    flat = ids.reshape(-1).clone()
    if drop:
        flat[torch.rand(flat.shape, generator=gen, device=DEV) < drop] = -1
    key = torch.where(flat < 0, torch.full_like(flat, g), flat)
    perm = torch.argsort(key, stable=True)
    kept = (flat >= 0)[perm]
    order = torch.where(kept, perm, torch.full_like(perm, -1))
    inv = torch.full_like(perm, -1)
    inv[perm] = torch.where(kept, torch.arange(perm.numel(), device=DEV), inv)
    return order.int(), inv.int()


def _tile_scales(s):
    """Scale bytes [G, N, K/32] in blocks of 128 rows x 4: [G, ceil(N/128), ceil(K/128), 512], byte
    16 (n % 32) + 4 (n / 32 % 4) + k / 32 % 4 of a block, zeros past N and K."""
    g, n, kb = s.shape
    nb, ka = -(-n // 128), -(-kb // 4)
    pad = torch.zeros((g, nb * 128, ka * 4), dtype=torch.uint8, device=s.device)
    pad[:, :n, :kb] = s
    return pad.view(g, nb, 4, 32, ka, 4).permute(0, 1, 4, 3, 2, 5).reshape(g, nb, ka, 512).contiguous()


def _untile_scales(t, n, kb):
    g, nb, ka, _ = t.shape
    return t.view(g, nb, ka, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(g, nb * 128, ka * 4)[:, :n, :kb]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    st = dict(case)
    op = case["op"]
    if op == "quantize":
        dt = _dtype(case["dtype"])
        if case["what"] == "rows":
            m, k = case["m"], case["k"]
            # a few channels carry outliers; one row in 16 is an empty slot of zeros
            x = _randn(gen, (m, k)) * (1 + 15 * (torch.rand(k, generator=gen, device=DEV) < 0.01))
            x[torch.rand(m, generator=gen, device=DEV) < 1 / 16] = 0
            st["x"] = x.to(dt)
            st["codes"] = torch.empty((m, k // 2), dtype=torch.uint8, device=DEV)
            st["scales"] = torch.empty((m, k // 32), dtype=torch.uint8, device=DEV)
        else:
            g, k, n = case["g"], case["k"], case["n"]
            st["x"] = _randn(gen, (g, k, n), dt, 0.02)
            st["codes"] = torch.empty((g, n, k // 2), dtype=torch.uint8, device=DEV)
            st["scales"] = torch.empty((g, -(-n // 128), -(-k // 128), 512), dtype=torch.uint8, device=DEV)
        st["values"] = torch.empty(st["x"].shape, dtype=torch.bfloat16, device=DEV)
    elif op == "experts":
        tokens, topk, g, k, n = (case[f] for f in ("tokens", "topk", "g", "k", "n"))
        ids = _route(tokens, topk, g, case["skew"], gen)
        sizes = torch.bincount(ids.reshape(-1), minlength=g)
        m = tokens * topk + case["spare"]   # `spare`: room for rows that this batch does not fill
        st["sizes"] = sizes.int()
        st["capacity"] = int(sizes.max())
        st["x"] = _randn(gen, (m, k), torch.bfloat16)
        # the layer's weights as a serving program keeps them: codes [G, N, K/2] and scales in blocks
        st["w"] = torch.empty((g, n, k // 2), dtype=torch.uint8, device=DEV)
        s = torch.empty((g, n, k // 32), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 27) // (n * k))
        for i in range(0, g, step):
            c, sc, _ = _quantize(_randn(gen, (min(step, g - i), n, k), std=0.02))
            st["w"][i:i + step], s[i:i + step] = c, sc
        st["ws"] = _tile_scales(s)
        st["codes"] = torch.empty((m, k // 2), dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty((m, k // 32), dtype=torch.uint8, device=DEV)
        st["out"] = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    elif op in ("unpermute_grad", "permute_grad"):
        tokens, topk, n = case["tokens"], case["topk"], case["n"]
        ids = _route(tokens, topk, case["g"], 0.5, gen)
        st["order"], st["inv"] = _sort(ids, case["g"], case["drop"], gen)
        if op == "unpermute_grad":
            st["dout"] = _randn(gen, (tokens, n), torch.bfloat16, 0.1)
            st["y"] = _randn(gen, (tokens * topk, n), torch.bfloat16)
            st["weights"] = torch.softmax(_randn(gen, (tokens, topk)), dim=1)
            st["dy"] = torch.empty((tokens * topk, n), dtype=torch.bfloat16, device=DEV)
            st["dw"] = torch.empty((tokens, topk), dtype=torch.float32, device=DEV)
        else:
            dt = _dtype(case["dtype"])
            st["dxs"] = _randn(gen, (tokens * topk, n), dt, 0.1)
            st["dx"] = torch.empty((tokens, n), dtype=dt, device=DEV)
    else:
        tokens, g, topk = case["tokens"], case["g"], case["topk"]
        st["logits"] = _randn(gen, (tokens, g), _dtype(case["dtype"]))
        top, ids = torch.topk(st["logits"].float(), topk, dim=1)
        st["ids"] = ids.int()
        st["weights"] = {"values": top, "softmax_topk": torch.softmax(top, dim=1),
                         "softmax": torch.softmax(st["logits"].float(), dim=1).gather(1, ids)}[case["mode"]].contiguous()
        st["dw"] = _randn(gen, (tokens, topk))
        st["dlogits"] = torch.empty((tokens, g), dtype=st["logits"].dtype, device=DEV)
    return st


# ------------------------------------------------------------------------------ plain forms
_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x):
    """fp32 x [..., K] -> codes [..., K/2], scale bytes [..., K/32], fp32 values [..., K]."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    s = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)
    a = b.abs() * ((254 - s) << 23).view(torch.float32).unsqueeze(-1)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    mags = torch.tensor(_MAGNITUDES, device=x.device)
    scale = torch.ldexp(torch.ones_like(amax), s - 127).unsqueeze(-1)
    values = torch.copysign(mags[code.int()] * scale, b).flatten(-2)
    code = (code + 8 * torch.signbit(b).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s.to(torch.uint8), values


def _decode(codes, s):
    """fp32 values [..., K] of codes [..., K/2] with scale bytes [..., K/32]."""
    e2m1 = torch.tensor(_MAGNITUDES + tuple(-v for v in _MAGNITUDES), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack((e2m1[byte & 15], e2m1[byte >> 4]), dim=1)
    v = torch.index_select(pair, 0, codes.reshape(-1).int()).view(*s.shape, 32)
    v *= torch.ldexp(torch.ones(s.shape, device=s.device), s.int() - 127).unsqueeze(-1)
    return v.flatten(-2)


def _plain_quantize(st):
    if st["what"] == "rows":
        codes, s, values = _quantize(st["x"])
        return codes, s, values.to(torch.bfloat16)
    codes, s, values = _quantize(st["x"].transpose(1, 2).float().contiguous())
    return codes, _tile_scales(s), values.to(torch.bfloat16).transpose(1, 2).contiguous()


def _plain_experts(st):
    m, k = st["x"].shape
    g, n = st["w"].shape[:2]
    x = _quantize(st["x"])[2]
    w = _decode(st["w"], _untile_scales(st["ws"], n, k // 32))
    ends = torch.cumsum(st["sizes"], 0)
    rows = torch.arange(m, device=DEV)
    group = torch.searchsorted(ends, rows, right=True)      # g for the rows past the last group
    start = torch.cat((ends - st["sizes"], ends[-1:]))
    pos = (rows - start[group]).clamp(max=st["capacity"] - 1)
    xp = torch.zeros((g + 1, st["capacity"], k), device=DEV)
    xp[group, pos] = x
    y = torch.bmm(xp[:g], w.transpose(1, 2))
    return torch.where((group < g).unsqueeze(1), y[group.clamp(max=g - 1), pos], 0.0).to(torch.bfloat16)


def _plain_unpermute_grad(st):
    t, k = st["weights"].shape
    kept = (st["inv"] >= 0).view(t, k)
    y = st["y"][st["inv"].clamp(min=0).long()].view(t, k, -1).float()
    dw = torch.where(kept, (y * st["dout"].float().unsqueeze(1)).sum(-1), 0.0)
    f = st["order"].clamp(min=0).long()
    dy = st["weights"].reshape(-1)[f].unsqueeze(1) * st["dout"].float()[f // k]
    return torch.where((st["order"] >= 0).unsqueeze(1), dy, 0.0).to(torch.bfloat16), dw


def _plain_permute_grad(st):
    t = st["dx"].shape[0]
    d = st["dxs"][st["inv"].clamp(min=0).long()].float()
    d = torch.where((st["inv"] >= 0).unsqueeze(1), d, 0.0)
    return d.view(t, -1, d.shape[1]).sum(1).to(st["dxs"].dtype)


def _plain_router_grad(st):
    w, dw, logits = st["weights"], st["dw"], st["logits"].float()
    out = torch.zeros_like(logits)
    if st["mode"] == "values":
        out.scatter_(1, st["ids"].long(), dw)
    else:
        s = (w * dw).sum(1, keepdim=True)
        if st["mode"] == "softmax_topk":
            out.scatter_(1, st["ids"].long(), w * (dw - s))
        else:
            e = torch.exp(logits - logits.amax(1, keepdim=True))
            out.scatter_(1, st["ids"].long(), w * dw)
            out -= e / e.sum(1, keepdim=True) * s
    return out.to(st["logits"].dtype)


# ------------------------------------------------------------------------------ the framework's calls
_plans = {}   # one plan for each problem shape, as a program keeps it


def _own(st):
    import group_gemm_gb300 as gg

    op = st["op"]
    if op == "quantize":
        call = gg.rdot_quantize_mxfp4 if st["what"] == "rows" else gg.rdot_quantize_mxfp4_weight
        call(st["x"], st["codes"], st["scales"], st["values"])
        return st["codes"], st["scales"], st["values"]
    if op == "experts":
        m, k = st["x"].shape
        g, n = st["w"].shape[:2]
        plan = _plans.get((m, k, n, g))
        if plan is None:
            plan = _plans[m, k, n, g] = gg.Plan(m, k, n, g, "forward_mxfp4", "e2m1", "bf16")
        gg.rdot_quantize_mxfp4(st["x"], st["codes"], st["scales"])
        gg.rdot_forward_mxfp4(plan.handle, st["codes"], st["scales"], st["w"], st["ws"], st["sizes"], st["out"],
                              plan.workspace)
        return st["out"]
    if op == "unpermute_grad":
        gg.rdot_moe_unpermute_grad(st["dout"], st["y"], st["order"], st["inv"], st["weights"], st["dy"], st["dw"])
        return st["dy"], st["dw"]
    if op == "permute_grad":
        gg.rdot_moe_permute_grad(st["dxs"], st["inv"], st["dx"])
        return st["dx"]
    gg.rdot_router_topk_grad(st["logits"], st["ids"], st["weights"], st["dw"], MODES[st["mode"]], st["dlogits"])
    return st["dlogits"]


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "experts": _plain_experts, "unpermute_grad": _plain_unpermute_grad,
            "permute_grad": _plain_permute_grad, "router_grad": _plain_router_grad}[state["op"]](state)


# ------------------------------------------------------------------------------ work and exact values
def work(case):
    op = case["op"]
    esize = 4 if case.get("dtype") == "f32" else 2
    if op == "quantize":
        n = case["m"] * case["k"] if case["what"] == "rows" else case["g"] * case["k"] * case["n"]
        return {"bytes": n * (esize + 0.5 + 1 / 32 + 2), "flops": 2 * n}
    if op == "experts":
        rows, k, n = case["tokens"] * case["topk"], case["k"], case["n"]
        routed = min(case["g"], rows)   # the most experts that can have a row
        if case["skew"]:                # how many a skewed routing reaches, on average
            p = [r ** -case["skew"] for r in range(1, case["g"] + 1)]
            routed = min(routed, sum(1 - (1 - q / sum(p)) ** rows for q in p))
        return {"bytes": 2 * rows * k + routed * n * k * (0.5 + 1 / 32) + 2 * (rows + case["spare"]) * n,
                "flops": 2 * rows * k * n}
    t = case["tokens"]
    if op == "unpermute_grad":
        c = t * case["topk"]
        return {"bytes": 2 * case["n"] * (t + 2 * c) + 16 * c, "flops": 3 * c * case["n"]}
    if op == "permute_grad":
        return {"bytes": esize * case["n"] * (t + t * case["topk"]) + 4 * t * case["topk"],
                "flops": t * case["topk"] * case["n"]}
    reads = 2 if case["mode"] == "softmax" else 1
    return {"bytes": esize * reads * t * case["g"] + 12 * t * case["topk"], "flops": 4 * t * case["g"]}


def _grid64(v):
    """v / scale in float64 to the nearest E2M1 magnitude (ties to the even code), saturated."""
    v = v.abs().clamp(max=6.0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).to(v.dtype)
    return torch.round(v / step) * step   # torch.round: half to even, and the even multiple has the even code


def _values64(x):
    """The MXFP4 values of x [..., K] in float64."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(torch.where(amax > 0, amax, torch.full_like(amax, 2.0 ** -126))).exponent - 1 - 2
    scale = torch.ldexp(torch.ones_like(amax), e.clamp(min=-127))
    return (torch.sign(b) * _grid64(b / scale) * scale).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        if case["what"] == "rows":
            return None, None, _values64(st["x"])
        out = torch.empty(st["x"].shape, dtype=torch.float64, device=DEV)
        for i in range(case["g"]):
            out[i] = _values64(st["x"][i].t()).t()
        return None, None, out
    if op == "experts":
        m, k = st["x"].shape
        n = case["n"]
        x = _values64(st["x"])
        s = _untile_scales(st["ws"], n, k // 32)
        out = torch.zeros((m, n), dtype=torch.float64, device=DEV)
        low = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=DEV)
        at = 0
        for i, rows in enumerate(st["sizes"].tolist()):
            if rows:
                c = torch.stack((st["w"][i] & 15, st["w"][i] >> 4), dim=-1).flatten(-2).int()
                w = torch.where(c >= 8, -low[c & 7], low[c & 7])
                scale = torch.ldexp(torch.ones(s[i].shape, dtype=torch.float64, device=DEV), s[i].int() - 127)
                w *= scale.repeat_interleave(32, 1)
                out[at:at + rows] = x[at:at + rows] @ w.t()
                at += rows
        return out
    k = case["topk"]
    if op == "unpermute_grad":
        dout, y = st["dout"].double(), st["y"].double()
        flat = torch.arange(case["tokens"] * k, device=DEV)
        kept = st["inv"].long() >= 0
        f, p = flat[kept], st["inv"].long()[kept]
        dw = torch.zeros(flat.numel(), dtype=torch.float64, device=DEV)
        dy = torch.zeros_like(y)
        for i in range(0, f.numel(), 8192):
            fi, pi = f[i:i + 8192], p[i:i + 8192]
            dw[fi] = torch.einsum("cn,cn->c", dout[fi // k], y[pi])
            dy[pi] = dout[fi // k] * st["weights"].double().reshape(-1)[fi].unsqueeze(1)
        return dy, dw.view(-1, k)
    if op == "permute_grad":
        out = torch.zeros(st["dx"].shape, dtype=torch.float64, device=DEV)
        inv = st["inv"].long().view(-1, k)
        for j in range(k):
            kept = inv[:, j] >= 0
            out[kept] += st["dxs"][inv[kept, j]].double()
        return out
    w, dw = st["weights"].double(), st["dw"].double()
    onehot = torch.zeros((*w.shape, case["g"]), dtype=torch.float64, device=DEV)
    onehot.scatter_(2, st["ids"].long().unsqueeze(2), 1.0)
    if case["mode"] == "values":
        return torch.einsum("tk,tke->te", dw, onehot)
    s = torch.einsum("tk,tk->t", w, dw).unsqueeze(1)
    if case["mode"] == "softmax_topk":
        return torch.einsum("tk,tke->te", w * (dw - s), onehot)
    return torch.einsum("tk,tke->te", w * dw, onehot) - torch.softmax(st["logits"].double(), dim=1) * s
