"""Single-CTA tensor-core kernels whose producer has issued all its loads when a consumer gives up.

The contraction is so short that a CTA's loads all fit its ring: the producer ends normally, and a consumer
whose wait runs out (the plan's limit is a nanosecond) leaves with loads in flight. They must land before
the CTA ends, not in the shared memory of the next call's CTAs: whole calls that follow at once on the
same stream give what they gave before any stop, bit for bit. No GPU fault is provoked: the waits simply run out.
"""
import numpy as np
import pytest
import torch

import group_gemm_gb300 as gg
import rdot_inputs as ri

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
SIZES = [60, 0, 40, 28]


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def _bf16(shape, seed, std=1.0):
    return torch.from_numpy(ri.host_normal(shape, seed, std)).to(torch.bfloat16).to(DEV)


def _mx(shape, seed, axis, std=1.0):
    q, s = ri.quantize_mx_e4m3(torch.from_numpy(ri.host_normal(shape, seed, std)), axis=axis)
    return q.to(DEV), s.to(DEV)


def _case(kind):
    """(a function that makes a plan, a function that runs one call on a plan, the output it writes)."""
    m, k, n, g = sum(SIZES), 128, 512, len(SIZES)
    sizes = list(SIZES)
    if kind.endswith("skinny"):
        sizes, m = [20, 0, 28, 0], 48
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    bf16, f32 = torch.bfloat16, torch.float32
    if kind in ("fwd", "fwd_skinny"):
        x, w, out = _bf16((m, k), 1), _bf16((g, k, n), 2, 0.05), torch.empty((m, n), dtype=bf16, device=DEV)
        flags = gg.RDOT_FLAG_NO_CTA_PAIR | (gg.RDOT_FLAG_NO_SKINNY if kind == "fwd" else 0)
        return (lambda: gg.Plan(m, k, n, g, "forward", "bf16", "bf16", flags=flags),
                lambda p: gg.rdot_forward(p.handle, x, w, gs, out, p.workspace), out)
    if kind in ("mxfp8", "mxfp8_skinny"):
        (x, xs), (w, ws) = _mx((m, k), 3, 1), _mx((g, k, n), 4, 1, 0.05)
        out = torch.empty((m, n), dtype=bf16, device=DEV)
        return (lambda: gg.Plan(m, k, n, g, "forward_mxfp8", "e4m3", "bf16"),
                lambda p: gg.rdot_forward_mxfp8(p.handle, x, xs, w, ws, gs, out, p.workspace), out)
    if kind == "mxfp8_dgrad":                       # contracts over the 128 columns of dy
        (dy, ds), (w, ws) = _mx((m, k), 5, 1), _mx((g, n, k), 6, 2, 0.05)
        out = torch.empty((m, n), dtype=bf16, device=DEV)
        return (lambda: gg.Plan(m, n, k, g, "grad_input_mxfp8", "e4m3", "bf16"),
                lambda p: gg.rdot_grad_input_mxfp8(p.handle, dy, ds, w, ws, gs, out, p.workspace), out)
    if kind == "wgrad":                             # contracts over a group's rows: one chunk of 64
        x, dy, out = _bf16((m, k), 7), _bf16((m, n), 8), torch.empty((g, k, n), dtype=f32, device=DEV)
        return (lambda: gg.Plan(m, k, n, g, "grad_weight", "bf16", "f32", flags=gg.RDOT_FLAG_NO_CTA_PAIR),
                lambda p: gg.rdot_grad_weight(p.handle, x, dy, gs, out, p.workspace), out)
    odt = bf16 if kind == "mxfp8_wgrad_bf16" else f32
    rows = lambda width, seed: [t.to(DEV) for t in ri.quantize_mx_e4m3_group_rows(
        torch.from_numpy(ri.host_normal((m, width), seed)), np.array(sizes, np.int32))]
    (x, xs), (dy, ds) = rows(k, 9), rows(n, 10)
    out = torch.empty((g, k, n), dtype=odt, device=DEV)
    return (lambda: gg.Plan(m, k, n, g, "grad_weight_mxfp8", "e4m3", "bf16" if odt is bf16 else "f32"),
            lambda p: gg.rdot_grad_weight_mxfp8(p.handle, x, xs, dy, ds, gs, out, p.workspace), out)


@pytest.mark.parametrize("kind", ["fwd", "fwd_skinny", "mxfp8", "mxfp8_skinny", "mxfp8_dgrad", "wgrad", "mxfp8_wgrad",
                                  "mxfp8_wgrad_bf16"])
def test_loads_land_before_a_stopped_cta_leaves(kind):
    make, call, out = _case(kind)
    stopping, whole = make(), make()
    call(whole)
    assert whole.status() == 0
    want = out.clone()
    gg.rdot_set_wait_timeout(stopping.handle, 1)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)      # twice the L2
    outs, stopped = [], 0
    for _ in range(4):
        cold.zero_()
        call(stopping)
        out.fill_(float("nan"))
        call(whole)
        outs.append(out.clone())
        flags = stopping.status()
        assert flags in (0, gg.RDOT_STATUS_BIT_TIMEOUT)
        stopped += flags != 0
        stopping.clear_status()
    assert whole.status() == 0 and stopped > 0
    for o in outs:
        assert torch.equal(o, want)
