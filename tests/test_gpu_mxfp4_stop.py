"""The MXFP4 kernels stopping early: what a stopped call leaves in flight never reaches a later one.

A plan's wait limit is set so short that waits run out (a stop, no fault), and calls with the default
limit follow at once on the same stream, without a host synchronisation in between: their output must be
that of a call made before any stop, bit for bit.
"""
import pytest
import torch

import group_gemm_gb300 as gg
from tests import _mxfp4 as mx

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
VARIANTS = {"pair": gg.RDOT_FLAG_CTA_PAIR, "skinny": gg.RDOT_FLAG_SKINNY}


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


class Case:
    """A plan for calls that stop, one for calls that do not, and the same operands for both."""

    def __init__(self, m, k, n, sizes, variant, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        byte = lambda *shape: torch.randint(0, 256, shape, generator=g, device=DEV).to(torch.uint8)
        scale = lambda *shape: torch.randint(124, 130, shape, generator=g, device=DEV).to(torch.uint8)
        groups = len(sizes)
        plan = lambda: gg.Plan(m, k, n, groups, "forward_mxfp4", "e2m1", "bf16", flags=VARIANTS[variant])
        self.stopping, self.whole = plan(), plan()
        self.x, self.xs, self.w = byte(m, k // 2), scale(m, k // 32), byte(groups, n, k // 2)
        self.ws = mx.tile_scales(scale(groups, n, k // 32))
        self.sizes = torch.tensor(sizes, dtype=torch.int32, device=DEV)
        self.out = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
        self.want = self.call(self.whole).clone()
        assert self.whole.status() == 0

    def call(self, plan):
        gg.rdot_forward_mxfp4(plan.handle, self.x, self.xs, self.w, self.ws, self.sizes, self.out, plan.workspace)
        return self.out

    def stopped(self):
        """A call that may stop; its output is not looked at."""
        self.call(self.stopping)
        self.out.fill_(float("nan"))

    def check(self, outs):
        torch.cuda.synchronize()
        assert self.whole.status() == 0
        assert self.stopping.status() in (0, gg.RDOT_STATUS_BIT_TIMEOUT)
        for o in outs:
            assert torch.equal(o, self.want)


@pytest.mark.parametrize("limit", [1, 1_000, 5_000])
def test_a_stop_with_scale_stores_issued(limit):
    """The swapped kernel's scale warps write a stage's scales to tensor memory before its weight codes have
    landed: with the weights out of L2 and the scales in it, that is where their wait runs out."""
    c = Case(48, 4096, 1024, [20, 0, 28, 0], "skinny", 1)
    gg.rdot_set_wait_timeout(c.stopping.handle, limit)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)      # twice the L2
    outs = []
    for _ in range(4):
        cold.zero_()
        c.x.clone(), c.xs.clone(), c.ws.clone()
        c.stopped()
        outs.append(c.call(c.whole).clone())
    c.check(outs)


@pytest.mark.parametrize("limit", [1, 1_000])
@pytest.mark.parametrize("variant,m,k,sizes", [("skinny", 48, 1024, [20, 0, 28, 0]),      # 4 of 8 stages
                                               ("skinny", 48, 2048, [20, 0, 28, 0]),      # all 8
                                               ("pair", 700, 1024, [300, 0, 400, 0]),     # 4 of 5, 4 of 10 scale stages
                                               ("pair", 700, 2560, [300, 0, 400, 0])])    # more than 5, 10 of 10
def test_a_stop_after_the_producers_have_finished(variant, m, k, sizes, limit):
    """All of a CTA's loads fit its rings, so the producers end normally while the consumers give up: the
    loads still land before the CTA leaves, not in the shared memory of the next call's CTA."""
    c = Case(m, k, 512, sizes, variant, 2)
    gg.rdot_set_wait_timeout(c.stopping.handle, limit)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)      # twice the L2
    outs = []
    for _ in range(4):
        cold.zero_()
        c.stopped()
        outs.append(c.call(c.whole).clone())
    c.check(outs)


@pytest.mark.parametrize("variant,m,k,sizes", [("skinny", 48, 8192, [20, 0, 28, 0]), ("pair", 700, 8192, [300, 0, 400, 0])])
def test_a_short_limit_takes_effect(variant, m, k, sizes):
    """A nanosecond runs out in every call (the first loads alone take longer) and is reported; the limit's
    default then gives the output of before."""
    c = Case(m, k, 512, sizes, variant, 3)
    gg.rdot_set_wait_timeout(c.stopping.handle, 1)
    for _ in range(4):
        c.stopping.clear_status()
        c.call(c.stopping)
        assert c.stopping.status() == gg.RDOT_STATUS_BIT_TIMEOUT
    gg.rdot_set_wait_timeout(c.stopping.handle, 0)
    c.stopping.clear_status()
    c.out.fill_(float("nan"))
    assert torch.equal(c.call(c.stopping), c.want) and c.stopping.status() == 0
