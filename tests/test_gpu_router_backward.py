"""moe_router_backward on the GPU against 64-bit products of the same inputs.

Tolerances. dx: room for operands of 11 bits, (2^-10 + E 2^-23) sum |dl||W| + 2^-33 E max|dl W|, then one rounding to
bf16, 2^-8 of the result. (W_g and dlogits in bf16 pairs, and for few tokens fp32, lie well inside that; what the pairs
keep is tested in test_gpu_router_precision.) dWg: dlogits in three
bf16 parts loses at most 2^-25; sums of 16 products at a time, 128 tokens x 3 parts = 24 additions of at most 2^-23
before promotion, then one fp32 addition per 128 tokens and per partial tile: (64 + T / 128 + 160) 2^-24 sum |dl||x|.
db: at most 4 additions a lane, 8 warps, then 64 bits: 16 2^-24 sum |dl|. Bases add one rounding."""
import numpy as np
import pytest
import torch

from fp8_grouped_gemm_fp32_b200 import api
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Case:
    def __init__(self, T, H, E, base=True, seed=0, wscale=0.02, dscale=1e-5):
        ensure_lib()
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + 7 * H + E)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.T, self.H, self.E = T, H, E
        self.x = rn(T, H).to(torch.bfloat16)
        self.Wg = wscale * rn(E, H)
        self.dl = dscale * rn(T, E) * torch.rand(T, 1, generator=g, device="cuda")
        self.dx0 = (dscale * wscale * rn(T, H)).to(torch.bfloat16) if base else None
        self.dWg0 = dscale * rn(E, H) if base else None
        self.db0 = dscale * rn(E) if base else None
        self.dx = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
        self.dWg = torch.full((E, H), 7.0, device="cuda")
        self.db = torch.full((E,), 7.0, device="cuda")
        self.ws = torch.full((api.moe_router_backward_workspace_size(T, H, E),), 0x5a, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        api.moe_router_backward(self.T, self.H, self.E, self.x, self.Wg, self.dl, self.dx0, self.dWg0, self.db0, self.dx,
                                self.dWg, self.db, self.ws, stream)
        return self

    def outputs(self):
        torch.cuda.synchronize()
        assert api.moe_get_device_status() == api.MOE_OK
        return [t.clone() for t in (self.dx, self.dWg, self.db)]

    def check(self):
        dx, dWg, db = (t.double() for t in self.outputs())
        x, W, dl = self.x.double(), self.Wg.double(), self.dl.double()
        z = lambda t: 0.0 if t is None else t.double()
        want = dl @ W + z(self.dx0)
        mag = dl.abs() @ W.abs()
        top = (dl.abs() * W.abs().amax(1)).amax(1, keepdim=True)
        tol = (2.0 ** -10 + self.E * 2.0 ** -23) * mag + 2.0 ** -33 * self.E * top
        assert ((dx - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
        want = dl.t() @ x + z(self.dWg0)
        tol = (64 + self.T / 128 + 160) * U * (dl.abs().t() @ x.abs()) + U * want.abs()
        assert ((dWg - want).abs() <= tol).all()
        want = dl.sum(0) + z(self.db0)
        assert ((db - want).abs() <= 16 * U * dl.abs().sum(0) + U * want.abs()).all()


@pytest.mark.parametrize("T,H,E", [(1, 128, 1), (2, 128, 8), (63, 256, 3), (64, 512, 16), (129, 384, 100), (200, 1408, 128),
                                   (257, 1408, 129), (130, 640, 200), (300, 256, 256), (257, 512, 257), (100, 384, 511),
                                   (140, 256, 512), (1000, 128, 64), (3000, 1024, 60), (2049, 2048, 160),
                                   (600, 128, 1), (700, 256, 9), (1025, 384, 16), (900, 256, 17), (640, 512, 32), (777, 128, 33),
                                   (1030, 1408, 65), (520, 256, 128), (515, 128, 129), (5000, 128, 8)])
@pytest.mark.parametrize("base", [False, True])
def test_matches_the_products(T, H, E, base):
    Case(T, H, E, base).run().check()


@pytest.mark.parametrize("wscale,dscale", [(1e-12, 1e-12), (1e12, 1e6), (0.02, 1e-25)])
@pytest.mark.parametrize("T,E", [(150, 24), (600, 24), (150, 160)])
def test_far_scales(T, E, wscale, dscale):
    Case(T, 256, E, False, wscale=wscale, dscale=dscale).run().check()


@pytest.mark.parametrize("T,E", [(200, 40), (600, 40), (200, 140)])
def test_experts_and_tokens_of_very_different_sizes(T, E):
    c = Case(T, 256, E)
    c.Wg *= 10.0 ** torch.linspace(-8, 8, E, device="cuda")[:, None]
    c.dl *= 10.0 ** torch.linspace(-10, 2, T, device="cuda")[:, None]
    c.Wg[5] = 0.0
    c.dl[17] = 0.0
    c.run().check()
    assert torch.equal(c.dx[17], c.dx0[17])


def test_no_tokens_gives_the_bases():
    c = Case(0, 256, 12)
    c.run()
    _, dWg, db = c.outputs()
    assert torch.equal(dWg, c.dWg0) and torch.equal(db, c.db0)
    c = Case(0, 256, 12, False)
    c.run()
    _, dWg, db = c.outputs()
    assert not dWg.any() and not db.any()


@pytest.mark.parametrize("E", [5, 30, 64, 100, 150, 300])
def test_in_place_equals_out_of_place_and_results_repeat(E):
    c = Case(700, 768, E)
    want = c.run().outputs()
    assert all(torch.equal(x, y) for x, y in zip(want, c.run().outputs()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.dx, c.dWg, c.db = c.dx0, c.dWg0, c.db0
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, c.run(s).outputs()))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,E", [(300, 40), (700, 12), (700, 40), (700, 100), (700, 200)])
def test_values_that_are_not_finite_stay_where_the_formula_puts_them(bad, T, E):
    c = Case(T, 256, E)
    clean = c.run().outputs()
    c.dl[123, 7] = bad
    dx, dWg, db = c.run().outputs()
    rows, cols = torch.arange(T, device="cuda") != 123, torch.arange(E, device="cuda") != 7
    assert torch.equal(dx[rows], clean[0][rows]) and not torch.isfinite(dx[123]).any()
    assert torch.equal(dWg[cols], clean[1][cols]) and not torch.isfinite(dWg[7]).any()
    assert torch.equal(db[cols], clean[2][cols]) and not torch.isfinite(db[7])


def test_captured_and_replayed_on_new_inputs():
    for T, E in ((400, 40), (1000, 40), (400, 200)):
        c = Case(T, 256, E)
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            c.run()
        for k in range(2):
            c.dl.copy_(1e-4 * torch.randn(T, E, device="cuda"))
            c.Wg.mul_(1.5)
            torch.cuda.synchronize()
            g.replay()
            c.check()


def test_gradient_against_differences():
    # L = <y, x W^T + b> is linear in each of x, W, b, so differences of the 64-bit L are exact up to rounding
    c = Case(40, 128, 9, False, wscale=0.1, dscale=0.3)
    dx, dWg, db = (t.double() for t in c.run().outputs())
    loss = lambda x, W, b: float((c.dl.double() * (x @ W.t() + b)).sum())
    x, W, b = c.x.double(), c.Wg.double(), torch.zeros(9, dtype=torch.float64, device="cuda")
    for i, j in ((0, 0), (7, 100), (39, 127)):
        d = torch.zeros_like(x)
        d[i, j] = 0.5
        want = loss(x + d, W, b) - loss(x - d, W, b)
        assert abs(want - float(dx[i, j])) <= 2.0 ** -7 * float((c.dl[i].abs().double() @ W[:, j].abs()))
    for e, h in ((0, 0), (8, 127), (3, 64)):
        d = torch.zeros_like(W)
        d[e, h] = 0.5
        want = loss(x, W + d, b) - loss(x, W - d, b)
        assert abs(want - float(dWg[e, h])) <= 256 * U * float((c.dl[:, e].abs().double() @ x[:, h].abs())) + 1e-9
        d = torch.zeros_like(b)
        d[e] = 0.5
        assert abs(loss(x, W, b + d) - loss(x, W, b - d) - float(db[e])) <= 16 * U * float(c.dl[:, e].abs().sum()) + 1e-9


@pytest.mark.parametrize("T,E", [(300, 16), (900, 70), (900, 140)])
def test_two_at_once_and_captured_behind_a_memset_and_a_copy(T, E):
    cases = [Case(T, 640, E), Case(T + 31, 640, E)]
    want = [[t.clone() for t in c.run().outputs()] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):                                     # each on its own stream, with its own workspace
        for c, s in zip(cases, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert all(torch.equal(x, y) for x, y in zip(w, c.outputs()))
    c, src, s = cases[0], cases[0].dl.clone(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.ws.zero_()
        c.dl.copy_(src)
        c.run()
    c.dl.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want[0], c.outputs()))
