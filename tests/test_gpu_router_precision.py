"""What moe_router_backward's split operands keep, against 64-bit products of the same inputs.

dx comes from W_g and dlogits in two bf16 parts each: what a pair leaves of a value is at most 2^-18 of it, and the
product of the two second parts, as large, is left out, so a term dl W is off by at most 3 2^-18 of it. The roundings
of different terms are unrelated: over E terms the error is about 2^-18 sqrt(sum (dl W)^2), asserted with a factor of
four in norm. Sums are fp32, 16 products at a time: 3 E / 16 additions of at most 2^-23 of a running sum, which (the
rows of a softmax's gradient sum to zero) stays near sqrt(sum (dl W)^2): 2^-18 of it at the most experts, inside the
same factor. Then one rounding to bf16, 2^-8 of the result."""
import pytest
import torch

from test_gpu_router_backward import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,E", [(600, 256, 40), (700, 384, 128), (600, 256, 129), (700, 1408, 160), (600, 512, 256),
                                   (900, 384, 257), (520, 640, 512)])
@pytest.mark.parametrize("common", [0.0, 10.0, 100.0])
def test_a_row_that_all_experts_share_cancels(T, H, E, common):
    c = Case(T, H, E, False)
    g = torch.Generator(device="cuda").manual_seed(E)
    p = torch.softmax(1.3 * torch.randn(T, E, generator=g, device="cuda"), 1)
    load = torch.rand(E, generator=g, device="cuda") / T
    c.dl = p * (load - (p * load).sum(1, keepdim=True))    # the balance loss's: every row sums to zero
    c.Wg = 0.02 * (torch.randn(E, H, generator=g, device="cuda") + common * torch.randn(H, generator=g, device="cuda"))
    dx = c.run().outputs()[0].double()
    W, dl = c.Wg.double(), c.dl.double()
    want = dl @ W
    terms = ((dl * dl) @ (W * W)).sqrt()
    assert (dx - want).norm() <= 2.0 ** -8 * want.norm() + 2.0 ** -16 * terms.norm()


@pytest.mark.parametrize("wscale,dscale", [(1e36, 1e-5), (1e36, 1e-33), (0.02, 1e-33), (1e-33, 1.0)])
@pytest.mark.parametrize("T,E", [(700, 40), (700, 160), (600, 300)])
def test_sizes_near_the_ends_of_the_type(T, E, wscale, dscale):
    Case(T, 256, E, False, wscale=wscale, dscale=dscale).run().check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,E", [(100, 12), (700, 40), (700, 100), (700, 200), (600, 400)])
def test_a_weight_that_is_not_finite_stays_in_its_column(bad, T, E):
    c = Case(T, 256, E)
    clean = c.run().outputs()
    c.Wg[E - 3, 77] = bad
    dx, dWg, db = c.run().outputs()
    cols = torch.arange(256, device="cuda") != 77
    assert torch.equal(dx[:, cols], clean[0][:, cols]) and not torch.isfinite(dx[:, 77]).any()
    assert torch.equal(dWg, clean[1]) and torch.equal(db, clean[2])
