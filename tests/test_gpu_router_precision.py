"""What moe_router_backward's split operands keep, against 64-bit products of the same inputs.

dx comes from W_g and dlogits in two bf16 parts each. Half a step of bf16 is 2^-8: what a pair leaves of a value is at
most 2^-16 of it, and the product of the two second parts, as large, is left out, so a term dl W is off by at most
3 2^-16 of it. Roundings are spread over their steps: each of the three is 2^-18.8 on average (root mean square), and those of
different terms are unrelated: over E terms the error is about 2^-18 sqrt(sum (dl W)^2), asserted with a factor of four in
norm. Sums are fp32, 16 products at a time: 3 E / 16 additions of at most 2^-23 of a running sum, which (the
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


@pytest.mark.parametrize("T,H,E", [(1030, 384, 8), (700, 256, 30), (1030, 256, 60), (700, 384, 100), (1030, 384, 200), (700, 256, 400)])
def test_the_third_part_of_dlogits_reaches_dWg(T, H, E):
    # Tokens in pairs that cancel down to their third part: dlogits +-(1 + 2^-9 + c 2^-20), parts 1, 2^-9 and c 2^-20, x one
    # of 1, -1, 2 for both. Every sum is a multiple of 2^-20 below 2^4, which fp32 and the tensor cores hold exactly.
    c = Case(T, H, E, False)
    g = torch.Generator(device="cuda").manual_seed(E)
    third = torch.randint(1, 8, (T, E), generator=g, device="cuda").float() * 2.0 ** -20
    sign = torch.tensor([1.0, -1.0], device="cuda").repeat(T // 2)[:, None]
    c.dl = sign * (1 + 2.0 ** -9 + third)
    half = torch.randint(0, 3, (T // 2, H), generator=g, device="cuda")
    c.x = torch.tensor([1.0, -1.0, 2.0], device="cuda", dtype=torch.bfloat16)[half].repeat_interleave(2, 0).contiguous()
    dWg = c.run().outputs()[1]
    want = c.dl.double().t() @ c.x.double()
    assert torch.count_nonzero(want) > 0.9 * E * H
    assert torch.equal(dWg.double(), want)


@pytest.mark.parametrize("T,H,E", [(100, 256, 8), (700, 256, 8), (700, 384, 40), (900, 1408, 100), (600, 512, 129), (700, 1408, 256),
                                   (900, 384, 300), (520, 640, 512)])
def test_dx_beside_a_base_that_nearly_cancels_it(T, H, E):
    # dx0 = -bf16(dlogits W_g): what is left is 2^-9 of it, and rounding that to bf16 hides nothing of the products' own
    # error, 3 2^-16 of each term and an fp32 addition for every 16 of three products' terms.
    c = Case(T, H, E, True)
    product = c.dl.double() @ c.Wg.double()
    c.dx0 = (-product).to(torch.bfloat16)
    dx = c.run().outputs()[0].double()
    mag = c.dl.double().abs() @ c.Wg.double().abs()
    tol = (3 * 2.0 ** -16 + 3 * E / 16 * 2.0 ** -23 + 2.0 ** -23) * mag
    want = product + c.dx0.double()
    assert ((dx - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()


@pytest.mark.parametrize("T,H,E", [(600, 16384, 512), (600, 16384, 64), (520, 16384, 200), (5000, 1024, 300), (9000, 384, 129),
                                   (4100, 2048, 448)])
@pytest.mark.parametrize("base", [False, True])
def test_the_most_columns_and_many_units(T, H, E, base):
    Case(T, H, E, base).run().check()
