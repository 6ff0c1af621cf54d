"""CPU checks of the training-side operators: the references against autograd and differences, the error of the
orthogonalisation's roundings, workspace sizes, and every refusal (returned before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

from fp8_grouped_gemm_fp32_b200 import api
from fp8_grouped_gemm_fp32_b200.build import build
from fp8_grouped_gemm_fp32_b200.inputs import CONFIGS
import training_refs as ref

INVALID, SHAPE, SMALL = api.MOE_ERR_INVALID_ARG, api.MOE_ERR_UNSUPPORTED_SHAPE, api.MOE_ERR_WORKSPACE_TOO_SMALL
OKP, ODD = 4096, 4100                        # never dereferenced: the calls return first


@pytest.fixture(scope="module")
def L():
    build()
    return api.lib()


def p(v):
    return ctypes.c_void_p(v) if v else None


def _balance_case(T, E, k, seed):
    r = np.random.default_rng(seed)
    logits = r.normal(size=(T, E))
    idx = np.argsort(-logits, 1)[:, :k]
    return r, logits, idx


def test_balance_reference_gradient_against_autograd_and_differences():
    T, E, k, off = 24, 7, 3, [0, 5, 5, 20, 22]
    r, logits, idx = _balance_case(T, E, k, 3)
    mask = (r.random(T) > 0.2).astype(np.uint8)
    got = ref.balance(logits, idx, mask, off, 0.3, 0.02, k)
    d, mag = ref.balance_grad(got, off, 0.3, 0.02, k, (1.5, -0.5))
    l = torch.tensor(logits, requires_grad=True)
    prob, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
    n, seqs, total = got["valid"][:-2], got["valid"][-2], got["valid"][-1]
    bal = zz = 0.0
    for s in range(len(off) - 1):
        rows = [t for t in range(off[s], off[s + 1]) if mask[t]]
        if rows:
            f = torch.tensor(E * got["counts"][s] / (k * n[s]))
            bal = bal + 0.3 / seqs * (f * prob[rows].mean(0)).sum()
            zz = zz + 0.02 / total * (lse[rows] ** 2).sum()
    (1.5 * bal - 0.5 * zz).backward()
    assert np.allclose(d, l.grad.numpy(), rtol=1e-12, atol=1e-15)
    assert (np.abs(d) <= mag * 1.5 * (1 + 1e-12)).all() and not d[20 + 2:].any()
    # differences, the counts held fixed
    for t, e in ((0, 0), (7, 3), (19, 6), (21, 1)):
        step, vals = 1e-6, []
        for sgn in (1, -1):
            x = logits.copy()
            x[t, e] += sgn * step
            vals.append(ref.balance(x, idx, mask, off, 0.3, 0.02, k, counts=got["counts"])["loss"])
        num = ((vals[0] - vals[1]) / (2 * step)) @ np.array([1.5, -0.5])
        assert abs(num - d[t, e]) < 1e-9


def test_uniform_router_has_loss_alpha():
    T, E, k = 64, 16, 2
    idx = (np.arange(T * k) % E).reshape(T, k)
    got = ref.balance(np.zeros((T, E)), idx, None, [0, T], 0.01, 0.0, k)
    assert abs(got["loss"][0] - 0.01) < 1e-15


@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (300, 1), (5, 7), (64, 64), (100, 260), (260, 100), (257, 513),
                                 (384, 128)])
@pytest.mark.parametrize("kind", ["noise", "low_rank", "decay"])
def test_orthogonalisation_roundings_stay_below_bf16_rounding(M, N, kind):
    # bf16 keeps a value to within 2^-8 of it; the iteration's own roundings add no more than that in norm
    G = ortho_matrix(M, N, kind, 11).to(torch.bfloat16)
    assert ref.rel_norm(ref.orthogonalise_model(G), ref.orthogonalise(G)) <= 2.0 ** -7


@pytest.mark.parametrize("M,N", [(128, 256), (384, 1024), (700, 300)])
@pytest.mark.parametrize("kind", ["noise", "low_rank", "decay", "spikes"])
def test_the_first_two_steps_at_once_add_little(M, N, kind):
    G = ortho_matrix(M, N, kind, 5)
    exact = ref.orthogonalise(G)
    plain, merged = (ref.rel_norm(ref.orthogonalise_model(G, merged=m), exact) for m in (False, True))
    assert merged <= 2.0 ** -8 and merged <= 1.5 * plain + 2.0 ** -11


def ortho_matrix(M, N, kind, seed):
    g = torch.Generator().manual_seed(seed + 1000 * M + N)
    if kind == "spikes":
        u = torch.linalg.qr(torch.randn(M, 4, generator=g))[0]
        v = torch.linalg.qr(torch.randn(N, 4, generator=g))[0]
        return 30 * u @ v.t() + torch.randn(M, N, generator=g) / (M ** 0.5 + N ** 0.5)
    if kind == "noise":
        return torch.randn(M, N, generator=g)
    r = min(M, N, 8) if kind == "low_rank" else min(M, N)
    s = torch.ones(r) if kind == "low_rank" else torch.arange(1, r + 1).float() ** -1.0
    return (torch.randn(M, r, generator=g) * s) @ torch.randn(r, N, generator=g) + 1e-3 * torch.randn(M, N, generator=g)


def test_workspace_sizes(L):
    assert api.moe_balance_workspace_size(8192, 256, 1) > 0
    assert api.moe_balance_workspace_size(0, 8, 1) > 0
    for bad in ((-1, 8, 1), ((1 << 30) + 1, 8, 1), (8, 0, 1), (8, 513, 1), (8, 8, 0), (8, 8, 65536)):
        assert api.moe_balance_workspace_size(*bad) == 0
    assert api.moe_router_backward_workspace_size(8192, 7168, 256) > 0
    for bad in ((-1, 128, 8), (8, 100, 8), (8, 128, 513), (8, 16512, 8), (1 << 24, 128, 8), (8, 0, 8), (8, 128, 0)):
        assert api.moe_router_backward_workspace_size(*bad) == 0
    assert api.moe_orthogonalise_workspace_size(2, 256, 512, True) > 0
    # a large batch runs in waves: its workspace stops growing
    assert api.moe_orthogonalise_workspace_size(4096, 2048, 4096) == api.moe_orthogonalise_workspace_size(8192, 2048, 4096)
    for bad in ((-1, 8, 8, 0), (2, 0, 8, 0), (2, 8, 0, 0), (2, 16385, 8, 0), (2, 8, 16385, 0), (2, 100, 8, 1), (0, 8, 8, 0)):
        assert api.moe_orthogonalise_workspace_size(*bad) == 0


def test_train_logits_offset(L):
    c = api.Config.from_moe(CONFIGS["prefill"])
    off = L.moe_train_logits_offset(ctypes.byref(c))
    assert off > 0 and off % 256 == 0
    assert off + 4 * c.T * c.E <= api.moe_workspace_size(c, 2)
    for name in ("decode", "decode_hash", "decode_w4"):
        bad = api.Config.from_moe(CONFIGS[name])
        assert L.moe_train_logits_offset(ctypes.byref(bad)) == 0
        with pytest.raises(ValueError):
            api.moe_train_logits(bad, torch.empty(16, dtype=torch.uint8))


BAL = dict(T=64, E=8, k=2, logits=OKP, idx=OKP, mask=0, off=0, S=1, alpha=0.01, beta=0.0, loss=OKP, counts=OKP, mp=OKP,
           lse=OKP, valid=OKP, ws=OKP, nbytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(S=0), INVALID), (dict(k=9), INVALID),
    (dict(E=513, k=2), SHAPE), (dict(E=64, k=33), SHAPE), (dict(S=65536, off=OKP), SHAPE), (dict(S=2), INVALID),
    (dict(T=1 << 30), SHAPE), (dict(T=(1 << 30) + 1, E=8, k=1), SHAPE), (dict(alpha=float("nan")), INVALID), (dict(beta=float("inf")), INVALID),
    (dict(logits=0), INVALID), (dict(logits=ODD), INVALID), (dict(idx=0), INVALID), (dict(mask=ODD), INVALID),
    (dict(off=ODD), INVALID), (dict(loss=0), INVALID), (dict(counts=ODD), INVALID), (dict(mp=0), INVALID),
    (dict(lse=0), INVALID), (dict(valid=0), INVALID), (dict(ws=0), INVALID), (dict(nbytes=16), SMALL)])
def test_balance_loss_refusals(L, change, code):
    a = dict(BAL, **change)
    assert L.moe_balance_loss(a["T"], a["E"], a["k"], p(a["logits"]), p(a["idx"]), p(a["mask"]), p(a["off"]), a["S"],
                              a["alpha"], a["beta"], p(a["loss"]), p(a["counts"]), p(a["mp"]), p(a["lse"]),
                              p(a["valid"]), p(a["ws"]), a["nbytes"], None) == code


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(E=513), SHAPE), (dict(S=2), INVALID), (dict(beta=float("nan")), INVALID),
    (dict(logits=0), INVALID), (dict(lse=0), INVALID), (dict(counts=0), INVALID), (dict(valid=ODD), INVALID),
    (dict(dloss=ODD), INVALID), (dict(dlogits=0), INVALID), (dict(dlogits=ODD), INVALID)])
def test_balance_loss_backward_refusals(L, change, code):
    a = dict(BAL, dloss=0, dlogits=OKP, **{})
    a.update(change)
    assert L.moe_balance_loss_backward(a["T"], a["E"], a["k"], p(a["logits"]), p(a["lse"]), p(a["counts"]),
                                       p(a["valid"]), p(a["mask"]), p(a["off"]), a["S"], a["alpha"], a["beta"],
                                       p(a["dloss"]), p(a["dlogits"]), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(E=0), INVALID), (dict(H=200), SHAPE), (dict(H=16512), SHAPE),
    (dict(E=513), SHAPE), (dict(T=1 << 24), SHAPE), (dict(x=0), INVALID), (dict(x=ODD), INVALID), (dict(Wg=0), INVALID),
    (dict(dl=0), INVALID), (dict(dx0=ODD), INVALID), (dict(dWg0=ODD), INVALID), (dict(db0=ODD), INVALID),
    (dict(dx=0), INVALID), (dict(dWg=0), INVALID), (dict(db=ODD), INVALID), (dict(ws=0), INVALID),
    (dict(ws=OKP + 16), INVALID), (dict(nbytes=64), SMALL)])
def test_router_backward_refusals(L, change, code):
    a = dict(T=64, H=256, E=8, x=OKP, Wg=OKP, dl=OKP, dx0=0, dWg0=0, db0=0, dx=OKP, dWg=OKP, db=OKP, ws=OKP,
             nbytes=1 << 30)
    a.update(change)
    assert L.moe_router_backward(a["T"], a["H"], a["E"], p(a["x"]), p(a["Wg"]), p(a["dl"]), p(a["dx0"]), p(a["dWg0"]),
                                 p(a["db0"]), p(a["dx"]), p(a["dWg"]), p(a["db"]), p(a["ws"]), a["nbytes"],
                                 None) == code


@pytest.mark.parametrize("change,code", [
    (dict(batch=-1), INVALID), (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(inter=2), INVALID),
    (dict(M=16385), SHAPE), (dict(N=16385), SHAPE), (dict(batch=16385), SHAPE), (dict(inter=1, M=100), SHAPE),
    (dict(type=2), INVALID), (dict(steps=0), INVALID), (dict(steps=33), INVALID), (dict(a=float("nan")), INVALID),
    (dict(a=20.0), INVALID),                   # singular values up to 20: past what fp16 X is scaled for
    (dict(a=2.0, b=0.0, c=0.0), INVALID),      # doubles every step
    (dict(b=-300.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(G=0), INVALID), (dict(G=ODD), INVALID), (dict(O=0), INVALID),
    (dict(ws=OKP + 16), INVALID), (dict(nbytes=64), SMALL), (dict(batch=0, G=0), api.MOE_OK)])
def test_orthogonalise_refusals(L, change, code):
    a = dict(batch=2, M=128, N=64, inter=0, G=OKP, type=0, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, scale=1.0,
             O=OKP, ws=OKP, nbytes=1 << 30)
    a.update(change)
    assert L.moe_orthogonalise(a["batch"], a["M"], a["N"], a["inter"], p(a["G"]), a["type"], a["steps"], a["a"], a["b"],
                               a["c"], a["eps"], a["scale"], p(a["O"]), p(a["ws"]), a["nbytes"], None) == code


def test_binding_refuses_host_and_strided_tensors(L):
    t = torch.zeros(8, 8)
    with pytest.raises(ValueError):
        api.moe_orthogonalise(1, 8, 8, False, t, 5, *ref.ORTHO, 1e-7, 1.0, t, t)
    with pytest.raises(ValueError):
        api.moe_orthogonalise(1, 8, 8, False, t.half(), 5, *ref.ORTHO, 1e-7, 1.0, t, t)
    with pytest.raises(ValueError):
        api.moe_balance_loss(8, 8, 1, t, t, None, None, 1, 0.1, 0.0, t, t, t, t, t, t)
    with pytest.raises(ValueError):
        api.moe_router_backward(8, 128, 8, t, t, t, None, None, None, t, t, t, t)


@pytest.mark.parametrize("M,N,inter", [(520, 520, False), (100, 1000, False), (128, 5000, True), (1000, 100, False), (60, 70, False),
                                       (256, 512, True), (300, 129, False), (2048, 4096, False), (16384, 100, False),
                                       (128, 16384, True)])
def test_orthogonalise_workspace_of_a_batch_serves_every_smaller_one(L, M, N, inter):
    sizes = [api.moe_orthogonalise_workspace_size(b, M, N, inter) for b in range(1, 400)]
    assert sizes == sorted(sizes)


def test_orthogonalise_takes_the_workspace_of_a_larger_batch(L):
    # Refused before any device work where the workspace is too small: a batch that fits goes on, and this machine has no
    # device to go on to.
    call = lambda batch, M, N, nbytes: L.moe_orthogonalise(batch, M, N, 0, p(OKP), 0, 5, *ref.ORTHO, 1e-7, 1.0, p(OKP), p(OKP),
                                                           nbytes, None)
    if torch.cuda.is_available():
        pytest.skip("would launch")
    for M, N in ((520, 520), (100, 1000)):
        for large in (19, 26, 30):
            n = api.moe_orthogonalise_workspace_size(large, M, N)
            assert all(call(b, M, N, n) not in (SMALL, api.MOE_OK) for b in range(1, large + 1))
    assert call(2, 520, 520, 4096) == SMALL


@pytest.mark.parametrize("E", [8, 60, 256, 512])
def test_balance_workspace_of_a_size_serves_every_smaller_one(L, E):
    size = api.moe_balance_workspace_size
    for S in (1, 16, 17, 100):
        got = [size(T, E, S) for T in range(0, 12000, 7)]
        assert got == sorted(got)
    for T in (64, 4736, 4737, 9000):
        got = [size(T, E, S) for S in range(1, 200)]
        assert got == sorted(got)


@pytest.mark.parametrize("H,E", [(128, 8), (1408, 100), (2048, 160), (512, 512)])
def test_router_workspace_of_a_count_of_tokens_serves_every_smaller_one(L, H, E):
    got = [api.moe_router_backward_workspace_size(T, H, E) for T in range(0, 3000)]
    assert got == sorted(got)


def _binding_calls():
    """Calls of the bindings with host tensors of the right types and sizes, by operator: name -> (call, tensors)."""
    T, E, k, S, H = 12, 8, 2, 3, 128
    f = lambda *s: torch.zeros(*s)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    b = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    fwd = dict(logits=f(T, E), topk_idx=i(T, k), token_mask=b(T), seq_offsets=i(S + 1), loss=f(2), counts=i(S, E),
               mean_prob=f(S, E), lse=f(T), seq_valid=i(S + 2), ws=b(1 << 20))
    bwd = dict(logits=f(T, E), lse=f(T), counts=i(S, E), seq_valid=i(S + 2), token_mask=b(T), seq_offsets=i(S + 1),
               dloss=f(2), dlogits=f(T, E))
    rb = dict(x=h(T, H), Wg=f(E, H), dlogits=f(T, E), dx0=h(T, H), dWg0=f(E, H), db0=f(E), dx=h(T, H), dWg=f(E, H), db=f(E),
              ws=b(1 << 20))
    ortho = dict(G=f(2, 2 * H, 16), O=h(2, 2 * H, 16), ws=b(1 << 20))
    return {
        "balance": (lambda a: api.moe_balance_loss(T=T, E=E, k=k, S=S, alpha=0.1, beta=0.0, **a), fwd),
        "balance_backward": (lambda a: api.moe_balance_loss_backward(T=T, E=E, k=k, S=S, alpha=0.1, beta=0.0, **a), bwd),
        "router": (lambda a: api.moe_router_backward(T=T, H=H, E=E, **a), rb),
        "ortho": (lambda a: api.moe_orthogonalise(2, H, 16, True, a["G"], 5, *ref.ORTHO, 1e-7, 1.0, a["O"], a["ws"]), ortho)}


@pytest.mark.parametrize("op", ["balance", "balance_backward", "router", "ortho"])
def test_binding_refuses_other_types_and_smaller_tensors(L, op):
    call, good = _binding_calls()[op]
    with pytest.raises(ValueError, match="CUDA tensors"):                  # all else is right
        call(good)
    for name, t in good.items():
        if name != "ws":                                                   # (the library is given its size)
            other = torch.int64 if t.dtype in (torch.int32, torch.uint8) else torch.float16
            with pytest.raises(ValueError, match=name):
                call(dict(good, **{name: t.to(other)}))
            with pytest.raises(ValueError, match=name):
                call(dict(good, **{name: t.view(-1)[:-1].contiguous()}))
            with pytest.raises(ValueError, match="CUDA tensors"):          # a larger one will do
                call(dict(good, **{name: torch.cat([t.view(-1), t.view(-1)])}))
    if "token_mask" in good:
        with pytest.raises(ValueError, match="CUDA tensors"):
            call(dict(good, token_mask=good["token_mask"].bool()))


@pytest.mark.parametrize("M,N,merged", [(128, 700, False), (300, 200, False), (512, 1024, True)])
@pytest.mark.parametrize("r", [1, 8])
@pytest.mark.parametrize("steps", [8, 10, 12])
def test_noise_outside_a_low_rank_stays_at_what_22_bits_of_x_leave(M, N, merged, r, steps):
    # Each value of X is off by at most 2^-22 of it; in the directions G lacks a^steps multiplies that. As much comes from the
    # products: B, rounded by at most 2^-11 of it, times what the first fp16 value lacks of X, at most 2^-11 of that, and |B|
    # is below a (the first two steps at once: Q in its place, below a^2, of growth a^2). 2^-21 in all. The bounds are reached
    # only where roundings line up (few distinct values, as here), the average is a quarter, which leaves room for the noise
    # of later steps and for singular values that end at 0.7.
    G = ref.low_rank(M, N, r)
    exact = ref.orthogonalise(G, steps)
    err = lambda spare: ref.rel_norm(ref.orthogonalise_model(G, steps, merged=merged, spare=spare), exact)
    assert err(5) <= 2.0 ** -21 * ref.ORTHO[0] ** steps / r ** 0.5 + 2.0 ** -8
    assert steps < 10 or err(5) < err(0)
