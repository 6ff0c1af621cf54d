"""moe_balance_loss and its gradient on the GPU against the 64-bit reference.

Tolerances, u = 2^-24 (half a step of fp32). A probability is exp of a difference of logits of size a = max|l|: the
difference is off by at most u a, the exponential by a few u, sum and quotient by a few more: (2 a + 16) u relative.
mean_prob adds at most 64 such values in one chain, 32 chains, then in 64 bits: + 96 u relative. lse: (2 a + 16) u
absolute. dlogits: the same (2 a + 16) u on each factor of terms whose sizes the reference gives, with E-term sums
in a lane of 16 and 5 shuffles: (4 a + 64) u of that size."""
import numpy as np
import pytest
import torch

from fp8_grouped_gemm_fp32_b200 import api
from gpu_helpers import ensure_lib, to_np
import training_refs as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Case:
    def __init__(self, T, E, k, off=None, mask=None, seed=0, logits=None, alpha=0.02, beta=1e-3):
        ensure_lib()
        r = np.random.default_rng(seed + 7 * T + E)
        self.T, self.E, self.k, self.alpha, self.beta = T, E, k, alpha, beta
        self.off = [0, T] if off is None else list(off)
        self.S = len(self.off) - 1
        self.logits = (1.5 * r.normal(size=(T, E)) + r.normal(size=E)).astype(np.float32) if logits is None else logits
        self.idx = np.argsort(-np.nan_to_num(self.logits), 1)[:, :k].astype(np.int32)
        self.mask = mask
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.d_logits, self.d_idx, self.d_mask = dev(self.logits), dev(self.idx), dev(mask)
        self.d_off = None if off is None else dev(np.asarray(off, np.int32))
        new = lambda *s, dt=torch.float32, v=7: torch.full(s, v, dtype=dt, device="cuda")
        self.loss, self.counts, self.mp = new(2), new(self.S, E, dt=torch.int32), new(self.S, E)
        self.lse, self.valid, self.dl = new(T), new(self.S + 2, dt=torch.int32), new(T, E)
        self.ws = new(api.moe_balance_workspace_size(T, E, self.S), dt=torch.uint8, v=0x5a)

    def forward(self, stream=None):
        api.moe_balance_loss(self.T, self.E, self.k, self.d_logits, self.d_idx, self.d_mask, self.d_off, self.S,
                             self.alpha, self.beta, self.loss, self.counts, self.mp, self.lse, self.valid, self.ws,
                             stream)
        return self

    def backward(self, dloss=None, stream=None):
        api.moe_balance_loss_backward(self.T, self.E, self.k, self.d_logits, self.lse, self.counts, self.valid,
                                      self.d_mask, self.d_off, self.S, self.alpha, self.beta, dloss, self.dl, stream)
        return self

    def results(self):
        torch.cuda.synchronize()
        return [to_np(t).copy() for t in (self.loss, self.counts, self.mp, self.lse, self.valid, self.dl)]

    def check(self, g=(1.0, 1.0), status=api.MOE_OK):
        loss, counts, mp, lse, valid, dl = self.results()
        assert api.moe_get_device_status() == status
        want = ref.balance(self.logits, self.idx, self.mask, self.off, self.alpha, self.beta, self.k)
        live = want["live"]
        inside = np.zeros(self.T, bool)
        inside[self.off[0]:self.off[-1]] = True
        a = float(np.abs(self.logits[live]).max()) if live.any() else 0.0
        pt = (2 * a + 16) * U
        assert np.array_equal(counts, want["counts"]) and np.array_equal(valid, want["valid"])
        assert (np.abs(mp - want["mean_prob"]) <= (pt + 96 * U) * want["mean_prob"]).all()
        assert np.abs(loss[0] - want["loss"][0]) <= (pt + 96 * U) * abs(want["loss"][0]) + 1e-37
        assert np.abs(loss[1] - want["loss"][1]) <= (2 * pt + 96 * U) * self.beta * (np.abs(want["lse"][live]).max(initial=0) + 1) ** 2
        assert (np.abs(lse[live] - want["lse"][live]) <= pt + U * np.abs(want["lse"][live])).all()
        assert (lse[inside & ~live] == 0).all() and (lse[~inside] == 7).all()
        d, mag = ref.balance_grad(want, self.off, self.alpha, self.beta, self.k, g)
        assert (np.abs(dl - d)[inside] <= (4 * a + 64) * U * mag[inside]).all()
        assert (dl[inside & ~live] == 0).all() and (dl[~inside] == 7).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (2, 7, 3), (63, 64, 2), (129, 65, 4), (300, 256, 8), (257, 257, 1),
                                   (513, 512, 32), (1000, 4, 2), (2500, 30, 3), (5000, 128, 8), (16, 200, 9), (17, 16, 2), (128, 256, 8),
                                   (129, 511, 31), (500, 90, 5), (512, 512, 8)])
def test_one_sequence(T, E, k):
    Case(T, E, k).forward().backward().check()


@pytest.mark.parametrize("E", [8, 60, 61, 100, 256, 300, 511])
@pytest.mark.parametrize("T", [250, 1500])
def test_ragged_masked_sequences_with_rows_behind_the_last(E, T):
    r = np.random.default_rng(E)
    cuts = np.sort(r.integers(3, T - 40, 40))
    off = [3, 3, *cuts, cuts[-1], cuts[-1] + 1]           # empty ones, a sequence of one token, rows left and right
    mask = (r.random(T) > 0.3).astype(np.uint8)
    mask[off[10]:off[12]] = 0                              # sequences that the mask empties
    c = Case(T, E, min(4, E), off, mask)
    c.forward().backward(torch.tensor([0.5, -2.0], device="cuda")).check((0.5, -2.0))


@pytest.mark.parametrize("T", [250, 700])
def test_every_token_its_own_sequence(T):
    Case(T, 16, 2, off=list(range(T + 1))).forward().backward().check()


def test_no_valid_token_and_no_token():
    c = Case(40, 8, 2, mask=np.zeros(40, np.uint8))
    c.forward().backward().check()
    assert (to_np(c.loss) == 0).all()
    c = Case(0, 8, 2)
    c.forward().backward()
    loss, counts, mp, lse, valid, dl = c.results()
    assert not loss.any() and not counts.any() and not mp.any() and not valid.any()
    c = Case(20, 8, 2, off=[5, 5, 5])
    c.forward().backward().check()


@pytest.mark.parametrize("T", [200, 900])
def test_masked_rows_may_hold_anything_and_minus_infinity_is_a_zero_probability(T):
    E = 40
    r = np.random.default_rng(5)
    logits = r.normal(size=(T, E)).astype(np.float32)
    mask = np.ones(T, np.uint8)
    for t, v in ((3, np.nan), (50, np.inf), (199, -np.inf)):
        mask[t] = 0
        logits[t] = v
    logits[:, 7] = -np.inf                                 # an expert that nothing may reach
    logits[10, :39] = -np.inf                              # a row with one finite logit
    logits[11] = np.where(np.isfinite(logits[11]), -3.0e38, logits[11])     # near the type's lowest value
    logits[11, :3] = 0.0
    c = Case(T, E, 3, mask=mask, logits=logits)
    c.alpha, c.beta = 0.02, 0.0
    c.forward().backward()
    loss, counts, mp, lse, valid, dl = c.results()
    want = ref.balance(logits, c.idx, mask, [0, T], 0.02, 0.0, 3)
    assert np.isfinite(loss).all() and np.isfinite(dl).all()
    assert (mp[:, 7] == 0).all() and (dl[:, 7] == 0).all()
    assert np.allclose(mp, want["mean_prob"], rtol=200 * U, atol=0) and np.allclose(loss[0], want["loss"][0], rtol=200 * U)
    assert (dl[[3, 50, 199]] == 0).all()


def test_an_undefined_row_stays_in_its_sequence():
    T, E = 90, 12
    logits = np.random.default_rng(1).normal(size=(T, E)).astype(np.float32)
    logits[40] = -np.inf                                   # valid, yet no finite logit
    logits[70, 3] = np.nan
    c = Case(T, E, 2, off=[0, 30, 60, 90], logits=logits)
    c.forward().backward()
    loss, counts, mp, lse, valid, dl = c.results()
    assert np.isnan(loss).all()
    assert np.isfinite(mp[0]).all() and np.isnan(mp[1]).all() and np.isnan(mp[2]).all()
    assert np.isfinite(np.delete(dl, [40, 70], 0)).all() and np.isnan(dl[40]).all() and np.isnan(dl[70]).all()


@pytest.mark.parametrize("T", [100, 800])
def test_slots_outside_the_experts_count_nowhere(T):
    c = Case(T, 8, 4)
    c.idx[::3, 1] = -1
    c.idx[1::3, 2] = 8
    c.idx[2::3, 0] = 2 ** 31 - 1
    c.d_idx.copy_(torch.from_numpy(c.idx))
    c.forward().backward().check()


@pytest.mark.parametrize("off", [[0, 50, 40, 90], [-5, 50, 60, 90], [0, 50, 60, 1000], [90, 50, 20, 0]])
@pytest.mark.parametrize("T", [90, 400])
def test_bad_offsets_are_reported_and_stay_in_bounds(off, T):
    c = Case(T, 16, 2, off=[0, 30, 60, T])
    c.d_off.copy_(torch.tensor(off, dtype=torch.int32))
    c.forward().backward()
    torch.cuda.synchronize()
    assert api.moe_get_device_status() == api.MOE_ERR_CAPACITY


@pytest.mark.parametrize("T", [200, 4000])
def test_results_repeat_bit_for_bit_and_on_another_stream(T):
    c = Case(T, 100, 6, off=[0, 100, T // 2 + 50, T - 1])
    first = c.forward().backward().results()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (None, s):
        for t in (c.loss, c.mp, c.dl[:T - 1]):
            t.fill_(7)
        torch.cuda.synchronize()
        again = c.forward(st).backward(stream=st).results()
        for x, y in zip(first, again):
            assert np.array_equal(x, y)


@pytest.mark.parametrize("T", [240, 3000])
def test_captured_and_replayed_on_new_inputs(T):
    c = Case(T, 64, 2, off=[0, 100, T])
    s = torch.cuda.Stream()
    c.forward().backward()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.forward().backward()
    r = np.random.default_rng(9)
    for _ in range(2):
        c.logits = r.normal(size=c.logits.shape).astype(np.float32)
        c.idx = np.argsort(-c.logits, 1)[:, :2].astype(np.int32)
        c.d_logits.copy_(torch.from_numpy(c.logits))
        c.d_idx.copy_(torch.from_numpy(c.idx))
        torch.cuda.synchronize()
        g.replay()
        c.check()


def test_gradient_against_differences():
    # beta and alpha of order one, so that fp32 losses resolve the step: central differences of the fp32 loss are
    # off by its rounding, 2 u |loss| / step, and by the third derivative, of order step^2
    T, E, k = 5, 6, 2
    c = Case(T, E, k, alpha=1.0, beta=0.1)
    base = c.forward().backward().results()
    dl = base[5]
    step = 2.0 ** -6
    for t in range(T):
        for e in range(E):
            vals = []
            for sgn in (1, -1):
                x = c.logits.copy()
                x[t, e] += np.float32(sgn * step)
                c.d_logits.copy_(torch.from_numpy(x))
                vals.append(c.forward().results()[0].astype(np.float64).sum())
            num = (vals[0] - vals[1]) / (2 * step)
            assert abs(num - dl[t, e]) <= 2 * 64 * U * abs(vals[0]) / step + 4 * step ** 2, (t, e)
    c.d_logits.copy_(torch.from_numpy(c.logits))


@pytest.mark.parametrize("T,E", [(60, 7), (100, 64), (700, 130), (600, 512)])
def test_rows_far_from_zero(T, E):
    # Rows shifted by up to 2^30 and rows with every logit at the type's lowest value (p = 1 / E). A row's probabilities
    # depend on its differences alone, whose size is at most d for all that are not negligible: (2 d + 16) u relative.
    r = np.random.default_rng(T)
    logits = r.normal(size=(T, E)).astype(np.float32)
    for t in range(T):
        shift = [0.0, 70.0, -70.0, 3e3, -3e3, 2e6, -2e6, 2.0 ** 30, -2.0 ** 30][t % 9]
        logits[t] += np.float32(shift)
    logits[5] = logits[20] = np.finfo(np.float32).min
    logits[21, 1:] = np.finfo(np.float32).min
    d = 128 * 1.5                                           # 2^30 + x keeps x to multiples of 64 or 128
    c = Case(T, E, min(3, E), logits=logits, beta=0.0).forward().backward()
    loss, counts, mp, lse, valid, dl = c.results()
    want = ref.balance(logits, c.idx, None, [0, T], c.alpha, 0.0, c.k)
    assert np.array_equal(counts, want["counts"])
    assert (np.abs(mp - want["mean_prob"]) <= (2 * d + 112) * U * want["mean_prob"]).all()
    assert abs(loss[0] - want["loss"][0]) <= (2 * d + 112) * U * want["loss"][0] and loss[1] == 0
    assert (np.abs(lse - want["lse"]) <= (2 * d + 16) * U + U * np.abs(want["lse"])).all()
    g, mag = ref.balance_grad(want, [0, T], c.alpha, 0.0, c.k)
    # rows within 64 of zero take p from lse as it was rounded: 64 more steps of u, twice
    assert (np.abs(dl - g) <= (4 * d + 64 + 256) * U * mag).all()
    c.beta = 1e-3                                           # the z-loss leaves fp32, its gradient does not
    c.forward().backward()
    loss, counts, mp, lse, valid, dl = c.results()
    want = ref.balance(logits, c.idx, None, [0, T], c.alpha, c.beta, c.k)
    g, mag = ref.balance_grad(want, [0, T], c.alpha, c.beta, c.k)
    assert loss[1] == np.inf and (np.abs(dl - g) <= (4 * d + 64 + 256) * U * mag).all()


@pytest.mark.parametrize("T", [0, 100, 900])
def test_captured_behind_a_memset_a_copy_and_a_joined_stream(T):
    c = Case(T, 64, 2)
    want = c.forward().backward().results()
    src, s, side = c.d_logits.clone(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.lse.zero_()
        side.wait_stream(s)
        with torch.cuda.stream(side):
            c.dl.fill_(3)
        c.d_logits.copy_(src)
        s.wait_stream(side)
        c.forward()
        c.loss.add_(0.0)
        c.backward()
    for _ in range(2):
        for t in (c.loss, c.counts, c.mp, c.d_logits):
            t.fill_(7)
        g.replay()
        for x, y in zip(want, c.results()):
            assert np.array_equal(x, y)


@pytest.mark.parametrize("T,E", [(200, 8), (2000, 8), (2000, 60), (2000, 256), (1500, 511)])
def test_probabilities_of_the_gradient_do_not_lose_bits_where_lse_is_large(T, E):
    # Rows up to 63 from zero whose logits lie within 1 of each other. The exponent of a probability is a = (l - lse) log2 e,
    # |a| <= log2 E + 1.45: rounded once, half a step is 2^floor(log2 a) u, a relative error of the exponential ln 2 times
    # that; exp2 is off by 2 steps, 4 u, and the constant log2 e by less than u over a row. All of it counts once for the
    # value and once in the row's sum, which has at most 16 + 5 additions; then a quotient and a product. Rounding
    # lse log2 e, or lse, scales a row alike, which dividing by its sum undoes: nothing grows with lse. With beta alone the
    # gradient is p times three more factors; with alpha alone a sum over the experts more.
    r = np.random.default_rng(E + T)
    shift = r.uniform(40, 62.5, (T, 1)) * r.choice([-1, 1], (T, 1))
    logits = (shift + r.uniform(-0.5, 0.5, (T, E))).astype(np.float32)
    adds = min(E, 16) + 5
    one = 4 + 1 + np.log(2) * 2.0 ** np.floor(np.log2(np.log2(E) + 1.45))
    p_u = 2 * one + adds + 2
    for alpha, beta, tol in ((0.0, 1.0, p_u + 6), (1.0, 0.0, 2 * p_u + adds + 6)):
        c = Case(T, E, min(E, 8), logits=logits, alpha=alpha, beta=beta).forward().backward()
        dl = c.results()[5]
        want = ref.balance(logits, c.idx, None, [0, T], alpha, beta, c.k)
        g, mag = ref.balance_grad(want, [0, T], alpha, beta, c.k)
        assert (np.abs(dl - g) <= tol * U * mag).all(), (np.abs(dl - g) / mag).max() / U


def test_runs_of_tokens_are_joined_in_64_bits():
    # Every sum within a run of tokens is exact here: a row is 1 on expert 0, or 2^-9 on each of 512 experts, and a run's
    # sums are below 2^12 in multiples of 2^-9. Their totals have more bits than fp32. Joined in 64 bits they are exact, and
    # mean_prob is the total over the valid tokens rounded once; joined in fp32, a warp's share near 2^17 moves in steps
    # of 2^-6 and every few masks end on another value.
    ensure_lib()
    T, E = 1 << 20, 512
    r = torch.Generator(device="cuda").manual_seed(3)
    even = torch.rand(T, generator=r, device="cuda") < 0.003
    logits = torch.full((T, E), -300.0, device="cuda")
    logits[:, 0] = 0.0
    logits[even] = 0.0
    new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")
    loss, counts, mp, lse, valid = new(2), new(1, E, dt=torch.int32), new(1, E), new(T), new(3, dt=torch.int32)
    ws = new(api.moe_balance_workspace_size(T, E), dt=torch.uint8)
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    for seed in range(64):
        mask = (torch.rand(T, generator=r, device="cuda") < 0.97).to(torch.uint8)
        api.moe_balance_loss(T, E, 1, logits, idx, mask, None, 1, 1.0, 0.0, loss, counts, mp, lse, valid, ws)
        n, m = int(mask.sum()), int((mask.bool() & even).sum())
        want = np.full(E, m / 512.0) / n
        want[0] = (n - m + m / 512.0) / n
        assert np.array_equal(to_np(mp)[0], want.astype(np.float32)), seed


@pytest.mark.parametrize("T,E,S", [(2600, 16, 2600), (9000, 8, 3001), (4000, 60, 5000), (300, 12, 3000), (2500, 4, 65535)])
def test_thousands_of_sequences(T, E, S):
    # beyond 1024 (backward) and 2048 (forward) sequences a block's first one is searched for; up to the limit of S
    r = np.random.default_rng(S)
    off = np.arange(T + 1) if S == T else np.concatenate([[2], np.sort(r.integers(2, T - 5, S - 1)), [T - 5]])
    mask = None if S == T else (r.random(T) > 0.2).astype(np.uint8)
    Case(T, E, min(2, E), off=off, mask=mask).forward().backward().check()


def test_bad_offsets_of_thousands_of_sequences_stay_in_bounds():
    T, S = 3000, 2500
    c = Case(T, 16, 2, off=list(range(S + 1)))
    c.d_off.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, (S + 1,), generator=torch.Generator().manual_seed(1), dtype=torch.int64).int())
    c.forward().backward()
    torch.cuda.synchronize()
    assert api.moe_get_device_status() == api.MOE_ERR_CAPACITY


@pytest.mark.parametrize("T,E,S", [(200, 8, 65535), (256, 65, 2500)])
def test_few_tokens_of_thousands_of_sequences(T, E, S):
    # the one-launch form; most sequences are empty
    r = np.random.default_rng(S)
    off = np.concatenate([[0], np.sort(r.integers(0, T, S - 1)), [T - 1]])
    Case(T, E, 2, off=off).forward().backward().check()
