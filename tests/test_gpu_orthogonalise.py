"""moe_orthogonalise on the GPU against the 64-bit iteration and against the same iteration with the kernel's roundings.

Tolerances (2-norm of the difference over the 2-norm). Against the exact iteration: rounding to bf16, 2^-8 at most, and
the roundings of the iteration, at most 2^-7 (asserted on the CPU of the model, for these sizes and kinds).
Against the model with the same roundings only one step can be compared: kernel and model part where an fp32 sum lands
on the other side of an fp16 rounding. Sums agree to about 2^-22, so a share 2^-11 of the values of A and B differ by a
step of 2^-11, in norm 2^-16.5; that makes a share of 2^-8 of the bf16 roundings differ by 2^-8: 2^-12, below 2^-9 with
room. A second step starts 2^-16.5 apart: a share 2^-5.5 of its fp16 values differ, 2^-14 in norm; the third 2^-12.5;
from there on the two round independently, and each is only known to be near the exact iterate."""
import numpy as np
import pytest
import torch

from fp8_grouped_gemm_fp32_b200 import api
from gpu_helpers import ensure_lib
from test_training_ops_cpu import ortho_matrix
import training_refs as ref

pytestmark = pytest.mark.gpu


def run(G, batch, M, N, inter=False, steps=5, coef=ref.ORTHO, eps=1e-7, scale=1.0, stream=None, ws=None, O=None):
    ensure_lib()
    if ws is None:
        ws = torch.full((api.moe_orthogonalise_workspace_size(batch, M, N, inter),), 0x5a, dtype=torch.uint8, device="cuda")
    O = torch.full(G.shape, 7.0, dtype=torch.bfloat16, device="cuda") if O is None else O
    api.moe_orthogonalise(batch, M, N, inter, G, steps, *coef, eps, scale, O, ws, stream)
    return O


def done(O):
    torch.cuda.synchronize()
    assert api.moe_get_device_status() == api.MOE_OK
    return O


def close(O, G, steps=5, coef=ref.ORTHO, eps=1e-7, scale=1.0):
    exact = scale * ref.orthogonalise(G.cpu(), steps, coef, eps)
    assert ref.rel_norm(O.cpu(), exact) <= 2.0 ** -8 + 2.0 ** -7


@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (300, 1), (5, 7), (64, 64), (100, 260), (260, 100), (257, 513), (384, 128),
                                 (512, 512), (130, 1000)])
@pytest.mark.parametrize("kind", ["noise", "low_rank", "decay"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matches_the_iteration(M, N, kind, dtype):
    G = torch.stack([(10.0 ** (i - 4)) * ortho_matrix(M, N, kind, i) for i in range(3)]).to(dtype).cuda()
    O = done(run(G, 3, M, N))
    for i in range(3):
        close(O[i], G[i])


@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (300, 1), (5, 7), (64, 64), (100, 260), (260, 100), (257, 513), (384, 128)])
@pytest.mark.parametrize("kind", ["noise", "low_rank", "decay"])
def test_one_step_matches_the_model_with_the_same_roundings(M, N, kind):
    G = ortho_matrix(M, N, kind, 4).to(torch.bfloat16).cuda()[None].contiguous()
    O = done(run(G, 1, M, N, steps=1))
    assert ref.rel_norm(O[0].cpu(), ref.orthogonalise_model(G[0].cpu(), 1).to(torch.bfloat16)) <= 2.0 ** -9


@pytest.mark.parametrize("M,N", [(1, 16384), (128, 128), (129, 128), (128, 129), (127, 640), (2000, 77), (90, 5000), (16384, 100)])
def test_a_short_side(M, N):
    # up to 128 one launch does everything; beside the limit the other kernel
    G = torch.stack([ortho_matrix(M, N, "decay", i) for i in range(2)]).to(torch.bfloat16).cuda()
    O = done(run(G, 2, M, N))
    for i in range(2):
        assert ref.rel_norm(O[i], ref.orthogonalise(G[i])) <= 2.0 ** -8 + 2.0 ** -7


@pytest.mark.parametrize("batch,M,N,inter", [(400, 60, 70, False), (40, 128, 500, False), (200, 128, 40, True), (75, 384, 100, True),
                                             (20, 100, 3000, False)])
def test_many_narrow_matrices(batch, M, N, inter):
    G = torch.randn(batch, 2 * M if inter else M, N, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    O = done(run(G, batch, M, N, inter))
    for i in (0, 1, batch // 2, batch - 2, batch - 1):
        for o, x in zip(ref.split(O[i]) if inter else O[i:i + 1], ref.split(G[i]) if inter else G[i:i + 1]):
            assert ref.rel_norm(o, ref.orthogonalise(x)) <= 2.0 ** -8 + 2.0 ** -7


@pytest.mark.parametrize("M,N", [(128, 64), (256, 512), (384, 130), (640, 600)])
def test_interleaved_pairs(M, N):
    pairs = torch.stack([torch.stack([ortho_matrix(M, N, "decay", 2 * i + j) for j in range(2)]) for i in range(3)])
    G = torch.stack([ref.interleave(q) for q in pairs]).to(torch.bfloat16).cuda()
    O = done(run(G, 3, M, N, True, scale=0.5))
    plain = done(run(pairs.reshape(6, M, N).to(torch.bfloat16).cuda(), 6, M, N, scale=0.5))
    for i in range(3):
        assert torch.equal(ref.split(O[i]), plain[2 * i:2 * i + 2])       # the layout changes nothing else
        for j in range(2):
            close(ref.split(O[i])[j], pairs[i, j].to(torch.bfloat16), scale=0.5)


@pytest.mark.parametrize("batch,M,N,inter", [(1, 1024, 1536, False), (2, 2100, 1030, False), (3, 1024, 2048, True), (1, 1153, 1801, False),
                                             (1, 1200, 1400, False), (6, 1500, 1000, False)])
@pytest.mark.parametrize("kind", ["noise", "low_rank", "decay", "spikes"])
def test_large_matrices(batch, M, N, inter, kind):
    # the sizes that take their first two steps at once, and some beside them; the iteration in 64 bits on the GPU
    pairs = torch.stack([ortho_matrix(M, N, kind, i) for i in range(batch * (2 if inter else 1))]).cuda()
    G = torch.stack([ref.interleave(p) for p in pairs.view(batch, 2, M, N)]) if inter else pairs
    O = done(run(G, batch, M, N, inter))
    O = torch.cat([ref.split(o) for o in O]) if inter else O
    for i in range(pairs.shape[0]):
        assert ref.rel_norm(O[i], ref.orthogonalise(pairs[i])) <= 2.0 ** -8 + 2.0 ** -8


@pytest.mark.parametrize("steps,coef", [(1, ref.ORTHO), (2, ref.ORTHO), (3, (1.875, -1.25, 0.375)), (2, (2.0, -1.5, 0.5))])
def test_large_matrices_with_other_steps_and_coefficients(steps, coef):
    G = ortho_matrix(1024, 1600, "noise", 8).cuda()[None].contiguous()
    O = done(run(G, 1, 1024, 1600, steps=steps, coef=coef))
    assert ref.rel_norm(O[0], ref.orthogonalise(G[0], steps, coef)) <= 2.0 ** -8 + 2.0 ** -7


def test_a_batch_of_more_than_one_wave():
    # waves of a large batch use the workspace in turn: every matrix as if alone
    M, N, batch = 520, 520, 30
    G = torch.stack([ortho_matrix(M, N, "decay", i) for i in range(batch)]).to(torch.bfloat16).cuda()
    assert api.moe_orthogonalise_workspace_size(batch, M, N) < batch * 10 * M * N
    O = done(run(G, batch, M, N))
    for i in (0, 13, 24, 25, 29):
        assert torch.equal(O[i], done(run(G[i:i + 1].contiguous(), 1, M, N))[0])


@pytest.mark.parametrize("steps,coef", [(1, ref.ORTHO), (2, (1.5, -0.5, 0.0)), (10, (1.875, -1.25, 0.375)), (32, (1.5, -0.5, 0.0))])
def test_other_steps_and_coefficients(steps, coef):
    G = ortho_matrix(200, 310, "noise", 5).cuda()[None].contiguous()
    close(done(run(G, 1, 200, 310, steps=steps, coef=coef))[0], G[0], steps, coef)


def test_zero_matrices_tiny_and_huge_ones():
    G = torch.stack([ortho_matrix(70, 90, "noise", i) for i in range(5)])
    G[1] = 0.0
    G[2] *= 1e-36                                         # its squares are far below fp32
    G[3] *= 1e36                                          # and above it
    G = G.cuda()
    O = done(run(G, 5, 70, 90, eps=1e-30))
    assert not O[1].any()
    for i in (0, 2, 3, 4):
        close(O[i], G[i], eps=1e-30)
    # where eps is larger than the norm, it damps
    O = done(run(G, 5, 70, 90, eps=1.0))
    close(O[0], G[0], eps=1.0)
    assert not done(run(torch.zeros(1, 70, 90, device="cuda"), 1, 70, 90)).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_matrix_leaves_the_others_alone(bad):
    G = torch.stack([ortho_matrix(150, 80, "noise", i) for i in range(3)]).cuda()
    clean = done(run(G, 3, 150, 80))
    G[1, 149, 79] = bad
    O = done(run(G, 3, 150, 80))
    assert torch.isnan(O[1]).all() and torch.equal(O[0], clean[0]) and torch.equal(O[2], clean[2])


def test_rows_beyond_the_matrices_are_left_alone():
    M, N = 77, 91
    G = ortho_matrix(M, N, "noise", 3).cuda()[None].contiguous()
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    run(G, 1, M, N, O=buf[:M * N].view(1, M, N))
    done(buf)
    assert (buf[M * N:] == 7).all()


def test_repeats_on_another_stream_and_two_at_once():
    G = torch.stack([ortho_matrix(300, 520, "decay", i) for i in range(4)]).cuda()
    want = done(run(G, 4, 300, 520))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):                                    # two calls in flight, each with its own workspace
        with torch.cuda.stream(a):
            outs.append(run(G, 4, 300, 520))
        with torch.cuda.stream(b):
            outs.append(run(G, 4, 300, 520))
    done(want)
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("M,N", [(200, 140), (64, 64), (100, 700), (1030, 1700)])
def test_captured_and_replayed_on_new_inputs(M, N):
    G = torch.stack([ortho_matrix(M, N, "decay", i) for i in range(2)]).cuda()
    ws = torch.empty(api.moe_orthogonalise_workspace_size(2, M, N), dtype=torch.uint8, device="cuda")
    O = run(G, 2, M, N, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        run(G, 2, M, N, ws=ws, O=O)
    for k in range(2):
        G.copy_(torch.stack([ortho_matrix(M, N, "noise", 10 * k + i) for i in range(2)]))
        torch.cuda.synchronize()
        g.replay()
        done(O)
        for i in range(2):
            assert ref.rel_norm(O[i], ref.orthogonalise(G[i])) <= 2.0 ** -8 + 2.0 ** -7


def test_two_graphs_with_their_own_workspaces_at_once():
    shapes = [(100, 700), (300, 520)]
    graphs, outs, wants = [], [], []
    for M, N in shapes:
        G = torch.stack([ortho_matrix(M, N, "decay", i) for i in range(3)]).cuda()
        ws = torch.empty(api.moe_orthogonalise_workspace_size(3, M, N), dtype=torch.uint8, device="cuda")
        wants.append(done(run(G, 3, M, N, ws=ws)).clone())
        O = torch.zeros_like(wants[-1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            run(G, 3, M, N, ws=ws, O=O)
        graphs.append((g, G, ws))
        outs.append(O)
    streams = [torch.cuda.Stream() for _ in shapes]
    for _ in range(3):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    done(outs[0])
    assert all(torch.equal(o, w) for o, w in zip(outs, wants))


@pytest.mark.parametrize("batch,M,N", [(3, 1000, 900), (12, 600, 700), (6, 1100, 1100), (4, 1536, 1024)])
def test_several_tiles_a_cta_of_several_matrices_repeat_and_equal_each_alone(batch, M, N):
    # a CTA goes from one matrix's last tile of a product to the next matrix's, which must not count the first early
    G = torch.stack([ortho_matrix(M, N, "decay", i) for i in range(batch)]).to(torch.bfloat16).cuda()
    ws = torch.empty(api.moe_orthogonalise_workspace_size(batch, M, N), dtype=torch.uint8, device="cuda")
    alone = torch.cat([done(run(G[i:i + 1].contiguous(), 1, M, N)) for i in range(batch)])
    want = done(run(G, batch, M, N, ws=ws))
    if min(M, N) >= 1024 and 2 * max(M, N) >= 3 * min(M, N):
        # The first two steps at once hold B_1 A, symmetric up to rounding only: (i, j) sums B_1[i, k] A[k, j], (j, i) sums
        # B_1[j, k] A[k, i], other products. A few tiles are all computed, many computed once and mirrored: other bits.
        for i in range(batch):
            assert ref.rel_norm(want[i], ref.orthogonalise(G[i])) <= 2.0 ** -8 + 2.0 ** -8
    else:
        assert torch.equal(want, alone)
    for _ in range(20):
        assert torch.equal(done(run(G, batch, M, N, ws=ws)), want)


@pytest.mark.parametrize("large,small,M,N,inter", [(26, 25, 520, 520, False), (19, 18, 100, 1000, False), (13, 12, 256, 512, True)])
def test_a_smaller_batch_in_a_larger_ones_workspace(large, small, M, N, inter):
    G = torch.randn(large, 2 * M if inter else M, N, generator=torch.Generator("cuda").manual_seed(M), device="cuda")
    ws = torch.empty(api.moe_orthogonalise_workspace_size(large, M, N, inter), dtype=torch.uint8, device="cuda")
    for n in (large, small, large):
        O = done(run(G[:n].contiguous(), n, M, N, inter, ws=ws))
        for i in (0, n - 1):
            o, x = (ref.split(O[i])[1], ref.split(G[i])[1]) if inter else (O[i], G[i])
            assert ref.rel_norm(o, ref.orthogonalise(x)) <= 2.0 ** -8 + 2.0 ** -7


@pytest.mark.parametrize("M,N", [(64, 64), (900, 100), (128, 700), (300, 200), (512, 1024), (1024, 1600)])
@pytest.mark.parametrize("steps", [5, 8, 10, 12])
def test_exactly_low_rank_at_many_steps(M, N, steps):
    # What the header states: X off by at most 2^-22 of a value, and as much from B's rounding times what the first fp16 value
    # lacks of X (2^-11 of either); of a step's sums over s, s / 16 additions drop at most 2^-23 of a running sum each, a
    # quarter of it on average over the drop and the sum's way up, s 2^-29 of a X in all; a to the power of the steps
    # multiplies them. At rank 1, one step at a time, the same iteration in fp32 is no closer.
    for r in (1, 8, 32):
        G = ref.low_rank(M, N, r, device="cuda")
        O = done(run(G[None].contiguous(), 1, M, N, steps=steps))[0]
        exact = ref.orthogonalise(G, steps)
        err = ref.rel_norm(O, exact)
        grown = ref.ORTHO[0] ** steps / r ** 0.5
        assert err <= 2.0 ** -8 + 2.0 ** -7 + (2.0 ** -21 + min(M, N) * 2.0 ** -29) * grown
        if r == 1 and min(M, N) < 1024:
            a, b, c = ref.ORTHO
            X = G.t() if M > N else G
            X = X / (X.norm() + 1e-7)
            for _ in range(steps):
                A = X @ X.t()
                X = a * X + (b * A + c * (A @ A)) @ X
            assert err <= 2.0 ** -8 + 2.0 ** -7 + ref.rel_norm(X.t() if M > N else X, exact)


@pytest.mark.parametrize("M,N", [(1, 16384), (100, 16000), (200, 16384), (16384, 150)])
def test_one_entry_alone_is_the_largest_value_that_is_stored(M, N):
    # X's largest entry is its largest singular value where G has a single one; exact: the scalar iteration
    G = torch.zeros(1, M, N, device="cuda")
    G[0, M // 2, N // 3] = -3.0
    for steps, (a, b, c) in ((5, ref.ORTHO), (2, (4.5, 0.0, 0.0)), (3, (1.9, 0.0, 0.0))):
        if b == 0.0:
            c, a = 0.0, min(a, 8.0 ** (1 / steps))         # singular values up to 8 at the end
        x = 1.0
        for _ in range(steps):
            x = a * x + b * x ** 3 + c * x ** 5
        O = done(run(G, 1, M, N, steps=steps, coef=(a, b, c)))
        assert abs(float(O[0, M // 2, N // 3]) + x) <= (2.0 ** -8 + 2.0 ** -7) * x
        assert int((O != 0).sum()) == 1
