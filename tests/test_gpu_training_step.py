"""The training side as it is used together: moe_forward_train, the balance loss on its logits, moe_backward, the
loss's gradient through the router added to it, and the orthogonalised update of dW13 and dW2."""
import numpy as np
import pytest
import torch

import oracle
from fp8_grouped_gemm_fp32_b200 import api
from fp8_grouped_gemm_fp32_b200.inputs import CONFIGS, interleave_w13, make_inputs, transpose_weights
from gpu_helpers import assert_close_bf16, ensure_lib, rel_errors, to_np
import training_refs as ref

pytestmark = pytest.mark.gpu


def test_a_training_step():
    ensure_lib()
    cfg = CONFIGS["tiny"].replace(bias="zipf", cap_num=5, cap_den=4)
    T, H, E, I, k = cfg.T, cfg.H, cfg.E, cfg.I, cfg.k
    inp = make_inputs(cfg).to("cuda")
    c = api.Config.from_moe(cfg)
    W13, S13 = interleave_w13(inp.W1q, inp.S1, inp.W3q, inp.S3)
    W13T, S13T, W2T, S2T = transpose_weights(W13, S13, inp.W2q, inp.S2)
    new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")
    y, idx, w = new(T, H, dt=torch.bfloat16), new(T, k, dt=torch.int32), new(T, k)
    counts, slot_row = new(E, dt=torch.int32), new(T * k, dt=torch.int32)
    fws = torch.full((api.moe_workspace_size(c, 2),), 0x5a, dtype=torch.uint8, device="cuda")
    api.moe_forward_train(c, inp.x, inp.Wg, inp.bias, inp.token_ids, W13, S13, inp.W2q, inp.S2, y, idx, w, counts,
                          slot_row, fws)
    logits = api.moe_train_logits(c, fws)
    want_logits = inp.x.double() @ inp.Wg.double().t() + inp.bias.double()
    mag = inp.x.double().abs() @ inp.Wg.double().abs().t()
    assert ((logits.double() - want_logits).abs() <= (H + 2) * 2.0 ** -24 * (mag + 1)).all()

    # the balance loss over the whole batch, its counts those of the permutation
    alpha, beta = 0.5, 0.1
    loss, bcounts, mp, lse, valid = new(2), new(1, E, dt=torch.int32), new(1, E), new(T), new(3, dt=torch.int32)
    bws = new(api.moe_balance_workspace_size(T, E), dt=torch.uint8)
    api.moe_balance_loss(T, E, k, logits, idx, None, None, 1, alpha, beta, loss, bcounts, mp, lse, valid, bws)
    dl = new(T, E)
    api.moe_balance_loss_backward(T, E, k, logits, lse, bcounts, valid, None, None, 1, alpha, beta, None, dl)
    torch.cuda.synchronize()
    assert torch.equal(bcounts[0], counts)
    kept = logits.clone()

    # backward of the layer, then the loss's gradient on top, in place
    dy = (torch.randn(T, H, generator=torch.Generator().manual_seed(7)) * 0.1).to(torch.bfloat16)
    dx, dWg, db = new(T, H, dt=torch.bfloat16), new(E, H), new(E)
    dW13, dW2 = new(E, 2 * I, H, dt=torch.bfloat16), new(E, H, I, dt=torch.bfloat16)
    gws = new(api.moe_backward_workspace_size(c), dt=torch.uint8)
    api.moe_backward(c, inp.x, inp.Wg, W13, S13, W13T, S13T, W2T, S2T, idx, w, slot_row, fws, dy.cuda(), dx, dWg, db,
                     dW13, dW2, gws, fwd_train=True)
    rws = new(api.moe_router_backward_workspace_size(T, H, E), dt=torch.uint8)
    api.moe_router_backward(T, H, E, inp.x, inp.Wg, dl, dx, dWg, db, dx, dWg, db, rws)
    torch.cuda.synchronize()
    assert api.moe_get_device_status() == api.MOE_OK
    assert torch.equal(kept, logits)                       # the backward leaves the logits in the workspace

    rb = oracle.backward(cfg, oracle.moe_inputs_to_numpy(inp), dy.view(torch.int16).numpy().view(np.uint16))
    r = ref.balance(to_np(logits), to_np(idx), None, [0, T], alpha, beta, k)
    want_dl, _ = ref.balance_grad(r, [0, T], alpha, beta, k)
    x, W = inp.x.double().cpu().numpy(), inp.Wg.double().cpu().numpy()
    want_dx = oracle.bf16_bits_to_f32(rb["dx"]).astype(np.float64) + want_dl @ W
    # moe_backward's bound (max 2e-2, mean 2e-3), and one more rounding to bf16 of each value (2^-8, 2^-9 on average)
    m, a = rel_errors(dx.double().cpu().numpy(), want_dx)
    assert m <= 2e-2 + 2.0 ** -8 and a <= 2e-3 + 2.0 ** -9, (m, a)
    for got, want in ((dWg, rb["dWg"] + want_dl.T @ x), (db, rb["db"] + want_dl.sum(0))):
        err = np.abs(got.double().cpu().numpy() - want).max() / np.abs(want).max()
        assert err < 1e-3, err                             # moe_backward's bound on the gate's gradients
    assert_close_bf16(to_np(dW13).reshape(E, -1), rb["dW13"].reshape(E, -1), "dW13")

    # the update: every expert's W1 and W3 gradient, and its W2 gradient
    O13, O2 = torch.empty_like(dW13), torch.empty_like(dW2)
    n = max(api.moe_orthogonalise_workspace_size(E, I, H, True), api.moe_orthogonalise_workspace_size(E, H, I))
    ows = new(n, dt=torch.uint8)
    api.moe_orthogonalise(E, I, H, True, dW13, 5, *ref.ORTHO, 1e-7, 1.0, O13, ows)
    api.moe_orthogonalise(E, H, I, False, dW2, 5, *ref.ORTHO, 1e-7, (H / I) ** 0.5, O2, ows)
    torch.cuda.synchronize()
    assert api.moe_get_device_status() == api.MOE_OK
    for e in (0, E - 1):
        for j in range(2):
            G = ref.split(dW13[e].cpu())[j]
            assert ref.rel_norm(ref.split(O13[e].cpu())[j], ref.orthogonalise(G)) <= 2.0 ** -8 + 2.0 ** -7
        assert ref.rel_norm(O2[e].cpu(), (H / I) ** 0.5 * ref.orthogonalise(dW2[e].cpu())) <= 2.0 ** -8 + 2.0 ** -7
