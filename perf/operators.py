"""The training-side operators next to moe_backward, as measured work: the router's balance loss with its
gradient, the router's dense gradient through its linear layer, and the orthogonalised update of the experts'
weight matrices. Each case has a plain form in elementary torch operations and the calls of this package."""
import math

import numpy as np
import torch

own = False

ORTHO = (3.4445, -4.7750, 2.0315)      # a, b, c of the quintic step X <- a X + (b A + c A^2) X, A = X X^T
STEPS = 5
EPS = 1e-7


# ---------------------------------------------------------------- cases
def _balance(name, T, E, k, S, mask, tail, direction="both"):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "S": S, "mask": mask, "tail": tail,
            "direction": direction}


def _router(name, T, H, E, base):
    return {"name": name, "op": "router", "T": T, "H": H, "E": E, "base": base}


def _ortho(name, batch, M, N, interleaved, dtype):
    return {"name": name, "op": "ortho", "batch": batch, "M": M, "N": N, "interleaved": interleaved, "dtype": dtype}


def listed():
    return [
        # one small step: the decode batch of 128 tokens over 256 experts, where launches are all the time
        _balance("balance_step", 128, 256, 8, 1, False, 0),
        # the prefill batch: 8192 tokens, 256 experts, top-8, one loss over the whole batch
        _balance("balance_prefill", 8192, 256, 8, 1, False, 0),
        # packed sequences of ragged lengths, padding tokens masked, unused rows behind the last sequence; an
        # expert count that is no multiple of 8; the loss alone, as an evaluation step takes it
        _balance("balance_ragged", 16381, 60, 4, 37, True, 96, "forward"),
        # a long packed batch at the most experts the layer takes
        _balance("balance_long", 65536, 512, 8, 16, True, 0),
        # the smallest layer: 256 tokens, 8 experts
        _router("router_small", 256, 512, 8, True),
        # 4096 tokens, 64 experts, added to the gradients that moe_backward left
        _router("router_page", 4096, 4096, 64, True),
        # the prefill batch at 256 experts, added to moe_backward's gradients
        _router("router_prefill", 8192, 7168, 256, True),
        # ragged counts of tokens and experts, the loss's gradient alone
        _router("router_ragged", 5003, 1408, 100, False),
        # the smallest layer's W1 and W3 gradients, interleaved as moe_backward writes them
        _ortho("ortho_small", 8, 256, 512, True, "bf16"),
        # four experts' W2 gradients of the 4096-wide layer (more rows than columns)
        _ortho("ortho_w2", 4, 4096, 2048, False, "bf16"),
        # one expert's W1 and W3 momenta (fp32) of the 7168-wide layer
        _ortho("ortho_w13", 1, 2048, 7168, True, "f32"),
        # odd sizes: rows and columns that no tile divides
        _ortho("ortho_odd", 3, 1001, 333, False, "f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("balance", "router", "ortho"))
    if op == "balance":
        T, E = _spread(rng, 16, 65536), _spread(rng, 8, 512)
        k = rng.randint(1, min(16, E))
        S = rng.choice((1, _spread(rng, 1, max(1, T // 16))))
        c = _balance("", T, E, k, S, rng.random() < 0.5, rng.choice((0, rng.randint(0, T // 8))),
                     rng.choice(("both", "both", "forward")))
    elif op == "router":
        T, H, E = _spread(rng, 64, 16384), 128 * _spread(rng, 4, 56), _spread(rng, 8, 512)
        while T * H * E > 8192 * 7168 * 256:
            T = T * 2 // 3
        c = _router("", T, H, E, rng.random() < 0.5)
    else:
        inter = rng.random() < 0.4
        M, N = _spread(rng, 64, 4096), _spread(rng, 64, 7168)
        if inter:
            M = 128 * max(1, min(16, round(M / 128)))
        batch = rng.randint(1, 8)
        while batch > 1 and batch * (2 if inter else 1) * min(M, N) * M * N > 2 * 2048 * 2048 * 7168:
            batch -= 1
        while (2 if inter else 1) * min(M, N) * M * N > 2 * 2048 * 2048 * 7168:
            N = N * 3 // 4
        c = _ortho("", batch, M, N, inter, rng.choice(("bf16", "f32")))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 31) + 17)


def _router_logits(g, T, E):
    # logits of x W_g^T + b in a trained router: a spread of 1.3, and experts of uneven popularity
    logits = 1.3 * torch.randn(T, E, generator=g, device="cuda")
    return logits + 0.7 * torch.randn(E, generator=g, device="cuda")


def _offsets(case, seed):
    T, S, tail = case["T"], case["S"], case["tail"]
    if S == 1 and tail == 0:
        return None
    r = np.random.default_rng(seed + 5)
    cuts = np.sort(r.integers(0, T - tail + 1, S - 1))
    return torch.tensor(np.concatenate([[0], cuts, [T - tail]]), dtype=torch.int32, device="cuda")


def _low_rank(g, M, N, dtype):
    # a weight gradient summed over some steps' tokens: directions of falling strength, some noise
    r = min(M, N, 256)
    s = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -0.7
    u = torch.randn(M, r, generator=g, device="cuda") * s
    v = torch.randn(r, N, generator=g, device="cuda")
    return (1e-3 * (u @ v + 0.05 * torch.randn(M, N, generator=g, device="cuda"))).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        st["logits"] = _router_logits(g, T, E)
        st["idx"] = st["logits"].topk(k, dim=1).indices.to(torch.int32)
        st["mask"] = (torch.rand(T, generator=g, device="cuda") > 0.1).to(torch.uint8) if case["mask"] else None
        st["offsets"] = _offsets(case, seed)
        st["alpha"], st["beta"] = 0.01, 1e-3
        st["dloss"] = torch.ones(2, device="cuda")
        dev = dict(device="cuda")
        st["loss"] = torch.zeros(2, **dev)
        st["counts"] = torch.zeros(S, E, dtype=torch.int32, **dev)
        st["mean_prob"] = torch.zeros(S, E, **dev)
        st["lse"] = torch.zeros(T, **dev)
        st["valid"] = torch.zeros(S + 2, dtype=torch.int32, **dev)
        st["dlogits"] = torch.zeros(T, E, **dev)
        if own:
            from fp8_grouped_gemm_fp32_b200 import api
            st["ws"] = torch.empty(api.moe_balance_workspace_size(T, E, S), dtype=torch.uint8, **dev)
    elif case["op"] == "router":
        T, H, E = case["T"], case["H"], case["E"]
        st["x"] = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        st["Wg"] = 0.02 * torch.randn(E, H, generator=g, device="cuda")
        p = torch.softmax(_router_logits(g, T, E), 1)
        c = 0.02 / T * torch.rand(E, generator=g, device="cuda")
        st["dlogits"] = p * (c - (p * c).sum(1, keepdim=True))
        st["dx0"] = st["dWg0"] = st["db0"] = None
        if case["base"]:
            # of the size of the loss's own gradient, so that neither hides the other's rounding
            unit = 0.01 / (T * E)
            st["dx0"] = (0.02 * unit * math.sqrt(E) * torch.randn(T, H, generator=g, device="cuda")).to(torch.bfloat16)
            st["dWg0"] = unit * math.sqrt(T) * torch.randn(E, H, generator=g, device="cuda")
            st["db0"] = unit * math.sqrt(T) * torch.randn(E, generator=g, device="cuda")
        st["dx"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        st["dWg"] = torch.empty(E, H, device="cuda")
        st["db"] = torch.empty(E, device="cuda")
        if own:
            from fp8_grouped_gemm_fp32_b200 import api
            st["ws"] = torch.empty(api.moe_router_backward_workspace_size(T, H, E), dtype=torch.uint8, device="cuda")
    else:
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        B, M, N = case["batch"], case["M"], case["N"]
        if case["interleaved"]:
            pairs = [torch.stack([_low_rank(g, M, N, dt) for _ in range(2)]) for _ in range(B)]
            st["G"] = torch.stack([_interleave(p) for p in pairs])
        else:
            st["G"] = torch.stack([_low_rank(g, M, N, dt) for _ in range(B)])
        st["O"] = torch.empty(st["G"].shape, dtype=torch.bfloat16, device="cuda")
        st["scale"] = math.sqrt(max(1.0, M / N))
        if own:
            from fp8_grouped_gemm_fp32_b200 import api
            n = api.moe_orthogonalise_workspace_size(B, M, N, case["interleaved"])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


def _interleave(p):
    """[2, M, N] -> [2M, N], rows in alternating blocks of 128 of the first and the second matrix."""
    _, M, N = p.shape
    return p.reshape(2, M // 128, 128, N).transpose(0, 1).reshape(2 * M, N).contiguous()


def _split(G):
    """[B, 2M, N] -> [2B, M, N], the inverse of _interleave for every entry."""
    B, M2, N = G.shape
    return G.reshape(B, M2 // 256, 2, 128, N).transpose(1, 2).reshape(2 * B, M2 // 2, N)


def _join(O, B):
    _, M, N = O.shape
    return O.reshape(B, 2, M // 128, 128, N).transpose(1, 2).reshape(B, 2 * M, N).contiguous()


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return {"balance": _plain_balance, "router": _plain_router, "ortho": _plain_ortho}[st["op"]](st)


def _run_own(st):
    from fp8_grouped_gemm_fp32_b200 import api
    if st["op"] == "balance":
        api.moe_balance_loss(st["T"], st["E"], st["k"], st["logits"], st["idx"], st["mask"], st["offsets"], st["S"],
                             st["alpha"], st["beta"], st["loss"], st["counts"], st["mean_prob"], st["lse"],
                             st["valid"], st["ws"])
        out = [st["loss"], st["counts"], st["mean_prob"], st["lse"], st["valid"]]
        if st["direction"] == "both":
            api.moe_balance_loss_backward(st["T"], st["E"], st["k"], st["logits"], st["lse"], st["counts"],
                                          st["valid"], st["mask"], st["offsets"], st["S"], st["alpha"], st["beta"],
                                          st["dloss"], st["dlogits"])
            out.append(st["dlogits"])
        return out
    if st["op"] == "router":
        api.moe_router_backward(st["T"], st["H"], st["E"], st["x"], st["Wg"], st["dlogits"], st["dx0"], st["dWg0"],
                                st["db0"], st["dx"], st["dWg"], st["db"], st["ws"])
        return [st["dx"], st["dWg"], st["db"]]
    api.moe_orthogonalise(st["batch"], st["M"], st["N"], st["interleaved"], st["G"], STEPS, *ORTHO, EPS, st["scale"],
                          st["O"], st["ws"])
    return st["O"]


def _plain_balance(st):
    T, E, k, S = st["T"], st["E"], st["k"], st["S"]
    logits, idx, mask, off = st["logits"], st["idx"], st["mask"], st["offsets"]
    m = logits.amax(1, keepdim=True)
    e = torch.exp(logits - m)
    z = e.sum(1, keepdim=True)
    p = e / z
    lse = (m + torch.log(z))[:, 0]
    tok = torch.arange(T, device="cuda")
    if off is None:
        seg = torch.zeros(T, dtype=torch.long, device="cuda")
        inside = torch.ones(T, dtype=torch.bool, device="cuda")
    else:
        seg = (tok[:, None] >= off[None, 1:-1]).sum(1) if S > 1 else torch.zeros(T, dtype=torch.long, device="cuda")
        inside = (tok >= off[0]) & (tok < off[-1])
    ok = inside if mask is None else inside & (mask != 0)
    w = ok.to(torch.float32)
    n = torch.zeros(S, device="cuda").index_add_(0, seg, w)
    counts = torch.zeros(S, E, device="cuda")
    counts.view(-1).index_add_(0, (seg[:, None] * E + idx).view(-1), w[:, None].expand(T, k).reshape(-1))
    if S == 1:
        psum = (p * w[:, None]).sum(0, keepdim=True)
    else:
        psum = torch.zeros(S, E, device="cuda").index_add_(0, seg, p * w[:, None])
    nn = n.clamp(min=1.0)[:, None]
    P = psum / nn
    f = counts * (E / k) / nn
    seqs, total = (n > 0).sum(), n.sum()
    loss = torch.stack([st["alpha"] * (f * P).sum() / seqs.clamp(min=1),
                        st["beta"] * (w * lse * lse).sum() / total.clamp(min=1)])
    valid = torch.cat([n, seqs[None].to(n.dtype), total[None]]).to(torch.int32)
    lse_out = torch.where(ok, lse, torch.zeros_like(lse))
    out = [loss, counts.to(torch.int32), P, lse_out, valid]
    if st["direction"] == "both":
        c = st["dloss"][0] * st["alpha"] / seqs.clamp(min=1) * f / nn
        c = c[0][None] if S == 1 else c[seg]
        d = p * (c - (p * c).sum(1, keepdim=True))
        d = d + st["dloss"][1] * 2.0 * st["beta"] / total.clamp(min=1) * lse[:, None] * p
        out.append(torch.where(ok[:, None], d, torch.zeros_like(d)))
    return out


def _plain_router(st):
    dl = st["dlogits"]
    dx = dl @ st["Wg"]
    dWg = dl.t() @ st["x"].float()
    db = dl.sum(0)
    if st["dx0"] is not None:
        dx, dWg, db = dx + st["dx0"].float(), dWg + st["dWg0"], db + st["db0"]
    return [dx.to(torch.bfloat16), dWg, db]


def _plain_ortho(st):
    a, b, c = ORTHO
    G = st["G"].float()
    X = _split(G) if st["interleaved"] else G
    tall = st["M"] > st["N"]
    if tall:
        X = X.transpose(1, 2)
    X = X / ((X * X).sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    if tall:
        X = X.transpose(1, 2)
    X = st["scale"] * X
    return (_join(X, st["batch"]) if st["interleaved"] else X).to(torch.bfloat16).contiguous()


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        both = case["direction"] == "both"
        b = 4 * T * E + 4 * T * k + 4 * T + 8 * S * E + (T if case["mask"] else 0)
        return {"bytes": b + (4 * T * E if both else 0), "flops": (10 if both else 5) * T * E}
    if case["op"] == "router":
        T, H, E = case["T"], case["H"], case["E"]
        b = 2 * T * H + 4 * E * H + 4 * T * E + 2 * T * H + 4 * E * H
        return {"bytes": b + (2 * T * H + 4 * E * H if case["base"] else 0), "flops": 4 * T * H * E}
    M, N = case["M"], case["N"]
    B = case["batch"] * (2 if case["interleaved"] else 1)
    s, l = min(M, N), max(M, N)
    size = 2 if case["dtype"] == "bf16" else 4
    # A and A^2 are symmetric: half of each product; the update is a whole one
    return {"bytes": B * M * N * (size + 2), "flops": B * STEPS * (s * s * l + s * s * s + 2 * s * s * l)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        logits = st["logits"].double()
        lse = torch.logsumexp(logits, 1)
        prob = torch.exp(logits - lse[:, None])
        off = [0, T] if st["offsets"] is None else st["offsets"].tolist()
        keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
        idx = st["idx"].long()
        n, counts, P = [], [], []
        for s in range(S):
            rows = slice(off[s], off[s + 1])
            kept = keep[rows]
            n.append(int(kept.sum()))
            counts.append(torch.bincount(idx[rows][kept].reshape(-1), minlength=E))
            P.append(prob[rows][kept].sum(0) / max(1, n[-1]))
        counts, P = torch.stack(counts), torch.stack(P)
        seqs, total = max(1, sum(v > 0 for v in n)), max(1, sum(n))
        nn = torch.tensor([max(1, v) for v in n], dtype=torch.float64, device="cuda")[:, None]
        f = E * counts.double() / (k * nn)
        live = torch.zeros(T, dtype=torch.bool, device="cuda")
        live[off[0]:off[-1]] = keep[off[0]:off[-1]]
        loss = torch.stack([st["alpha"] * (f * P).sum() / seqs, st["beta"] * (lse[live] ** 2).sum() / total])
        valid = torch.tensor(n + [sum(v > 0 for v in n), sum(n)], dtype=torch.int32, device="cuda")
        out = [loss, counts.to(torch.int32), P, torch.where(live, lse, 0.0), valid]
        if case["direction"] == "both":
            d = torch.zeros(T, E, dtype=torch.float64, device="cuda")
            for s in range(S):
                rows = slice(off[s], off[s + 1])
                c = st["alpha"] / seqs * f[s] / nn[s]
                q = prob[rows]
                g = q * c - q * (q @ c)[:, None] + 2 * st["beta"] / total * lse[rows, None] * q
                d[rows] = torch.where(keep[rows, None], g, 0.0)
            out.append(d)
        return out
    if case["op"] == "router":
        dl = st["dlogits"].double()
        dx, dWg, db = dl @ st["Wg"].double(), dl.t() @ st["x"].double(), dl.sum(0)
        if case["base"]:
            dx, dWg, db = dx + st["dx0"].double(), dWg + st["dWg0"].double(), db + st["db0"].double()
        return [dx, dWg, db]
    a, b, c = ORTHO
    G = st["G"].double()
    mats = _split(G) if case["interleaved"] else G
    out = torch.empty_like(mats)
    for i in range(mats.shape[0]):
        X = mats[i] if case["M"] <= case["N"] else mats[i].t()
        X = X / (torch.linalg.matrix_norm(X) + EPS)
        for _ in range(STEPS):
            A = X @ X.t()
            X = a * X + b * (A @ X) + c * (A @ (A @ X))
        out[i] = st["scale"] * (X if case["M"] <= case["N"] else X.t())
    return _join(out, case["batch"]) if case["interleaved"] else out
