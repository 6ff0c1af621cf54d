"""64-bit references of the training-side operators (balance loss, the router's dense gradient, orthogonalised
updates) in numpy and torch on the CPU, written from their formulas."""
from __future__ import annotations

import numpy as np
import torch

ORTHO = (3.4445, -4.7750, 2.0315)


def balance(logits, idx, mask, off, alpha, beta, k, counts=None):
    """loss [2], counts [S, E], mean_prob [S, E], lse [T], valid [S + 2], live [T] (valid tokens inside a
    sequence). `counts` overrides the counted slots (constants of the gradient)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    S = len(off) - 1
    m = np.where(np.isfinite(l).any(1), l.max(1, initial=-np.inf), 0.0) if T else np.zeros(0)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        ex = np.exp(l - m[:, None])
        lse = m + np.log(ex.sum(1))
        p = ex / ex.sum(1, keepdims=True)      # exp(l - lse) would lose log E beside lowest values
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    cnt, mp, n = np.zeros((S, E)), np.zeros((S, E)), np.zeros(S, np.int64)
    live = np.zeros(T, bool)
    for s in range(S):
        rows = np.arange(off[s], off[s + 1])
        rows = rows[keep[rows]]
        live[rows] = True
        n[s] = rows.size
        ids = np.asarray(idx)[rows].reshape(-1)
        ids = ids[(ids >= 0) & (ids < E)]
        cnt[s] = np.bincount(ids, minlength=E)
        if rows.size:
            mp[s] = p[rows].sum(0) / rows.size
    if counts is not None:
        cnt = counts
    seqs, total = int((n > 0).sum()), int(n.sum())
    nn = np.maximum(n, 1)[:, None]
    loss = np.array([alpha * (E * cnt / (k * nn) * mp).sum() / max(seqs, 1),
                     beta * (lse[live] ** 2).sum() / max(total, 1)])
    valid = np.concatenate([n, [seqs, total]])
    return dict(loss=loss, counts=cnt, mean_prob=mp, lse=lse, valid=valid, live=live, p=p)


def balance_grad(r, off, alpha, beta, k, g=(1.0, 1.0)):
    """dlogits [T, E] from balance()'s results, and the size of the terms it is a difference of."""
    p, lse = r["p"], r["lse"]
    T, E = p.shape
    seqs, total = max(int(r["valid"][-2]), 1), max(int(r["valid"][-1]), 1)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for s in range(len(off) - 1):
        n = max(int(r["valid"][s]), 1)
        c = g[0] * alpha * E * r["counts"][s] / (k * n * n * seqs)
        for t in range(off[s], off[s + 1]):
            if r["live"][t]:
                z = 2 * g[1] * beta / total * lse[t]
                d[t] = p[t] * (c - p[t] @ c) + z * p[t]
                mag[t] = p[t] * (np.abs(c) + p[t] @ np.abs(c) + abs(z))
    return d, mag


def orthogonalise(G, steps=5, coef=ORTHO, eps=1e-7):
    """The iteration in 64 bits, X of one matrix [M, N] (before any output scale)."""
    a, b, c = coef
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    X = X / (X.norm() + eps)
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.t() if tall else X


def orthogonalise_model(G, steps=5, coef=ORTHO, eps=1e-7, merged=False, spare=0):
    """The same with the kernel's roundings, sums in 64 bits: products of fp16 X, 64 A and 64 B; X carried as two
    fp16 values that both enter a X; X times a power of two near the square root of the longer side, and `spare` bits more
    (the kernel's: 5). merged: the first two steps at once, as large matrices take them."""
    a, b, c = coef
    h = lambda t: t.to(torch.float16).double()
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    S = 2.0 ** (np.floor(0.5 * np.log2(max(X.shape)) + 0.5) + spare)
    X = X / (X.norm() + eps) * S
    if merged:
        hi = h(X)
        P = h(hi @ hi.t() * (64 / S ** 2))
        B1 = h(b * P + c / 64 * (P @ P))
        D = h(B1 @ P / 64)
        A2 = h(a * a * P + 2 * a * D + B1 @ D / 64)
        B2 = h(b * A2 + c / 64 * (A2 @ A2))
        X = a * a * (hi + h(X - hi)) + h(a * (B1 + B2) + B2 @ B1 / 64) @ hi / 64
    for _ in range(steps - 2 if merged else steps):
        hi = h(X)
        P = h(hi @ hi.t() * (64 / S ** 2))
        Q = h(b * P + c / 64 * (P @ P))
        X = a * (hi + h(X - hi)) + Q @ hi / 64
    X = X / S
    return X.t() if tall else X


def low_rank(M, N, r, seed=0, device="cpu"):
    """A matrix of exactly rank r in fp32: products of small whole numbers."""
    g = torch.Generator().manual_seed(seed + 1000 * M + N + r)
    u, v = (torch.randint(-9, 10, s, generator=g).float() for s in ((M, r), (r, N)))
    return (u @ v).to(device)


def rel_norm(x, y):
    x, y = torch.as_tensor(x).double(), torch.as_tensor(y).double()
    return float((x - y).norm() / max(float(y.norm()), 1e-300))


def interleave(pair):
    """[2, M, N] -> [2M, N] in alternating blocks of 128 rows."""
    _, M, N = pair.shape
    return pair.reshape(2, M // 128, 128, N).transpose(0, 1).reshape(2 * M, N).contiguous()


def split(W):
    """[2M, N] -> [2, M, N], the inverse of interleave."""
    M2, N = W.shape
    return W.reshape(M2 // 256, 2, 128, N).transpose(0, 1).reshape(2, M2 // 2, N)
