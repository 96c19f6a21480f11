"""64-bit definitions of the row-routed products (low-rank adapters picked by
row, their gradients, a mixture-of-experts layer) on CPU tensors, each with the
bound its tests use.

Bounds.  u = 2^-24.  A sum of n products in fp32, in any order and with
truncating additions, is off by at most n * 2u * sum |terms|; a kept factor of
22 significant bits adds 2^-22 of its terms; the result's rounding to half adds
2^-11 |result| and, below the normal range, 2^-25."""
import torch

U2 = 2.0 ** -23      # 2u
HALF = 2.0 ** -11    # half rounding, relative
TINY = 2.0 ** -25    # half rounding, subnormal


def d(x):
    return x.double()


def half_tol(ref, n, terms):
    return HALF * ref.abs() + TINY + (n + 8) * U2 * terms + 2.0 ** -22 * terms


def f32_tol(ref, n, terms):
    return 2.0 ** -24 * ref.abs() + (n + 8) * U2 * terms + 2.0 ** -21 * terms


def rows_by_adapter(ids, n):
    return {a: torch.where(ids == a)[0] for a in range(n)}


def lora(X, W, C0, A, B, ids, scales, alpha, beta):
    """(ref, tol) of alpha (X W + s (X A) B) + beta C0."""
    X, W, A, B = d(X), d(W), d(A), d(B)
    M, K = X.shape
    R = A.shape[2]
    ref, terms = X @ W, X.abs() @ W.abs()
    for a, rows in rows_by_adapter(ids, A.shape[0]).items():
        s = float(scales[a]) if scales is not None else 1.0
        ref[rows] += s * (X[rows] @ A[a]) @ B[a]
        terms[rows] += abs(s) * (X[rows].abs() @ A[a].abs()) @ B[a].abs()
    ref, terms = alpha * ref, abs(alpha) * terms
    if beta:
        ref = ref + beta * d(C0)
        terms = terms + abs(beta) * d(C0).abs()
    return ref, half_tol(ref, K + R, terms)


def lora_grad(G, X, W, A, B, ids, scales, alpha, beta, dA0, dB0):
    """{name: (ref, tol)} of dX, dA, dB."""
    G, X, W, A, B = d(G), d(X), d(W), d(A), d(B)
    M, N = G.shape
    K, R = A.shape[1:]
    dX, tX = G @ W.t(), G.abs() @ W.abs().t()
    dA, tA = torch.zeros_like(A), torch.zeros_like(A)
    dB, tB = torch.zeros_like(B), torch.zeros_like(B)
    for a, rows in rows_by_adapter(ids, A.shape[0]).items():
        s = float(scales[a]) if scales is not None else 1.0
        U, tU = s * (G[rows] @ B[a].t()), abs(s) * (G[rows].abs() @ B[a].abs().t())
        V, tV = s * (X[rows] @ A[a]), abs(s) * (X[rows].abs() @ A[a].abs())
        dX[rows] += U @ A[a].t()
        tX[rows] += tU @ A[a].abs().t()
        dA[a], tA[a] = X[rows].t() @ U, X[rows].abs().t() @ tU
        dB[a], tB[a] = V.t() @ G[rows], tV.t() @ G[rows].abs()
    out = {}
    for name, g, t, n, old in (("dX", dX, tX, N + R, None), ("dA", dA, tA, M + N, dA0),
                               ("dB", dB, tB, M + K, dB0)):
        g, t = alpha * g, abs(alpha) * t
        if old is not None and beta:
            g, t = g + beta * d(old), t + abs(beta) * d(old).abs()
        out[name] = (g, half_tol(g, n, t) if name == "dX" else f32_tol(g, n, t))
    return out


def moe(X, Wr, W1, W2, Y0, topk, renormalize, beta):
    """(ids, probs, probs_tol, Y, Y_tol, margin): margin is the least distance,
    in units of the logits' own error bound, between a chosen expert's logit and
    the next one in order (below 1 the order is not determined)."""
    X, Wr = d(X), d(Wr)
    T, H = X.shape
    E, I = W2.shape[0], W2.shape[1]
    l, tl = X @ Wr, X.abs() @ Wr.abs()
    dl = (H + 8) * U2 * tl
    order = torch.sort(l, dim=1, descending=True, stable=True)
    ids = order.indices[:, :topk]
    margin = float("inf")
    if E > 1 and T:
        gaps = order.values[:, :-1] - order.values[:, 1:]
        margin = float((gaps[:, :topk] / (2 * dl.max(dim=1, keepdim=True).values + 1e-300)).min())
    p = torch.gather(torch.softmax(l, dim=1), 1, ids)
    if renormalize:
        p = p / p.sum(1, keepdim=True)
    # softmax: every exponent off by at most 2 dl, exp and the sums by 2^-20
    ptol = p * (4 * dl.max(dim=1, keepdim=True).values + 2.0 ** -20 + E * U2)
    Y, tY = torch.zeros((T, H), dtype=torch.float64), torch.zeros((T, H), dtype=torch.float64)
    eY = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for k in range(topk):
            w1, w2 = d(W1[ids[t, k]]), d(W2[ids[t, k]])
            gu, tg = X[t] @ w1, X[t].abs() @ w1.abs()
            g, u = gu[:I], gu[I:]
            e = (H + 8) * U2 * tg
            s = g * torch.sigmoid(g)
            h = s * u
            # |silu'| <= 1.1; silu itself from exp and a division: 2^-20
            eh = 1.1 * e[:I] * (u.abs() + e[I:]) + s.abs() * e[I:] + 2.0 ** -20 * h.abs()
            eh = eh + 2.0 ** -22 * h.abs() + 2.0 ** -25
            Y[t] += p[t, k] * (h @ w2)
            th = h.abs() @ w2.abs()
            tY[t] += p[t, k] * th
            eY[t] += p[t, k] * (eh @ w2.abs()) + ptol[t, k] * th
    if beta:
        Y, tY = Y + beta * d(Y0), tY + abs(beta) * d(Y0).abs()
    tol = HALF * Y.abs() + TINY + eY + (I + topk + 8) * U2 * tY
    return ids, p, ptol, Y, tol, margin


def check(got, ref, tol, what=""):
    got = d(got)
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d out of tolerance, worst %g x at %s" % (
        what, int(bad.sum()), bad.numel(), float(((got - ref).abs() / tol).nan_to_num(1e30).max()),
        torch.nonzero(bad)[0].tolist())
