"""64-bit definitions of the dense block's operators (gated projections and their
gradients, products with transposed operands, 8-bit products, quantised tokens)
on CPU tensors, each with the bound its tests use.

Bounds.  u = 2^-24.  A sum of n products in fp32, in any order and with truncating
additions, is off by at most n * 2u * sum |terms| (sum_tol); a result's rounding to half
adds 2^-11 |result| and, below the normal range, 2^-25, to float 2^-24 |result|.

f is evaluated with ex2.approx (2 units of 2^-23) of a product that is rounded (half a unit of
|x| and as much for its constant), rcp.approx (1), for gelu a
polynomial fitted to 1.8e-7 (1.5 units, and as much again for its roundings), an addition and two
products (half a unit each), and an argument that is itself rounded, by up to three units: a relative error of f of at most act_rel(g), in
which the argument's rounding counts by the derivative of the exponent (|g| for silu, g^2
for gelu, about 1.6 |g| + 0.08 |g|^3 for gelu_tanh).  f' is a sum of two such terms, of
magnitudes at most 1 and |g f''|-like 0.6: off by at most 2 act_rel(g).  f is
Lipschitz with 1.13, f' with 0.8; relu's f' is 0 or 1 within the sum's error of 0."""
import torch

from routed_ref import HALF, TINY, U2, check, d  # noqa: F401

ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def sum_tol(n, terms):
    return (n + 8) * U2 * terms


def half_round(ref):
    return HALF * ref.abs() + TINY


def act_both(act, g):
    """f(g) and f'(g) in the type of g."""
    F = torch.nn.functional
    f = {"silu": F.silu, "gelu": F.gelu, "relu": F.relu,
         "gelu_tanh": lambda x: F.gelu(x, approximate="tanh")}[act]
    x = g.detach().clone().requires_grad_(True)
    y = f(x)
    (dy,) = torch.autograd.grad(y.sum(), x) if x.numel() else (torch.zeros_like(x),)
    return y.detach(), dy


def act_rel(g):
    a = g.abs()
    return 2.0 ** -23 * (8 + 4 * a + a * a + 0.3 * a ** 3)


def gu(X, W, sx=None, sw=None):
    """G, U and their bounds."""
    X, W = d(X), d(W)
    N = W.shape[1] // 2
    S, t = X @ W, X.abs() @ W.abs()
    e = sum_tol(X.shape[1], t)
    if sx is not None:
        s = d(sx)[:, None] * d(sw)[None, :]
        S, e = S * s, e * s + 4 * U2 * (S * s).abs()
    return S[:, :N], S[:, N:], e[:, :N], e[:, N:]


def joined(act, G, U, eG, eU):
    """(ref, tol) of f(G) .* U in half."""
    f, _ = act_both(act, G)
    ef = 1.13 * eG + act_rel(G) * f.abs()
    C = f * U
    return C, half_round(C) + ef * (U.abs() + eU) + f.abs() * eU + U2 * C.abs()


def glu(X, W, act):
    return joined(act, *gu(X, W))


def glu_grad(dC, X, W, act):
    """(ref, tol) of dGU in half."""
    G, U, eG, eU = gu(X, W)
    f, df = act_both(act, G)
    c = d(dC).abs()
    ed = 0.8 * eG + 2 * act_rel(G) if act != "relu" else (G.abs() <= eG).double()
    dG, dU = d(dC) * U * df, d(dC) * f
    tG = c * (ed * (U.abs() + eU) + df.abs() * eU) + 2 * U2 * dG.abs()
    tU = c * (1.13 * eG + act_rel(G) * f.abs()) + U2 * dU.abs()
    ref = torch.cat([dG, dU], 1)
    return ref, half_round(ref) + torch.cat([tG, tU], 1)


def i8_sums(X, W):
    """The integer sums and their bound: exact where no partial sum can reach 2^24."""
    X, W = d(X), d(W)
    S, t = X @ W, X.abs() @ W.abs()
    return S, sum_tol(X.shape[1], t) * (t >= 2.0 ** 24)


def i8(X, W, sx, sw, act=None, beta=0.0, C0=None):
    """(ref, tol) of the scaled 8-bit product; two roundings of each scaled sum."""
    S, e = i8_sums(X, W)
    s = (d(sx) if sx is not None else torch.ones(X.shape[0], dtype=torch.float64))[:, None] * \
        (d(sw) if sw is not None else torch.ones(W.shape[1], dtype=torch.float64))[None, :]
    S, e = S * s, e * s + U2 * (S * s).abs()
    if act is not None:
        N = W.shape[1] // 2
        return joined(act, S[:, :N], S[:, N:], e[:, :N], e[:, N:])
    if beta:
        S, e = S + beta * d(C0), e + U2 * (S.abs() + abs(beta) * d(C0).abs())
    return S, half_round(S) + e


def to_i8(X):
    """(Q, scales): the exact rounding, in integers (a half is a multiple of 2^-24)."""
    n = (d(X) * 2.0 ** 24).numpy().astype(object)
    Q = torch.zeros(X.shape, dtype=torch.int8)
    for i, row in enumerate(n):
        row = [int(v) for v in row]
        a = max((abs(v) for v in row), default=0)
        if a:
            for k, v in enumerate(row):
                q, r = divmod(2 * 127 * abs(v) + a, 2 * a)     # nearest, ties up
                if r == 0 and q % 2:
                    q -= 1                                     # ties to even
                Q[i, k] = q if v >= 0 else -q
    a = X.abs().float().amax(1) if X.shape[1] else torch.zeros(X.shape[0])
    return Q, a / torch.full_like(a, 127.0)


def product(A, B, alpha=1.0, beta=0.0, C0=None, f32=False):
    """(ref, tol) of alpha A B + beta C0."""
    A, B = d(A), d(B)
    ref, t = alpha * (A @ B), abs(alpha) * (A.abs() @ B.abs())
    if beta:
        ref, t = ref + beta * d(C0), t + abs(beta) * d(C0).abs()
    return ref, (U2 * ref.abs() if f32 else half_round(ref)) + sum_tol(A.shape[1], t)
