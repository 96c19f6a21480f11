"""The row-routed products of the library, as a user's program calls them.

Three operators whose weights go by row of the left operand:

* ``lora``: a shared projection with the low-rank adapters of many requests
  beside it, C := X.W + s[a].(X.A[a]).B[a] with a = ids[row] (-1: none);
* ``grad``: its gradients, dX (half) and dA, dB (float), the projection frozen;
* ``moe``: a whole mixture-of-experts layer (router, top-k, gated experts,
  weighted sum) for a few tokens.

``own`` picks the library's calls; otherwise the same in elementary torch
operations in 32 bits, rounded once.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request's next token through a projection with four resident adapters
        dict(name="lora_one", op="lora", M=1, N=2048, K=2048, R=16, adapters=4, order="mixed"),
        # a decoding batch: 64 requests over 32 adapters, some with none
        dict(name="lora_decode", op="lora", M=64, N=4096, K=4096, R=16, adapters=32, order="mixed"),
        # a short mixed prompt batch through an odd-width head; rows off the 16-byte grid
        dict(name="lora_ragged", op="lora", M=1000, N=1001, K=4096, R=8, adapters=5, order="runs"),
        # prompts of eight requests, each a run of rows
        dict(name="lora_prompt", op="lora", M=4096, N=4096, K=4096, R=32, adapters=8, order="runs"),
        # one micro-batch of a small layer's adapters
        dict(name="grad_small", op="grad", M=256, N=1024, K=1024, R=8, adapters=4, order="runs"),
        # sequences of uneven lengths, some rows without an adapter, an odd rank
        dict(name="grad_ragged", op="grad", M=1500, N=2048, K=1000, R=24, adapters=6, order="runs"),
        # a full training batch of eight adapters on one square projection
        dict(name="grad_large", op="grad", M=4096, N=4096, K=4096, R=16, adapters=8, order="runs"),
        # three tokens, two of sixteen small experts: latency is what counts
        dict(name="moe_small", op="moe", T=3, H=1024, I=512, E=16, topk=2, renorm=True),
        # single-token decoding, eight of 64 fine-grained experts
        dict(name="moe_one", op="moe", T=1, H=2048, I=1024, E=64, topk=8, renorm=True),
        # a ragged batch: widths that end inside a tile, unnormalised weights
        dict(name="moe_ragged", op="moe", T=37, H=1000, I=712, E=24, topk=3, renorm=False),
        # a decoding batch over most of the 64 experts
        dict(name="moe_batch", op="moe", T=16, H=4096, I=1024, E=64, topk=8, renorm=True),
        # a larger decoding batch that touches every one of 32 wide experts
        dict(name="moe_many", op="moe", T=64, H=4096, I=2048, E=32, topk=4, renorm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, odd=0.0):
    """A layer width: mostly a multiple of 64, else of 8, rarely odd."""
    x = _log(rng, lo, hi)
    u = rng.random()
    if u < odd:
        return x | 1
    x = x // 64 * 64 if u < 0.7 else x // 8 * 8
    return 3136 if x == 3072 else x


def draw(rng):
    op = rng.choice(["lora", "lora", "grad", "moe", "moe"])
    if op == "moe":
        while True:
            T, E = _log(rng, 1, 64), _log(rng, 4, 128)
            topk = min(E, rng.choice([1, 2, 3, 4, 6, 8]))
            H, I = _width(rng, 512, 4096), _width(rng, 256, 2048)
            if T * topk * H * I <= 256 * 4096 * 2048 and E * H * I <= 64 * 4096 * 1024:
                break
        return dict(op=op, T=T, H=H, I=I, E=E, topk=topk, renorm=rng.random() < 0.6)
    while True:
        lo = 1 if op == "lora" else 32
        M = _log(rng, lo, 4096)
        N, K = _width(rng, 256, 8192, 0.1), _width(rng, 256, 8192)
        if M * N * K <= 4096 ** 3:
            break
    R = rng.choice([4, 8, 8, 12, 16, 16, 16, 24, 32, 32, 48, 64])
    n = _log(rng, 1, 32)
    order = "runs" if op == "grad" or M > 256 else rng.choice(["mixed", "runs"])
    return dict(op=op, M=M, N=N, K=K, R=R, adapters=n, order=order)


# ----------------------------------------------------------------- inputs
def _normal(g, shape, std, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "moe":
        T, H, I, E, k = (case[x] for x in ("T", "H", "I", "E", "topk"))
        s["X"] = _normal(g, (T, H), 1.0)                       # normalised hidden states
        s["Wr"] = _normal(g, (H, E), 2.0 / math.sqrt(H))       # a router with clear preferences
        s["W1"] = _normal(g, (E, H, 2 * I), 1.0 / math.sqrt(H))   # gate columns, then up columns
        s["W2"] = _normal(g, (E, I, H), 1.0 / math.sqrt(I))
        s["Y"] = torch.empty((T, H), dtype=torch.float16, device=DEV)
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["probs"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        return s
    M, N, K, R, n = (case[x] for x in ("M", "N", "K", "R", "adapters"))
    s["X"] = _normal(g, (M, K), 1.0)
    s["W"] = _normal(g, (K, N), 1.0 / math.sqrt(K))
    s["A"] = _normal(g, (n, K, R), 1.0 / math.sqrt(K))
    s["B"] = _normal(g, (n, R, N), 0.5 / math.sqrt(R))
    s["scales"] = torch.empty(n, dtype=torch.float32, device=DEV).uniform_(0.5, 2.0, generator=g)
    # -1 (no adapter) is one more choice among the adapters
    if case["order"] == "runs":
        cuts = torch.rand(M, generator=g, device=DEV) < (n + 1.0) / M
        which = torch.randint(-1, n, (M,), generator=g, device=DEV)
        start = torch.where(cuts, torch.arange(M, device=DEV), 0)
        s["ids"] = which[torch.cummax(start, 0).values].int()
    else:
        s["ids"] = torch.randint(-1, n, (M,), generator=g, device=DEV).int()
    if case["op"] == "lora":
        s["C"] = torch.empty((M, N), dtype=torch.float16, device=DEV)
    else:
        s["dC"] = _normal(g, (M, N), 0.05)
        s["dX"] = torch.empty((M, K), dtype=torch.float16, device=DEV)
        s["dA"] = torch.empty((n, K, R), dtype=torch.float32, device=DEV)
        s["dB"] = torch.empty((n, R, N), dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------ plain forms
def _by_adapter(s):
    """scales[a] where row m has adapter a, else 0: (M, adapters)."""
    hit = s["ids"][:, None] == torch.arange(s["adapters"], device=s["ids"].device)[None, :]
    return torch.where(hit, s["scales"][None, :], 0.0)


def _plain_lora(s):
    X, W, A, B = (s[x].float() for x in ("X", "W", "A", "B"))
    n, K, R = A.shape
    V = (X @ A.permute(1, 0, 2).reshape(K, n * R)).view(-1, n, R) * _by_adapter(s)[:, :, None]
    return (X @ W + V.reshape(-1, n * R) @ B.reshape(n * R, -1)).half()


def _plain_grad(s):
    G, X, W, A, B = (s[x].float() for x in ("dC", "X", "W", "A", "B"))
    n, K, R = A.shape
    N = W.shape[1]
    sel = _by_adapter(s)[:, :, None]
    Acat, Bcat = A.permute(1, 0, 2).reshape(K, n * R), B.reshape(n * R, N)
    V = ((X @ Acat).view(-1, n, R) * sel).reshape(-1, n * R)
    U = ((G @ Bcat.t()).view(-1, n, R) * sel).reshape(-1, n * R)
    dX = G @ W.t() + U @ Acat.t()
    dA = (X.t() @ U).view(K, n, R).permute(1, 0, 2).contiguous()
    dB = (V.t() @ G).view(n, R, N)
    return {"dX": dX.half(), "dA": dA, "dB": dB}


def _plain_moe(s):
    X, k, I = s["X"].float(), s["topk"], s["I"]
    logits = X @ s["Wr"].float()
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    e = torch.exp(best - best[:, :1])
    p = e[:, :k] / e.sum(1, keepdim=True)
    if s["renorm"]:
        p = p / p.sum(1, keepdim=True)
    ids = ids[:, :k]
    gu = X[:, None, None, :] @ s["W1"][ids].float()            # (T, k, 1, 2I)
    gate, up = gu[..., :I], gu[..., I:]
    y = (gate / (1.0 + torch.exp(-gate)) * up) @ s["W2"][ids].float()
    return {"Y": (p[:, :, None] * y[:, :, 0]).sum(1).half(), "ids": ids.int(), "probs": p}


# -------------------------------------------------------------------- run
def run(state):
    s = state
    if not own:
        return {"lora": _plain_lora, "grad": _plain_grad, "moe": _plain_moe}[s["op"]](s)
    import dense_gemm_03_gb300 as g
    if s["op"] == "lora":
        g.gemm_f16_lora(s["X"], s["W"], s["C"], s["A"], s["B"], s["ids"], s["scales"])
        return s["C"]
    if s["op"] == "grad":
        g.gemm_f16_lora_grad(s["dC"], s["X"], s["W"], s["A"], s["B"], s["ids"], s["scales"],
                             s["dX"], s["dA"], s["dB"])
        return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}
    g.gemm_f16_moe(s["X"], s["Wr"], s["W1"], s["W2"], s["Y"], s["topk"], ids=s["ids"],
                   probs=s["probs"], renormalize=s["renorm"])
    return {"Y": s["Y"], "ids": s["ids"], "probs": s["probs"]}


def work(case):
    if case["op"] == "moe":
        T, H, I, E, k = (case[x] for x in ("T", "H", "I", "E", "topk"))
        active = E * (1.0 - (1.0 - k / E) ** T)     # experts that some token is expected to take
        return {"bytes": 2 * (2 * T * H + H * E + 3 * active * H * I) + 8 * T * k,
                "flops": 6 * T * k * H * I + 2 * T * H * E}
    M, N, K, R, n = (case[x] for x in ("M", "N", "K", "R", "adapters"))
    used = min(n, M)
    if case["op"] == "lora":
        return {"bytes": 2 * (M * K + K * N + M * N + used * R * (K + N)) + 4 * (M + n),
                "flops": 2 * M * N * K + 2 * M * R * (K + N)}
    return {"bytes": 2 * (M * N + 2 * M * K + K * N + used * R * (K + N)) + 4 * n * R * (K + N)
                     + 4 * (M + n),
            "flops": 2 * M * N * K + 2 * M * R * (3 * K + 2 * N)}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        T, H, I, k = case["T"], case["H"], case["I"], case["topk"]
        X = s["X"].double()
        logits = X @ s["Wr"].double()
        top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        p = torch.gather(torch.softmax(logits, dim=1), 1, top)
        if case["renorm"]:
            p = p / p.sum(dim=1, keepdim=True)
        Y = torch.zeros((T, H), dtype=torch.float64, device=X.device)
        for e in torch.unique(top).tolist():
            rows, slot = torch.where(top == e)
            gu = X[rows] @ s["W1"][e].double()
            h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
            Y.index_add_(0, rows, p[rows, slot][:, None] * (h @ s["W2"][e].double()))
        return {"Y": Y, "ids": None, "probs": p}
    X, W = s["X"].double(), s["W"].double()
    rows_of = {a: torch.where(s["ids"] == a)[0] for a in range(case["adapters"])}
    if case["op"] == "lora":
        C = X @ W
        for a, rows in rows_of.items():
            C[rows] += s["scales"][a].double() * (X[rows] @ s["A"][a].double()) @ s["B"][a].double()
        return C
    G = s["dC"].double()
    dX = G @ W.t()
    dA = torch.zeros(s["dA"].shape, dtype=torch.float64, device=X.device)
    dB = torch.zeros(s["dB"].shape, dtype=torch.float64, device=X.device)
    for a, rows in rows_of.items():
        A, B, sc = s["A"][a].double(), s["B"][a].double(), s["scales"][a].double()
        U = sc * (G[rows] @ B.t())
        dX[rows] += U @ A.t()
        dA[a] = X[rows].t() @ U
        dB[a] = sc * (X[rows] @ A).t() @ G[rows]
    return {"dX": dX, "dA": dA, "dB": dB}
