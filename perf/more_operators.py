"""The dense block of a language model, trained in half and served in 8 bits, as a
user's program calls it.

* ``glu``: the gated projections with their activation, C := f(X.Wg) * (X.Wu), W = [Wg Wu];
* ``grad``: their backward pass, the gates' gradients dGU, dX and dW, from dC, X and W;
* ``trans``: products with transposed operands (the gradients of any projection), half or
  float result;
* ``i8``: the product in 8-bit integers with a scale for each token and each channel,
  plain or gated;
* ``to_i8``: tokens rounded to 8-bit integers with a scale each.

``own`` picks the library's calls; otherwise the same in elementary torch operations in
32 bits, rounded once.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request's next token through a small block: latency is what counts
        dict(name="glu_one", op="glu", M=1, K=2048, N=4096, act="silu"),
        # a mixed prompt batch, widths off the 16-byte grid
        dict(name="glu_ragged", op="glu", M=777, K=1000, N=1501, act="gelu"),
        # prompts or a training batch through a full block
        dict(name="glu_prompt", op="glu", M=4096, K=4096, N=8192, act="silu"),
        # a micro-batch of uneven sequences
        dict(name="grad_ragged", op="grad", M=1500, K=1000, N=1368, act="gelu_tanh"),
        # a training batch of a full layer
        dict(name="grad_large", op="grad", M=4096, K=2048, N=4096, act="silu"),
        # dX of a projection for a short batch: dC.W^T, an odd number of tokens
        dict(name="dx_short", op="trans", M=331, N=2048, K=4096, ta=False, tb=True, f32=False),
        # a projection's weight gradient in float, X^T.dC over the tokens of a batch
        dict(name="dw_batch", op="trans", M=4096, N=4096, K=8192, ta=True, tb=False, f32=True),
        # single-token decoding through an 8-bit projection
        dict(name="i8_one", op="i8", M=1, K=4096, N=4096, act=""),
        # a decoding batch through the gated projections of an 8-bit block
        dict(name="i8_decode", op="i8", M=48, K=4096, N=8192, act="silu"),
        # prompts through an 8-bit projection
        dict(name="i8_prompt", op="i8", M=4096, K=4096, N=4096, act=""),
        # the tokens of a decoding batch, rows off the 16-byte grid
        dict(name="to_i8_decode", op="to_i8", M=24, K=4099),
        # the tokens of a prompt batch
        dict(name="to_i8_prompt", op="to_i8", M=8192, K=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, odd=0.15):
    """A layer width: mostly a multiple of 64, else of 8, now and then odd."""
    x = _log(rng, lo, hi)
    u = rng.random()
    if u < odd:
        return x | 1
    return x // 64 * 64 if u < 0.7 else x // 8 * 8


def draw(rng):
    op = rng.choice(["glu", "glu", "grad", "trans", "i8", "i8", "to_i8"])
    act = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
    if op == "to_i8":
        return dict(op=op, M=_log(rng, 1, 8192), K=_width(rng, 128, 8192))
    while True:
        if op == "trans":
            ta, tb = rng.choice([(True, False), (True, False), (False, True), (True, True)])
            M, N = (_width(rng, 128, 4096) for _ in "MN")
            K = _log(rng, 64, 8192)
            case = dict(op=op, M=M if ta else K // 2, N=N, K=K if ta else M, ta=ta, tb=tb,
                        f32=rng.random() < 0.5)
        else:
            M = _log(rng, 64 if op == "grad" else 1, 4096)
            K, N = _width(rng, 256, 8192), _width(rng, 256, 8192)
            if op == "i8":
                act = rng.choice(["", "", act])
            case = dict(op=op, M=M, K=K, N=N, act=act)
        if M * N * K <= {"glu": 4096 * 4096 * 8192, "grad": 4096 * 2048 * 4096,
                         "trans": 4096 * 4096 * 8192, "i8": 4096 ** 3}[op]:
            return case


# ----------------------------------------------------------------- inputs
def _normal(g, shape, std, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _quantised(x, dim):
    """Normal values as 8-bit integers with a scale for each row (dim 1) or column (dim 0)."""
    scale = x.abs().amax(dim, keepdim=True) / 127.0
    return torch.round(x / scale).to(torch.int8), scale.reshape(-1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    M, K = case["M"], case["K"]
    f16 = dict(dtype=torch.float16, device=DEV)
    if case["op"] == "to_i8":
        # hidden states whose tokens differ in magnitude
        rows = torch.exp2(torch.randint(-3, 4, (M, 1), generator=g, device=DEV).float())
        s["X"] = (_normal(g, (M, K), 1.0, torch.float32) * rows).half()
        s["Q"] = torch.empty((M, K), dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(M, dtype=torch.float32, device=DEV)
        return s
    N = case["N"]
    if case["op"] == "trans":
        s["A"] = _normal(g, (K, M) if case["ta"] else (M, K), 1.0)
        s["B"] = _normal(g, (N, K) if case["tb"] else (K, N), 1.0 / math.sqrt(K))
        s["C"] = torch.empty((M, N), dtype=torch.float32 if case["f32"] else torch.float16, device=DEV)
        return s
    cols = 2 * N if case["act"] else N
    if case["op"] == "i8":
        s["X"], s["sx"] = _quantised(_normal(g, (M, K), 1.0, torch.float32), 1)
        s["W"], s["sw"] = _quantised(_normal(g, (K, cols), 1.0 / math.sqrt(K), torch.float32), 0)
        s["C"] = torch.empty((M, N), **f16)
        return s
    s["X"] = _normal(g, (M, K), 1.0)                      # normalised hidden states
    s["W"] = _normal(g, (K, cols), 1.0 / math.sqrt(K))    # N gate columns, then N up columns
    if case["op"] == "glu":
        s["C"] = torch.empty((M, N), **f16)
    else:
        s["dC"] = _normal(g, (M, N), 0.1)
        s["dGU"] = torch.empty((M, cols), **f16)
        s["dX"] = torch.empty((M, K), **f16)
        s["dW"] = torch.empty((K, cols), **f16)
    return s


# ------------------------------------------------------------ plain forms
def _gate(act, g):
    """f(g) and f'(g)."""
    if act == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    if act == "gelu":
        p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)                          # gelu_tanh: (1 + tanh z) / 2 = 1 / (1 + e^-2z)
    p = 1.0 / (1.0 + torch.exp(-2.0 * c * (g + 0.044715 * g * g * g)))
    return g * p, p + g * 2.0 * c * (1.0 + 3.0 * 0.044715 * g * g) * p * (1.0 - p)


def _plain(s):
    if s["op"] == "to_i8":
        x = s["X"].float()
        amax = x.abs().amax(1, keepdim=True)
        q = torch.round(127.0 * x / torch.where(amax > 0, amax, 1.0))
        by = torch.full_like(amax, 127.0)                 # (a tensor: divided, not multiplied by 1/127)
        return {"Q": q.to(torch.int8), "scales": (amax / by)[:, 0]}
    if s["op"] == "trans":
        A, B = s["A"].float(), s["B"].float()
        return ((A.t() if s["ta"] else A) @ (B.t() if s["tb"] else B)).to(s["C"].dtype)
    X, W, N = s["X"].float(), s["W"].float(), s["N"]
    gu = X @ W
    if s["op"] == "i8":
        gu = gu * s["sx"][:, None] * s["sw"][None, :]
        if not s["act"]:
            return gu.half()
    g, u = gu[:, :N], gu[:, N:]
    f, df = _gate(s["act"], g)
    if s["op"] != "grad":
        return (f * u).half()
    dC = s["dC"].float()
    dGU = torch.cat([dC * u * df, dC * f], 1)
    return {"dGU": dGU.half(), "dX": (dGU @ W.t()).half(), "dW": (X.t() @ dGU).half()}


# -------------------------------------------------------------------- run
def run(state):
    s = state
    if not own:
        return _plain(s)
    import dense_gemm_03_gb300 as g
    op = s["op"]
    if op == "glu":
        g.gemm_f16_glu(s["X"], s["W"], s["C"], s["act"])
        return s["C"]
    if op == "grad":
        g.gemm_f16_glu_grad(s["dC"], s["X"], s["W"], s["dGU"], s["dX"], s["dW"], s["act"])
        return {"dGU": s["dGU"], "dX": s["dX"], "dW": s["dW"]}
    if op == "trans":
        call = g.gemm_f16_trans_f32out if s["f32"] else g.gemm_f16_trans
        call(s["A"], s["B"], s["C"], s["ta"], s["tb"])
        return s["C"]
    if op == "i8":
        g.gemm_i8(s["X"], s["W"], s["C"], s["sx"], s["sw"], s["act"] or None)
        return s["C"]
    g.f16_to_i8(s["X"], s["Q"], s["scales"])
    return {"Q": s["Q"], "scales": s["scales"]}           # whole numbers: equal in both forms


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "to_i8":
        return {"bytes": 3 * M * K + 4 * M, "flops": 3 * M * K}
    N = case["N"]
    if case["op"] == "trans":
        return {"bytes": 2 * (M * K + K * N) + (4 if case["f32"] else 2) * M * N, "flops": 2 * M * N * K}
    cols = 2 * N if case["act"] else N
    if case["op"] == "i8":
        return {"bytes": M * K + K * cols + 2 * M * N + 4 * (M + cols), "flops": 2 * M * K * cols}
    if case["op"] == "glu":
        return {"bytes": 2 * (M * K + K * cols + M * N), "flops": 2 * M * K * cols}
    return {"bytes": 2 * (M * N + 2 * M * K + 2 * K * cols + M * cols), "flops": 6 * M * K * cols}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "to_i8":
        return {"Q": None, "scales": s["X"].double().abs().max(dim=1).values / 127.0}
    if op == "trans":
        A, B = s["A"].double(), s["B"].double()
        return torch.einsum("km,kn->mn" if case["ta"] else "mk,kn->mn", A, B.t() if case["tb"] else B)
    X, W, N = s["X"].double(), s["W"].double(), case["N"]
    if op == "i8":
        X, W = X * s["sx"].double().unsqueeze(1), W * s["sw"].double()
        if not case["act"]:
            return X @ W
    G, U = X @ W[:, :N], X @ W[:, N:]
    F = torch.nn.functional
    f = {"silu": F.silu, "relu": F.relu, "gelu": F.gelu,
         "gelu_tanh": lambda x: F.gelu(x, approximate="tanh")}[case["act"]]
    if op != "grad":
        return f(G) * U
    dC = s["dC"].double()
    G = G.requires_grad_(True)
    a = f(G)
    dG, = torch.autograd.grad(a, G, dC * U)
    dU = dC * a.detach()
    return {"dGU": torch.cat([dG, dU], dim=1), "dX": dG @ W[:, :N].t() + dU @ W[:, N:].t(),
            "dW": torch.cat([X.t() @ dG, X.t() @ dU], dim=1)}
