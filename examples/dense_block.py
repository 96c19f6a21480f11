"""A gated feed-forward block, trained in half and served in 8 bits, as a program calls it.

    python examples/dense_block.py

The block is Y = X + (f(X W1g) * (X W1u)) W2.  The program

1. trains W1 and W2 toward another block's outputs: forward gemm_f16_glu and gemm_f16,
   backward gemm_f16_trans (dH = dY W2^T), gemm_f16_trans_f32out (dW2, two micro-batches
   added up in float) and gemm_f16_glu_grad (dX, dW1);
2. rounds the weights to 8 bits by channel, and serves tokens with f16_to_i8 and gemm_i8,
   the gated product and the one that is added onto the residual.

Prints what it measured; returns a dict of the same when called as main().
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dense_gemm_03_gb300 as g

ACT = "silu"


def half(*shape):
    return torch.empty(shape, dtype=torch.float16, device="cuda")


def forward(x, w1, w2):
    """The block on rows x: its hidden rows and its outputs."""
    h, y = half(x.shape[0], w2.shape[0]), x.clone()
    g.gemm_f16_glu(x, w1, h, ACT)
    g.gemm_f16(h, w2, y, beta=1.0)          # onto the residual
    return h, y


def backward(x, w1, w2, h, dy, dw1, dw2, first):
    """Adds the weights' gradients onto dw1 and dw2 (float; zero first if `first`)."""
    dh, dgu = half(*h.shape), half(h.shape[0], 2 * h.shape[1])
    g.gemm_f16_trans(dy, w2, dh, trans_b=True)
    g.gemm_f16_trans_f32out(h, dy, dw2, trans_a=True, beta=0.0 if first else 1.0)
    g.gemm_f16_glu_grad(dh, x, w1, dgu, act=ACT)
    g.gemm_f16_trans_f32out(x, dgu, dw1, trans_a=True, beta=0.0 if first else 1.0)


def rounded(w):
    """Weights as 8-bit integers with a scale for each channel (column)."""
    scale = (w.float().abs().amax(0) / 127).clamp_min(1e-30)
    return torch.round(w.float() / scale).to(torch.int8), scale


def serve(x, w1, s1, w2, s2):
    """The block in 8 bits."""
    q1, a1 = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
    h, y = half(x.shape[0], w2.shape[0]), x.clone()
    g.f16_to_i8(x, q1, a1)
    g.gemm_i8(q1, w1, h, a1, s1, ACT)
    q2, a2 = torch.empty(h.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
    g.f16_to_i8(h, q2, a2)
    g.gemm_i8(q2, w2, y, a2, s2, beta=1.0)
    return y


def main(H=256, I=512, T=512, steps=20, rate=0.1):
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda")
    master = [draw(H, 2 * I) * H ** -0.5, draw(I, H) * I ** -0.5]
    target = [(w + 0.3 * draw(*w.shape) * w.shape[0] ** -0.5).half() for w in master]
    grads = [torch.empty_like(w) for w in master]
    losses = []
    for _ in range(steps):
        w1, w2 = (w.half() for w in master)
        loss = 0.0
        for micro in range(2):
            x = draw(T, H).half()
            h, y = forward(x, w1, w2)
            off = (y - forward(x, *target)[1]).float()
            loss += float((off * off).mean()) / 2
            backward(x, w1, w2, h, (off / T).half(), *grads, first=micro == 0)
        losses.append(loss)
        for w, dw in zip(master, grads):
            w -= rate * dw
    w1, w2 = (w.half() for w in master)
    x = draw(32, H).half()
    exact = forward(x, w1, w2)[1].float()
    in_8_bits = serve(x, *rounded(w1), *rounded(w2)).float()
    off = float((in_8_bits - exact).norm() / (exact - x.float()).norm())
    torch.cuda.synchronize()
    assert g.debug_status() == 0
    print("loss %.4f -> %.4f; 32 tokens in 8 bits are %.2f%% of the block's own output off"
          % (losses[0], losses[-1], 100 * off))
    return {"losses": losses, "off": off, "grads": grads, "weights": (w1, w2), "target": target}


if __name__ == "__main__":
    main()
