"""The row-routed products together, as a server and a trainer of one decoder
block would call them.

    python examples/adapters_and_experts.py

A block here is a projection with the low-rank adapters of many requests beside
it (gemm_f16_lora) and a mixture-of-experts layer added onto its input
(gemm_f16_moe with beta = 1, the residual).  The program

1. runs a prompt of three requests, each with its own adapter, through the
   projection, then decodes single tokens for all three at once: the decoding
   rows equal what the same rows of a prompt give;
2. trains the three adapters together, the projection frozen, with
   gemm_f16_lora_grad (two micro-batches accumulated with beta = 1), until each
   has learned its own target map.

Prints what it measured; returns a dict of the same when called as main().
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dense_gemm_03_gb300 as g


def block(x, p, ids):
    """One block on rows x whose requests' adapters are ids; returns the new
    hidden rows and the experts each row took."""
    M, H = x.shape
    y = torch.empty((M, H), dtype=torch.float16, device=x.device)
    g.gemm_f16_lora(x, p["W"], y, p["A"], p["B"], ids, p["scales"])
    out = y.clone()                                      # the residual, y + experts(y)
    experts = torch.empty((M, p["topk"]), dtype=torch.int32, device=x.device)
    g.gemm_f16_moe(y, p["Wr"], p["W1"], p["W2"], out, p["topk"], ids=experts, beta=1.0)
    return out, experts


def parameters(H, I, E, topk, R, adapters, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).half()

    return dict(W=normal(H, H, std=H ** -0.5), A=normal(adapters, H, R, std=H ** -0.5),
                B=normal(adapters, R, H, std=0.3), scales=torch.ones(adapters, device="cuda"),
                Wr=normal(H, E, std=H ** -0.5), W1=normal(E, H, 2 * I, std=H ** -0.5),
                W2=normal(E, I, H, std=I ** -0.5), topk=topk)


def serve(H=512, lengths=(40, 75, 60)):
    """Prompt rows of three requests, then their last tokens again as a decoding
    batch of three: the largest difference between the two."""
    p = parameters(H, I=256, E=8, topk=2, R=16, adapters=3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((sum(lengths), H), generator=gen, device="cuda").half()
    ids = torch.repeat_interleave(torch.arange(3), torch.tensor(lengths)).int().cuda()
    prompt, took = block(x, p, ids)
    last = torch.cumsum(torch.tensor(lengths), 0).cuda() - 1
    decoded, took1 = block(x[last].contiguous(), p, ids[last].contiguous())
    same = (took[last] == took1).all(dim=1)    # a near tie may choose another expert
    diff = (prompt[last].float() - decoded.float())[same].abs().max().item()
    return {"rows": sum(lengths), "decode_difference": diff, "same_experts": int(same.sum())}


def train(H=256, N=320, R=8, adapters=3, rows=192, steps=60, lr=0.05):
    """Each adapter learns the difference to its own target map from rows of a
    mixed batch; mean squared error before and after."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    W = (torch.randn((H, N), generator=gen, device="cuda") * H ** -0.5).half()
    A = torch.randn((adapters, H, R), generator=gen, device="cuda") * H ** -0.5
    B = torch.zeros((adapters, R, N), device="cuda")
    target = [torch.randn((H, 4), generator=gen, device="cuda") @
              torch.randn((4, N), generator=gen, device="cuda") * 0.5 * H ** -0.5
              for _ in range(adapters)]
    scales = torch.full((adapters,), 2.0, device="cuda")
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    mA, mB = [torch.zeros_like(A), torch.zeros_like(A)], [torch.zeros_like(B), torch.zeros_like(B)]
    losses = []
    for step in range(steps):
        total = 0.0
        for micro in range(2):
            x = torch.randn((rows, H), generator=gen, device="cuda").half()
            ids = torch.randint(0, adapters, (rows,), generator=gen, device="cuda").int()
            want = x.float() @ W.float()
            for a in range(adapters):
                want[ids == a] += x[ids == a].float() @ target[a]
            y = torch.empty((rows, N), dtype=torch.float16, device="cuda")
            Ah, Bh = A.half(), B.half()
            g.gemm_f16_lora(x, W, y, Ah, Bh, ids, scales)
            err = y.float() - want
            total += (err ** 2).mean().item() / 2
            # no dX: this is the first layer
            g.gemm_f16_lora_grad((err / rows).half(), x, W, Ah, Bh, ids, scales, dA=dA, dB=dB,
                                 beta=float(micro > 0))
        losses.append(total)
        for w, d, (m, v) in ((A, dA, mA), (B, dB, mB)):   # Adam
            m.mul_(0.9).add_(d, alpha=0.1)
            v.mul_(0.99).addcmul_(d, d, value=0.01)
            mh, vh = m / (1 - 0.9 ** (step + 1)), v / (1 - 0.99 ** (step + 1))
            w.sub_(lr * mh / (vh.sqrt() + 1e-8))
    return {"loss_before": losses[0], "loss_after": losses[-1]}


def main():
    r = {**serve(), **train()}
    torch.cuda.synchronize()
    assert g.debug_status() == 0
    return r


if __name__ == "__main__":
    for k, v in main().items():
        print("%-18s %s" % (k, v))
