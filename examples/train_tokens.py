"""A small selective state-space language model, trained on synthetic tokens with this package's operators.

    python examples/train_tokens.py [--steps 200] [--state-bits 8]

One layer as in the pages' block: tokens are embedded straight into [B, E, L], two halves of an input projection make x
and the gate z, the causal conv + SiLU makes u, a projection of u makes the step size, B and C, the selective scan
runs over the sequence, an output projection goes back to the model's width, and the table gives the logits of the
next token.  The embedding, the conv, the scan, all their gradients and the optimizer are HIP kernels of the
package; the projections are torch matrix products in the same [B, channels, L] layout.

The data: sequences over an alphabet in which a token repeats what stood `lag` positions before, with some noise.  A
model without memory cannot do better than the alphabet's entropy; the loss falls well below it.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_76_amd as ssm  # noqa: E402


def project(w, x):
    """w [O, I] times every column of x [B, I, L], as one product of two matrices: [B, O, L]."""
    B, n, L = x.shape
    return (w @ x.transpose(0, 1).reshape(n, B * L)).view(-1, B, L).transpose(0, 1).contiguous()


class Model:
    """Parameters in bf16 but for the scan's A, D and bias and the conv, which their kernels take in fp32."""

    def __init__(self, rows, width, inner, dstate, rank, device, seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def matrix(n, m, gain=1.0):
            return (torch.randn(n, m, generator=g) * gain / math.sqrt(m)).to(device, torch.bfloat16)

        self.dims = (rank, dstate)
        p = {"table": matrix(rows, width), "in_x": matrix(inner, width), "in_z": matrix(inner, width),
             "to_ssm": matrix(rank + 2 * dstate, inner), "to_dt": matrix(inner, rank), "out": matrix(width, inner, 0.5)}
        f = {"conv_w": (torch.rand(inner, 4, generator=g) - 0.5), "conv_b": torch.zeros(inner),
             "A_log": torch.arange(1, dstate + 1).float().log().repeat(inner, 1), "D": torch.ones(inner),
             # step sizes from 1e-3 to 1e-1, through the inverse of the softplus
             "dt_bias": torch.expm1(torch.empty(inner).uniform_(math.log(1e-3), math.log(1e-1), generator=g).exp()).log()}
        p.update({k: v.to(device) for k, v in f.items()})
        self.p = {k: v.requires_grad_(True) for k, v in p.items()}

    def logits(self, tokens):
        p, (rank, n) = self.p, self.dims
        e = ssm.embedding(tokens, p["table"], scale=math.sqrt(p["table"].shape[1]), channels_first=True)  # [B,E,L]
        x, z = project(p["in_x"], e), project(p["in_z"], e)
        u, _ = ssm.causal_conv1d(x, p["conv_w"], p["conv_b"])
        s = project(p["to_ssm"], u)
        delta = project(p["to_dt"], s[:, :rank])
        Bm, Cm = s[:, rank:rank + n].contiguous(), s[:, rank + n:].contiguous()
        y, _ = ssm.selective_scan(u, delta, -p["A_log"].exp(), Bm, Cm, p["D"], z, p["dt_bias"])
        h = e + project(p["out"], y)
        h = h * torch.rsqrt(h.float().square().mean(1, keepdim=True) + 1e-6).to(h.dtype)
        return project(p["table"], h).transpose(1, 2).float()  # [B,L,V]


def batch(rows, B, L, lag, g, device):
    t = torch.randint(0, rows, (B, L + 1), generator=g)
    for i in range(lag, L + 1):
        t[:, i] = torch.where(torch.rand(B, generator=g) < 0.9, t[:, i - lag], t[:, i])
    return t[:, :-1].to(device), t[:, 1:].to(device)


def train(steps=200, state_bits=32, rows=16, width=64, inner=128, dstate=16, lag=3, B=8, L=128, device="cuda", say=print):
    """Returns the losses of all steps."""
    model = Model(rows, width, inner, dstate, 8, device)
    opt = ssm.AdamW(model.p.values(), lr=3e-3, betas=(0.9, 0.99), weight_decay=0.01, state_bits=state_bits,
                    max_grad_norm=1.0)
    g = torch.Generator().manual_seed(1)
    losses = []
    for k in range(steps):
        tokens, wanted = batch(rows, B, L, lag, g, device)
        loss = torch.nn.functional.cross_entropy(model.logits(tokens).reshape(-1, rows), wanted.reshape(-1))
        for p in model.p.values():
            p.grad = None
        loss.backward()
        norm = opt.step()
        losses.append(loss.detach())
        if k % 20 == 0 or k == steps - 1:
            say("step %4d  loss %.4f  gradient norm %.3f  (without memory: %.4f)" % (k, losses[-1], norm, math.log(rows)))
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    train(a.steps, a.state_bits)
