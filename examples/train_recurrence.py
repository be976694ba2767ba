"""A small language model of residual blocks around the gated linear recurrence, trained on synthetic tokens, and then
writing some of its own.

    python examples/train_recurrence.py [--steps 200] [--layers 2] [--dropout 0.1]

Tokens are embedded straight into [B, E, L]; that is the stream.  Every block normalises it (with the branch of the block
before added on the way, and dropped out in training), projects it to the recurrence's input, its two gates and an output
gate, runs the causal conv and the recurrence over the sequence and projects back.  The embedding, the norms with their
dropout, the conv, the recurrence, all their gradients and the optimizer are HIP kernels of the package; the projections
are torch matrix products.

Writing takes one token at a time: the conv's and the recurrence's states are all that is kept of what was written.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_76_amd as ssm  # noqa: E402
from train_tokens import batch, project  # noqa: E402


class Model:
    """Parameters in bf16 but for those that the kernels take in fp32."""

    def __init__(self, rows, width, inner, layers, device, dropout=0.0, seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.layers, self.inner, self.dropout = layers, inner, dropout

        def matrix(n, m, gain=1.0):
            return (torch.randn(n, m, generator=g) * gain / math.sqrt(m)).to(device, torch.bfloat16)

        self.p = {"table": matrix(rows, width), "norm": torch.ones(width, device=device)}
        for k in range(layers):
            self.p.update({
                "norm%d" % k: torch.ones(width, device=device), "in%d" % k: matrix(4 * inner, width),
                "out%d" % k: matrix(width, inner, 0.5), "conv_w%d" % k: (torch.rand(inner, 4, generator=g) - 0.5).to(device),
                "conv_b%d" % k: torch.zeros(inner, device=device),
                # memories from three to a thousand steps at gates of 1/2
                "decay%d" % k: torch.linspace(math.log(0.7), math.log(2e-3), inner, device=device),
                "r_bias%d" % k: torch.zeros(inner, device=device), "i_bias%d" % k: torch.zeros(inner, device=device)})
        for t in self.p.values():
            t.requires_grad_(True)

    def scale(self):
        return math.sqrt(self.p["table"].shape[1])

    def logits(self, tokens, seed=None):
        """[B, L, V]; seed: of the dropout, None for none."""
        p, drop = self.p, dict(p=self.dropout, seed=seed) if seed is not None and self.dropout else {}
        hidden = ssm.embedding(tokens, p["table"], scale=self.scale(), dtype=torch.float32, channels_first=True)
        branch = None
        for k in range(self.layers + 1):
            w = p["norm%d" % k] if k < self.layers else p["norm"]
            if branch is None:
                y = ssm.layer_norm(hidden, w, rms=True, channels_first=True).bfloat16()
            else:
                y, hidden = ssm.layer_norm(branch, w, None, hidden, rms=True, channels_first=True, call=k, **drop)
            if k == self.layers:
                return project(p["table"], y).transpose(1, 2).float()
            x, r, i, z = (t.contiguous() for t in project(p["in%d" % k], y).split(self.inner, 1))
            u, _ = ssm.causal_conv1d(x, p["conv_w%d" % k], p["conv_b%d" % k])
            h, _ = ssm.gated_recurrence(u, r, i, p["decay%d" % k].exp(), p["r_bias%d" % k], p["i_bias%d" % k], z)
            branch = project(p["out%d" % k], h)

    @torch.no_grad()
    def states(self, B):
        """What writing keeps, for B sequences: the conv's and the recurrence's state of every layer."""
        d = self.p["norm"].device
        return [(torch.zeros(B, self.inner, 3, dtype=torch.bfloat16, device=d), torch.zeros(B, self.inner, device=d))
                for _ in range(self.layers)]

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits [B, V] of the tokens [B] that come next, the states taken one token on."""
        p = self.p
        hidden = ssm.embedding_fwd(tokens, p["table"], scale=self.scale(), dtype=torch.float32)
        branch = None
        for k in range(self.layers + 1):
            w = p["norm%d" % k] if k < self.layers else p["norm"]
            if branch is None:
                y = ssm.layer_norm_fwd(hidden, w, rms=True, stats=False)[0].bfloat16()
            else:
                y, hidden, _ = ssm.layer_norm_fwd(branch, w, None, hidden, rms=True, stats=False)
            if k == self.layers:
                return (y @ p["table"].t()).float()
            x, r, i, z = (t.contiguous() for t in (y @ p["in%d" % k].t()).split(self.inner, 1))
            conv, state = states[k]
            u = ssm.conv1d_update(conv, x, p["conv_w%d" % k], p["conv_b%d" % k])
            h = ssm.recurrence_update(state, u, r, i, p["decay%d" % k].exp(), p["r_bias%d" % k], p["i_bias%d" % k], z)
            branch = h @ p["out%d" % k].t()


def train(steps=200, layers=2, dropout=0.1, rows=16, width=64, inner=64, lag=3, B=8, L=128, device="cuda", say=print):
    """(the model, the losses of all steps)."""
    model = Model(rows, width, inner, layers, device, dropout)
    opt = ssm.AdamW(model.p.values(), lr=3e-3, betas=(0.9, 0.99), weight_decay=0.01, max_grad_norm=1.0)
    g = torch.Generator().manual_seed(1)
    losses = []
    for k in range(steps):
        tokens, wanted = batch(rows, B, L, lag, g, device)
        loss = torch.nn.functional.cross_entropy(model.logits(tokens, seed=k).reshape(-1, rows), wanted.reshape(-1))
        for p in model.p.values():
            p.grad = None
        loss.backward()
        norm = opt.step()
        losses.append(loss.detach())
        if k % 20 == 0 or k == steps - 1:
            say("step %4d  loss %.4f  gradient norm %.3f  (without memory: %.4f)" % (k, losses[-1], norm, math.log(rows)))
    return model, [float(x) for x in losses]


def write(model, tokens, count):
    """The most likely `count` tokens behind tokens [B, L], one at a time."""
    states, out = model.states(tokens.shape[0]), []
    for t in range(tokens.shape[1]):
        logits = model.step(tokens[:, t].contiguous(), states)
    for _ in range(count):
        out.append(logits.argmax(1))
        logits = model.step(out[-1], states)
    return torch.stack(out, 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--dropout", type=float, default=0.1)
    a = ap.parse_args()
    model, _ = train(a.steps, a.layers, a.dropout)
    start = batch(16, 1, 24, 3, torch.Generator().manual_seed(5), "cuda")[0]
    print("behind", start[0].tolist(), "the model writes", write(model, start, 12)[0].tolist())
