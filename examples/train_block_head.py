"""Training a head with residual gated feed-forward blocks on convolution features,
by AdamW.

Features (rows of channels, as a channels-innermost convolution leaves them) go through
a layer norm and `blocks` blocks, each a gated feed-forward block on the normalised
rows whose output is normalised, gated and added to the residual stream, and a linear
classifier under softmax cross entropy. The residual stream and the parameters are fp32,
the products run in `dtype`; the optimizer's states have 8 bits, and it leaves the
products' copies of the weights with each step.

    python examples/train_block_head.py [--steps 60] [--classes 200] [--dtype bf16]

The data is synthetic: every pixel's class picks one of a few random patterns that a
frozen convolution layer sees through noise.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import cnn_convolution_amd as conv


class BlockHead:
    """layer norm -> blocks of (feed-forward, norm, gate, residual sum, norm) -> classifier."""

    def __init__(self, channels, hidden, classes, blocks, dtype, device, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def rnd(*shape):
            return torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5
        vec = lambda value: torch.full((channels,), value, device=device)      # noqa: E731
        self.dtype, self.blocks = dtype, blocks
        # norms and gates first, then the products' weights; 4 vectors and 3 matrices a block
        self.vectors = [vec(1.0), vec(0.0)] + [v for _ in range(blocks) for v in (vec(0.5), vec(1.0), vec(1.0), vec(0.0))]
        self.weights = [w for _ in range(blocks)
                        for w in (rnd(hidden, channels), rnd(hidden, channels), rnd(channels, hidden))] + [rnd(classes, channels)]
        self.params = self.vectors + self.weights
        self.copies = None if dtype is torch.float32 else [w.to(dtype) for w in self.weights]
        self.state = conv.adamw_state(self.params, bits=8)
        self.step_number = 0

    def gradients(self, x, labels):
        """(mean loss over the labelled rows, gradients of the parameters) for rows x."""
        w = self.weights if self.copies is None else self.copies
        v = self.vectors
        scale = 1024.0 if self.dtype is torch.float16 else 1.0      # half-precision gradients in the type's range
        x = x.float()
        h, mean, rstd = conv.layer_norm(x, v[0], v[1], out_dtype=self.dtype)
        stream, kept = x, []
        for k in range(self.blocks):
            gate, post, weight, bias = v[2 + 4 * k:6 + 4 * k]
            args = dict(gate=gate, post_weight=post, weight=weight)
            y, saved = conv.feed_forward(h, *w[3 * k:3 * k + 3])
            out, z, stats = conv.residual_norm(y, stream, bias=bias, **args)
            kept.append((h, y, saved, out, stats, args))
            stream, h = out, z
        loss, lse = conv.linear_cross_entropy(h, w[-1], labels)
        count = ((labels >= 0) & (labels < w[-1].shape[0])).sum()
        grad = (scale / count).expand(labels.numel()).float().contiguous()
        dh, dw = conv.linear_cross_entropy_backward(grad, h, w[-1], labels, lse)
        dvec, dmat, dstream = [], [dw], None
        for k in reversed(range(self.blocks)):
            h, y, saved, out, stats, args = kept[k]
            dstream, dy, g = conv.residual_norm_backward(dh, dstream, y, out, stats, **args)
            dh, *dff = conv.feed_forward_backward(dy, h, *w[3 * k:3 * k + 3], saved)
            dvec, dmat = [g["gate"], g["post_weight"], g["weight"], g["bias"]] + dvec, dff + dmat
        _, dgamma, dbeta = conv.layer_norm_backward(dh, x, v[0], mean, rstd)
        grads = [dgamma, dbeta] + dvec + dmat
        self.scale = scale
        return loss.sum() / count, grads if scale == 1.0 else [g.float() / scale for g in grads]

    def step(self, x, labels, lr):
        loss, grads = self.gradients(x, labels)
        self.step_number += 1
        decay = [0.0] * len(self.vectors) + [0.01] * len(self.weights)
        copies = None if self.copies is None else [None] * len(self.vectors) + self.copies
        conv.adamw(self.params, grads, self.state, self.step_number, lr, weight_decay=decay, copies=copies, seed=1)
        return loss


def train(steps=60, classes=200, dtype=torch.bfloat16, channels=256, hidden=512, blocks=2, lr=3e-3, seed=1, device="cuda"):
    """Losses of the training steps."""
    gen = torch.Generator(device=device).manual_seed(seed)
    patterns = torch.randn(classes, 8, generator=gen, device=device)
    filt = torch.randn(channels, 8, 1, 1, generator=gen, device=device)
    head = BlockHead(channels, hidden, classes, blocks, dtype, device, seed)
    losses = []
    for _ in range(steps):
        labels = torch.randint(0, classes, (4, 32, 32), generator=gen, device=device)
        x = patterns[labels].permute(0, 3, 1, 2).contiguous()
        x = x + 0.1 * torch.randn(x.shape, generator=gen, device=device)
        labels[:, 0, :] = labels[:, -1, :] = labels[:, :, 0] = labels[:, :, -1] = -1     # the border is unlabelled
        rows = conv.conv2d(x, filt).permute(0, 2, 3, 1).reshape(-1, channels)
        losses.append(head.step(rows, labels.reshape(-1), lr))
    return [v.item() for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--classes", type=int, default=200)
    ap.add_argument("--dtype", choices=["f32", "f16", "bf16"], default="bf16")
    a = ap.parse_args()
    types = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
    for k, loss in enumerate(train(a.steps, a.classes, types[a.dtype])):
        if k % 10 == 0 or k + 1 == a.steps:
            print(f"step {k:4d}  loss {loss:.4f}")
