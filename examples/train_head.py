"""Training a head on frozen convolution features, per pixel.

A convolution layer with fixed weights gives features (channels innermost); the
head is a layer norm over the channels, dropout, and a linear classifier of
every pixel under softmax cross entropy. The head's parameters are trained with
plain SGD in fp32; the classifier's products run in the features' type.

    python examples/train_head.py [--steps 60] [--classes 200] [--dtype bf16]

The data is synthetic: every pixel's class picks one of a few random
patterns that the frozen layer sees through noise.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import cnn_convolution_amd as conv


class PixelHead:
    """layer norm -> dropout -> linear classifier with softmax cross entropy."""

    def __init__(self, channels, classes, dtype, device, dropout_p=0.1, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.gamma = torch.ones(channels, device=device)
        self.beta = torch.zeros(channels, device=device)
        self.w = torch.randn(classes, channels, generator=gen, device=device) * channels ** -0.5
        self.dtype, self.p = dtype, dropout_p

    def loss(self, features, labels):
        """Mean loss over the labelled pixels (labels outside [0, classes) are
        ignored), without dropout."""
        z, _, _ = conv.layer_norm(features, self.gamma, self.beta)
        loss, _ = conv.linear_cross_entropy(z.reshape(-1, z.shape[-1]), self.w.to(self.dtype), labels)
        return loss.sum() / ((labels >= 0) & (labels < self.w.shape[0])).sum()

    def step(self, features, labels, lr, lr_norm, seed):
        """One SGD step (lr_norm for the layer norm's parameters); returns the mean loss before it (with dropout). The
        dropout mask is a function of the seed and is made again for the
        backward pass."""
        drop = dict(dropout_p=self.p, seed=seed)
        z, mean, rstd = conv.layer_norm(features, self.gamma, self.beta, **drop)
        rows, w = z.reshape(-1, z.shape[-1]), self.w.to(self.dtype)
        loss, lse = conv.linear_cross_entropy(rows, w, labels)
        count = ((labels >= 0) & (labels < w.shape[0])).sum()
        # half-precision gradients are scaled into the type's range
        scale = 1024.0 if self.dtype is torch.float16 else 1.0
        grad = (scale / count).expand(labels.numel()).float().contiguous()
        dz, dw = conv.linear_cross_entropy_backward(grad, rows, w, labels, lse)
        _, dgamma, dbeta = conv.layer_norm_backward(dz.reshape(z.shape), features, self.gamma, mean, rstd, **drop)
        for param, g, rate in ((self.w, dw, lr), (self.gamma, dgamma, lr_norm), (self.beta, dbeta, lr_norm)):
            param.sub_(g.float(), alpha=rate / scale)
        return loss.sum() / count


def make_batch(patterns, n, size, gen, device):
    """Images [n][3][size][size] whose pixels show their class's pattern, and
    int64 labels per pixel with the border unlabelled."""
    classes = patterns.shape[0]
    labels = torch.randint(0, classes, (n, size, size), generator=gen, device=device)
    x = patterns[labels].permute(0, 3, 1, 2) + 0.1 * torch.randn(n, patterns.shape[1], size, size, generator=gen,
                                                                 device=device)
    labels[:, 0, :] = labels[:, -1, :] = labels[:, :, 0] = labels[:, :, -1] = -1
    return x.contiguous(), labels.reshape(-1)


def train(steps=60, classes=200, dtype=torch.bfloat16, channels=256, lr=2.0, lr_norm=0.1, seed=1,
          device="cuda"):
    """Losses of the training steps, and the loss of a held-out batch before and after."""
    gen = torch.Generator(device=device).manual_seed(seed)
    patterns = torch.randn(classes, 8, generator=gen, device=device)
    # the frozen layer: channels-innermost output in the training type
    filt = torch.randn(channels, 1, 1, 8, generator=gen, device=device).to(dtype)

    def features(x):
        x = x.permute(0, 2, 3, 1).contiguous().to(dtype)
        return conv.conv2d(x, filt, out_dtype=dtype, layout="nhwc")

    if dtype is torch.float32:                      # the channels-innermost layout takes half precision only
        filt = filt.reshape(channels, 8, 1, 1)

        def features(x):                            # noqa: F811
            return conv.conv2d(x, filt).permute(0, 2, 3, 1).contiguous()

    head = PixelHead(channels, classes, dtype, device, seed=seed)
    held, held_labels = make_batch(patterns, 4, 32, gen, device)
    held = features(held)
    before = head.loss(held, held_labels).item()
    losses = []
    for k in range(steps):
        x, labels = make_batch(patterns, 8, 32, gen, device)
        losses.append(head.step(features(x), labels, lr, lr_norm, seed=k))
    return [v.item() for v in losses], before, head.loss(held, held_labels).item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--classes", type=int, default=200)
    ap.add_argument("--dtype", choices=["f32", "f16", "bf16"], default="bf16")
    a = ap.parse_args()
    types = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
    losses, before, after = train(a.steps, a.classes, types[a.dtype])
    for k in range(0, len(losses), 10):
        print(f"step {k:4d}  loss {losses[k]:.4f}")
    print(f"held-out loss {before:.4f} -> {after:.4f}")
