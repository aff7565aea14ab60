"""The end of a language model's training step: the last norm, the output layer and
the cross entropy, forward and backward, without the logits.

forward:   h = stream + x;  y = rmsnorm(h) * gain;  loss = mean of the cross entropy
           of y W^T over the rows with a target, plus z_loss times the mean square
           of its normalizer (the logarithm of the exponentials' sum)
backward:  the gradients of the stream (and of x, the same), of the gain and of W.

    python examples/lm_head.py [--dim 4096] [--vocab 131072] [--tokens 8192]

times a training step and the scoring of one token on one GPU.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_precision_gemms_amd as A  # noqa: E402


class LmHead:
    def __init__(self, gain, w, eps=1e-5, z_loss=0.0):
        """gain [D]; w [V, D], bf16."""
        self.gain, self.w, self.eps, self.z_loss = gain, w, eps, z_loss

    def forward(self, x, stream, targets):
        """(loss, what backward needs); targets int64 [T], one outside 0 .. V - 1: left out."""
        n = A.adahop_rmsnorm(x, self.gain, stream, eps=self.eps, mx8=False, bf16=True, save_rstd=True)
        r = A.adahop_xent(n.y, self.w, targets)
        counts = ((targets >= 0) & (targets < self.w.shape[0])).float()
        total = counts.sum().clamp(min=1)
        loss = (r.loss.sum() + self.z_loss * (r.lse.square() * counts).sum()) / total
        return loss, (n, r.lse, targets, counts / total)

    def backward(self, saved):
        n, lse, targets, share = saved
        dlse = 2 * self.z_loss * lse * share if self.z_loss else None
        dy, dw = A.adahop_xent_backward(n.y, self.w, targets, lse, share, dlse)
        dstream, dgain = A.adahop_rmsnorm_backward(dy, n.h, self.gain, n.rstd)
        return dstream, dgain, dw


def _time(f, n):
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--dim", type=int, default=4096)
    p.add_argument("--vocab", type=int, default=131072)
    p.add_argument("--tokens", type=int, default=8192)
    o = p.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    head = LmHead(1 + normal(o.dim, std=0.1), normal(o.vocab, o.dim, std=o.dim ** -0.5), z_loss=1e-4)
    for tokens in (1, o.tokens):
        x, stream = normal(tokens, o.dim, std=0.5), normal(tokens, o.dim)
        targets = torch.randint(0, o.vocab, (tokens,), generator=gen, device="cuda")
        ms = _time(lambda: head.forward(x, stream, targets), 10)
        print(f"forward, {tokens} tokens: {ms * 1e3:.1f} us")
    print(f"forward and backward, {o.tokens} tokens: "
          f"{_time(lambda: head.backward(head.forward(x, stream, targets)[1]), 5):.3f} ms")


if __name__ == "__main__":
    main()
