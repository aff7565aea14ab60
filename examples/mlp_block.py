"""A pre-norm gated MLP block on microscaled operands, forward and backward.

forward:   h = stream + x;  y = rmsnorm(h) * gain, in MXFP8
           a = silu(y Wg^T) * (y Wu^T), in MXFP8;  out = a Wd^T + h
backward:  the gradients of the stream, of x (the same), of the norm's gain and
           of both weight matrices, with MXFP8's and MXFP4's roundings passed
           through; the products of gradients are adahop_gemm's input and weight
           gradients, on any of its routes.

    python examples/mlp_block.py [--dim 4096] [--hidden 14336] [--weights MXFP4]

times a decoding step of one token, a prompt and a training step on one GPU.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_precision_gemms_amd as A  # noqa: E402


class MlpBlock:
    def __init__(self, gain, gate_up, down, weights="MXFP8", eps=1e-5):
        """gain [D]; gate_up [2 F, D] (gate rows, then up rows) and down [D, F], bf16."""
        self.gain, self.gate_up, self.down, self.eps = gain, gate_up, down, eps
        self.gate_up_mx, self.down_mx = (self.quantize(w, weights) for w in (gate_up, down))

    @staticmethod
    def quantize(w, weights):
        if weights == "MXFP8":
            return A.adahop_mx8_quant(w)
        return A.adahop_iht_quant(w, "COLS", hadamard_block=0)[:2]

    def forward(self, x, stream, train=False):
        """The stream after the block, and what backward needs."""
        n = A.adahop_rmsnorm(x, self.gain, stream, eps=self.eps, save_rstd=train)
        a = A.adahop_linear_mx((n.codes, n.scales), self.gate_up_mx, act="SILU", gated=True,
                               out_dtype="MXFP8", save_z=train)
        out = A.adahop_linear_mx((a.out, a.scales), self.down_mx, residual=n.h).out
        return out, (n, a) if train else None

    def backward(self, dout, saved, route="BF16"):
        """From the gradient of the stream after the block: those of the stream
        before it (and of x), the gain, gate_up and down."""
        n, a = saved
        dact = A.adahop_gemm("DGRAD", dout, self.down, route=route)
        ddown = A.adahop_gemm("WGRAD", dout, A.adahop_mx8_dequant(a.out, a.scales), route=route)
        dz, _ = A.adahop_act_backward(dact, a.z, act="SILU", gated=True)
        dy = A.adahop_gemm("DGRAD", dz, self.gate_up, route=route)
        dgate_up = A.adahop_gemm("WGRAD", dz, A.adahop_mx8_dequant(n.codes, n.scales), route=route)
        dstream, dgain = A.adahop_rmsnorm_backward(dy, n.h, self.gain, n.rstd, dout)
        return dstream, dgain, dgate_up, ddown


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
    p.add_argument("--hidden", type=int, default=14336)
    p.add_argument("--weights", choices=("MXFP8", "MXFP4"), default="MXFP4")
    p.add_argument("--tokens", type=int, default=4096)
    o = p.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    block = MlpBlock(1 + normal(o.dim, std=0.1), normal(2 * o.hidden, o.dim, std=0.02),
                     normal(o.dim, o.hidden, std=0.02), o.weights)
    for tokens in (1, 32, o.tokens):
        x, stream = normal(tokens, o.dim, std=0.5), normal(tokens, o.dim)
        ms = _time(lambda: block.forward(x, stream), 20)
        print(f"forward, {tokens} tokens: {ms * 1e3:.1f} us")
    dout = normal(o.tokens, o.dim, std=1e-3)

    def step():
        _, saved = block.forward(x, stream, train=True)
        return block.backward(dout, saved)

    print(f"forward and backward, {o.tokens} tokens: {_time(step, 5):.3f} ms")


if __name__ == "__main__":
    main()
