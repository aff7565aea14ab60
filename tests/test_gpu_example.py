"""examples/mlp_block.py against the block's definition in 64 bits, its MXFP8
and MXFP4 roundings passed through."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import mlp_block  # noqa: E402

import mxfp4_precision_gemms_amd as A  # noqa: E402
from test_gpu_linear import DEV, decode, decode4, rand  # noqa: E402

pytestmark = pytest.mark.gpu


class _Held(torch.autograd.Function):
    """A value in the forward pass, the identity in the backward."""

    @staticmethod
    def forward(ctx, x, value):
        return value

    @staticmethod
    def backward(ctx, g):
        return g, None


@pytest.mark.parametrize("weights", ["MXFP8", "MXFP4"])
@pytest.mark.parametrize("T,D,F", [(1, 64, 96), (37, 128, 256), (300, 256, 544)])
def test_block(T, D, F, weights):
    gain = (1 + rand(D, seed=1, std=0.1)).to(torch.bfloat16)
    gate_up = rand(2 * F, D, seed=2, std=D ** -0.5, dtype=torch.bfloat16)
    down = rand(D, F, seed=3, std=F ** -0.5, dtype=torch.bfloat16)
    x, stream = rand(T, D, seed=4, dtype=torch.bfloat16), rand(T, D, seed=5, std=2.0, dtype=torch.bfloat16)
    dout = rand(T, D, seed=6, dtype=torch.bfloat16)
    block = mlp_block.MlpBlock(gain.to(DEV), gate_up.to(DEV), down.to(DEV), weights)
    out, saved = block.forward(x.to(DEV), stream.to(DEV), train=True)
    grads = block.backward(dout.to(DEV), saved)
    n, a = saved

    # The definition, with the values that the formats hold in their places
    # (forward's weights quantized, backward's as they are).
    de = decode if weights == "MXFP8" else decode4
    s = stream.double().requires_grad_()
    g, wgu, wd = (t.double().requires_grad_() for t in (gain, gate_up, down))
    h = _Held.apply(s + x.double(), n.h.cpu().double())
    y = _Held.apply(h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-5) * g, decode(n.codes, n.scales))
    z = _Held.apply(y @ wgu.t(), decode(n.codes, n.scales) @ de(*block.gate_up_mx).t())
    act = _Held.apply(torch.nn.functional.silu(z[:, :F]) * z[:, F:], decode(a.out, a.scales))
    want = decode(a.out, a.scales) @ de(*block.down_mx).t() + n.h.cpu().double()
    (act @ wd.t() + h).backward(dout.double())

    def close(got, ref, roundings):
        # bf16 roundings of up to 2^-8 each in a row, in the root mean square
        assert float((got.cpu().double() - ref).norm()) <= roundings * 2.0 ** -8 * float(ref.norm())

    close(out, want, 1)
    # z's, dact's, dz's (and dy's) rounding before each result's own
    dstream, dgain, dgate_up, ddown = grads
    close(ddown, wd.grad, 1)
    close(dgate_up, wgu.grad, 4)
    close(dgain, g.grad, 5)
    close(dstream, s.grad, 5)


def test_block_serves_as_it_trains():
    D, F = 128, 256
    args = [t.to(DEV) for t in (torch.ones(D, dtype=torch.bfloat16),
                                rand(2 * F, D, seed=7, dtype=torch.bfloat16),
                                rand(D, F, seed=8, dtype=torch.bfloat16))]
    block = mlp_block.MlpBlock(*args, weights="MXFP4")
    x, s = (rand(5, D, seed=k, dtype=torch.bfloat16).to(DEV) for k in (9, 10))
    assert torch.equal(block.forward(x, s)[0], block.forward(x, s, train=True)[0])
