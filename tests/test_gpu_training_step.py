"""A training step's end and a block with MXFP8 checkpoints, run together as they
would be (examples/lm_head.py, examples/mlp_block.py), against their formulas in 64
bits at the values that the formats hold."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import lm_head  # noqa: E402
import mlp_block  # noqa: E402

import mxfp4_precision_gemms_amd as A  # noqa: E402
from test_gpu_linear import DEV, act_ref, decode, norm_back_ref, rand  # noqa: E402

pytestmark = pytest.mark.gpu


def close(got, ref, roundings):
    # bf16 roundings of up to 2^-8 each in a row, in the root mean square
    assert float((got.cpu().double() - ref).norm()) <= roundings * 2.0 ** -8 * float(ref.norm())


def block_of(D, F, checkpoints, seed=1):
    gain = (1 + rand(D, seed=seed, std=0.1)).to(torch.bfloat16)
    gate_up = rand(2 * F, D, seed=seed + 1, std=D ** -0.5, dtype=torch.bfloat16)
    down = rand(D, F, seed=seed + 2, std=F ** -0.5, dtype=torch.bfloat16)
    return gain, gate_up, down, mlp_block.MlpBlock(gain.to(DEV), gate_up.to(DEV), down.to(DEV), checkpoints=checkpoints)


@pytest.mark.parametrize("T,D,F", [(1, 64, 96), (37, 128, 256), (300, 256, 544)])
def test_block_with_checkpoints(T, D, F):
    gain, gate_up, down, block = block_of(D, F, "MXFP8")
    x, stream = rand(T, D, seed=4, dtype=torch.bfloat16), rand(T, D, seed=5, std=2.0, dtype=torch.bfloat16)
    dout = rand(T, D, seed=6, dtype=torch.bfloat16)
    out, saved = block.forward(x.to(DEV), stream.to(DEV), train=True)
    plain = block_of(D, F, "BF16")[3]
    assert torch.equal(out, plain.forward(x.to(DEV), stream.to(DEV))[0])
    dstream, dgain, dgate_up, ddown = block.backward(dout.to(DEV), saved)
    y, rstd, h8, z8 = saved
    h, z = decode(*h8), decode(*z8)
    # what is kept lies within MXFP8's half step (2^-4 of a value, 2^-10 of a
    # block's scale, which is at most 2^-7 of its largest) of what was
    n = A.adahop_rmsnorm(x.to(DEV), gain.to(DEV), stream.to(DEV))
    ref = n.h.cpu().double()
    top = ref.abs().view(T, -1, 32).amax(2).repeat_interleave(32, 1)
    assert bool(((h - ref).abs() <= ref.abs() * 2.0 ** -4 + top * 2.0 ** -17).all())
    f, slope = act_ref(z[:, :F], "SILU")
    dact = dout.double() @ down.double()
    dz = torch.cat((dact * z[:, F:] * slope, dact * f), 1)
    dx, _, dg, _ = norm_back_ref(dz @ gate_up.double(), h, gain, rstd.cpu(), dout)
    close(ddown, dout.double().t() @ (f * z[:, F:]), 2)          # out's rounding, then its own
    close(dgate_up, dz.t() @ decode(*y), 3)                      # dact's, dz's, its own
    close(dgain, dg, 4)                                          # and dy's
    close(dstream, dx, 4)


@pytest.mark.parametrize("z_loss", [0.0, 1e-2])
@pytest.mark.parametrize("T,V,D", [(1, 33, 64), (37, 1000, 128), (300, 5003, 256)])
def test_head(T, V, D, z_loss):
    gain = (1 + rand(D, seed=11, std=0.1)).to(torch.bfloat16)
    w = rand(V, D, seed=12, std=2 * D ** -0.5, dtype=torch.bfloat16)
    x, stream = rand(T, D, seed=13, dtype=torch.bfloat16), rand(T, D, seed=14, std=2.0, dtype=torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(15))
    if T > 1:
        y[::7] = -100
    head = lm_head.LmHead(gain.to(DEV), w.to(DEV), z_loss=z_loss)
    loss, saved = head.forward(x.to(DEV), stream.to(DEV), y.to(DEV))
    dstream, dgain, dw = head.backward(saved)
    n = saved[0]
    yd = n.y.cpu().double().requires_grad_()
    wd = w.double().requires_grad_()
    z = yd @ wd.t()
    lse = torch.logsumexp(z, 1)
    there = (y >= 0).double()
    own = lse - z.gather(1, y.clamp(min=0)[:, None])[:, 0]
    want = (there * (own + z_loss * lse.square())).sum() / there.sum()
    want.backward()
    assert abs(float(loss) - float(want)) <= 1e-5 * (1 + abs(float(want)))
    dx, _, dg, _ = norm_back_ref(yd.grad, n.h.cpu(), gain, n.rstd.cpu(), None)
    close(dw, wd.grad, 2)                                        # the logits' gradient's rounding, its own
    close(dgain, dg, 3)
    close(dstream, dx, 3)


@pytest.mark.parametrize("z_loss", [0.0, 1e-2])
@pytest.mark.parametrize("T,V,D", [(2, 33, 64), (37, 1000, 128)])
def test_head_with_targets_past_the_vocabulary(T, V, D, z_loss):
    """Padding by a number past the vocabulary's last is padding as -100 is: the same
    loss and the same gradients."""
    gain = (1 + rand(D, seed=51, std=0.1)).to(torch.bfloat16).to(DEV)
    w = rand(V, D, seed=52, std=2 * D ** -0.5, dtype=torch.bfloat16).to(DEV)
    x, stream = (rand(T, D, seed=s, dtype=torch.bfloat16).to(DEV) for s in (53, 54))
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(55)).to(DEV)
    head = lm_head.LmHead(gain, w, z_loss=z_loss)
    got = []
    for padding in (-100, V, 2 ** 40):
        y[::2] = padding
        loss, saved = head.forward(x, stream, y)
        got.append([loss, *head.backward(saved)])
    assert float(got[0][0]) > 0
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_step_in_a_graph():
    """Block, head and their gradients captured together, replayed on new inputs
    with eager work between, equal the eager step."""
    T, V, D, F = 130, 2003, 128, 256
    block = block_of(D, F, "MXFP8", seed=21)[3]
    head = lm_head.LmHead(torch.ones(D, device=DEV, dtype=torch.bfloat16),
                          rand(V, D, seed=24, std=0.2, dtype=torch.bfloat16).to(DEV), z_loss=1e-3)
    x, stream = (rand(T, D, seed=s, dtype=torch.bfloat16).to(DEV) for s in (25, 26))
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(27)).to(DEV)

    def step():
        out, saved = block.forward(x, stream, train=True)
        n = A.adahop_rmsnorm(out, head.gain, mx8=False, bf16=True, save_rstd=True)
        r = A.adahop_xent(n.y, head.w, y)
        share = torch.full_like(r.loss, 1 / T)
        dy, dw = A.adahop_xent_backward(n.y, head.w, y, r.lse, share, 1e-3 * share * r.lse)
        dout, dgain = A.adahop_rmsnorm_backward(dy, out, head.gain, n.rstd)
        return [r.loss, r.lse, dw, dgain, *block.backward(dout, saved)]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.copy_(rand(T, D, seed=30 + k, dtype=torch.bfloat16))
        y.copy_(torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(40 + k)))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(held, step()):
            assert torch.equal(got, want), k
        torch.cuda.synchronize()
