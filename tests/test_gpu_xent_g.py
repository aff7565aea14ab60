"""How the cross entropy's gradient holds that of the logits, g: as two bf16 numbers
(SPLIT) or one (BF16).

Tolerances beyond those derived in test_gpu_xent.py (u = 2^-24): the nearest bf16
is off by at most 2^-8 |g|; what it leaves is exact in fp32 (a number of 24 bits less
its first 8), and the nearest bf16 to that is off by at most 2^-8 of it: 2^-16 |g|
together. SPLIT's sums have twice the terms, whose magnitudes add up to at most (1 +
2^-7) |g|. What lies below fp32's (and bf16's) smallest normal number, m = 2^-126, may
count as 0: an exponential, which takes |dloss + dlse| |scale| m from g; g; and its
second number; and a product or sum of dh and dw, 2 (n + 1) of them. (Logits 1e3 apart
have probabilities of 1e-90 and below, which no fp32 number stands for.)"""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_xent import DEV, U, case, check, logits, say
from tile_cases import DH, DW, flat

pytestmark = pytest.mark.gpu
M = 2.0 ** -126


def gradients(h, w, y, lse, dloss, dlse, scale, dt, g):
    """dh, dw in 64 bits and how far each may be off."""
    z, ez = logits(h, w, scale)
    V = w.shape[0]
    there = (y >= 0) & (y < V)
    own = torch.where(there, dloss.double(), torch.zeros_like(dloss, dtype=torch.float64))
    every = own if dlse is None else own + dlse.double()
    x = z - lse.double()[:, None]
    p = x.exp()
    hot = torch.zeros_like(z).scatter_(1, y.clamp(0, V - 1)[:, None], 1.0)
    gz = scale * (every[:, None] * p - own[:, None] * hot)
    # the exponential of an argument that is off by e is off by e^e - 1 of itself
    eg = abs(scale) * every.abs()[:, None] * p * torch.expm1(ez[:, None] + (4 + 3 * x.abs()) * U)
    eg = eg + 4 * U * abs(scale) * own[:, None].abs() * hot
    step = 2.0 ** -16 if g == "SPLIT" else 2.0 ** -8
    eg = eg * (1 + step) + step * gz.abs() + M * (abs(scale) * every.abs()[:, None] + 2)
    terms = 2 * (1 + 2.0 ** -7) if g == "SPLIT" else 1 + 2.0 ** -8
    hd, wd = h.double(), w.double()
    half = torch.finfo(dt).eps / 2
    dh, dw = gz @ wd, gz.t() @ hd
    eh = eg @ wd.abs() + terms * (V + 2) * U * (gz.abs() @ wd.abs())
    ew = eg.t() @ hd.abs() + terms * (h.shape[0] + 2) * U * (gz.abs().t() @ hd.abs())
    eh, ew = eh + 2 * (V + 1) * M, ew + 2 * (h.shape[0] + 1) * M
    return dh, dw, eh * (1 + half) + half * dh.abs(), ew * (1 + half) + half * dw.abs()


# short sums, whose own rounding leaves g's to be seen; tiles of 64, 128 and 256 rows
SIZES = [(1, 1, 8), (1, 300, 64), (3, 5, 8), (17, 16, 128), (130, 200, 264), (255, 256, 128), (257, 511, 136)]


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", ["SPLIT", "BF16"])
def test_precision(T, V, D, dt, g):
    say("g", T, V, D, dt, g)
    h, w, y, dloss, dlse = case(T, V, D, seed=T + V + 2)
    lse = torch.logsumexp(logits(h, w, 0.8)[0], 1).float()
    more = {} if g == "SPLIT" else {"g": g}                    # SPLIT is what a call without g takes
    dh, dw = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, scale=0.8, dh_dtype=dt, dw_dtype=dt, **more)
    rh, rw, eh, ew = gradients(h, w, y, lse, dloss, dlse, 0.8, dt, g)
    check("dh", dh, rh, eh)
    check("dw", dw, rw, ew)


def whole_numbers(T, V, D, seed):
    """Inputs whose logits are all 0 and lse 0, so that g_tv is dloss_t + dlse_t less,
    at the target, dloss_t: whole numbers of 16 bits. w has values in the first half
    of the columns, h in the second, at most 127 of +-1 in each: all sums are whole
    numbers below 2^23, exact in any order."""
    gen = torch.Generator().manual_seed(seed)

    def sparse(rows, first, last):
        m = torch.zeros(rows, D)
        n = min(rows, 127)
        at = torch.stack([torch.randperm(rows, generator=gen)[:n] for _ in range(min(8, last - first))], 1)
        cols = torch.arange(first, last)
        m[at[:, cols % at.shape[1]], cols] = torch.randint(0, 2, (n, last - first), generator=gen).float() * 2 - 1
        return m.to(torch.bfloat16).to(DEV)

    half = D // 16 * 8
    w, h = sparse(V, 0, half), sparse(T, half, D)
    y = torch.randint(-3, V, (T,), generator=gen)
    dlse = torch.randint(1, 1 << 15, (T,), generator=gen).float()
    dloss = torch.randint(1, 1 << 15, (T,), generator=gen).float()
    return h, w, y.to(DEV), dloss.to(DEV), dlse.to(DEV)


@pytest.mark.parametrize("which,c", [("dh", c) for c in flat(DH)] + [("dw", c) for c in flat(DW)])
@pytest.mark.parametrize("g", ["SPLIT", "BF16"])
def test_every_tile_exactly(which, c, g):
    """Both numbers of every element reach their sums once, in every tile, whole and
    in parts."""
    T, V, D = c
    say("exactly", which, T, V, D, g)
    h, w, y, dloss, dlse = whole_numbers(T, V, D, seed=T + V)
    dh, dw = A.adahop_xent_backward(h, w, y, torch.zeros(T, device=DEV), dloss, dlse, g=g, dh_dtype=torch.float32,
                                    dw_dtype=torch.float32, h_grad=which == "dh", w_grad=which == "dw")
    there = (y >= 0).float()
    each, at = dlse + there * dloss, dlse                     # elsewhere, at the target
    if g == "BF16":
        each, at = each.to(torch.bfloat16).float(), at.to(torch.bfloat16).float()
    hot = torch.zeros(T, V, dtype=torch.float64, device=DEV).scatter_(1, y.clamp(min=0)[:, None], there.double()[:, None])
    less = (at - each).double()[:, None] * hot
    if which == "dh":
        want = each.double()[:, None] * w.double().sum(0) + less @ w.double()
        got = dh
    else:
        want = (each.double()[:, None] * h.double()).sum(0) + less.t() @ h.double()
        got = dw
    assert float(want.abs().amax()) > 1000 and torch.equal(got.double(), want)


@pytest.mark.parametrize("T,V,D,piece", [(70, 1300, 72, 256), (513, 1300, 136, 1024), (300, 2049, 520, 512)])
def test_pieces_exactly(T, V, D, piece):
    say("pieces exactly", T, V, D, piece)
    h, w, y, dloss, dlse = whole_numbers(T, V, D, seed=T)
    both = [A.adahop_xent_backward(h, w, y, torch.zeros(T, device=DEV), dloss, dlse, dh_dtype=torch.float32,
                                   dw_dtype=torch.float32, piece=p) for p in (0, piece)]
    for a, b in zip(*both):
        assert float(a.abs().amax()) > 1000 and torch.equal(a, b)


@pytest.mark.parametrize("T,V,D,piece", [(40, 1000, 72, 256), (513, 1300, 136, 1024)])
def test_one_number_in_pieces(T, V, D, piece):
    h, w, y, dloss, dlse = case(T, V, D, seed=T + piece)
    lse = torch.logsumexp(logits(h, w, 1.0)[0], 1).float()
    a = A.XentBackwardArgs(T, V, D, 16, D, 16, D, 16, 16, 16, None, 16, D, 16, D, piece, 1.0, 1, 1, 0, g=A.XENT_G["BF16"])
    need = A.lib().adahop_xent_backward_args_workspace_size(a)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    dh, dw = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, dh_dtype=torch.float32, piece=piece, g="BF16", ws=ws)
    assert bool((ws[need:] == 0xA5).all())
    rh, _, eh, _ = gradients(h, w, y, lse, dloss, dlse, 1.0, torch.float32, "BF16")
    _, rw, _, ew = gradients(h, w, y, lse, dloss, dlse, 1.0, torch.bfloat16, "BF16")
    check("dh", dh, rh, eh)
    check("dw", dw, rw, ew)
    again = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, dh_dtype=torch.float32, piece=piece, g="BF16")
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


def test_past_the_largest_bf16():
    """An element of g between bf16's largest number and fp32's: infinite in bf16, and
    not a NaN for what that leaves."""
    h = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(1, 8, dtype=torch.bfloat16, device=DEV)
    far = torch.full((1,), 3.4e38, device=DEV)
    y, zero = torch.tensor([-1], device=DEV), torch.zeros(1, device=DEV)
    for g in ("SPLIT", "BF16"):
        dh, _ = A.adahop_xent_backward(h, w, y, zero, zero, far, g=g, dh_dtype=torch.float32)
        assert bool((dh == float("inf")).all())


@pytest.mark.parametrize("g", ["SPLIT", "BF16"])
def test_targets_of_32_bits(g):
    h, w, y, dloss, dlse = case(300, 2049, 136, seed=13)
    lse = A.adahop_xent(h, w, y).lse
    both = [A.adahop_xent_backward(h, w, t, lse, dloss, dlse, g=g) for t in (y, y.to(torch.int32))]
    for a, b in zip(*both):
        assert torch.equal(a, b)


def test_in_a_graph():
    """Both ways captured with a workspace each, replayed together on new inputs with
    eager work between."""
    T, V, D = 200, 5000, 264
    h, w, y, dloss, dlse = case(T, V, D, seed=14)
    lse = A.adahop_xent(h, w, y).lse
    held, graphs = [], []
    for g in ("SPLIT", "BF16"):
        a = A.XentBackwardArgs(T, V, D, 16, D, 16, D, 16, 16, 16, None, 16, D, 16, D, 1024, 1.0, 1, g=A.XENT_G[g])
        ws = torch.empty(A.lib().adahop_xent_backward_args_workspace_size(a), dtype=torch.uint8, device=DEV)
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            A.adahop_xent_backward(h, w, y, lse, dloss, dlse, dh=dh, dw=dw, piece=1024, ws=ws, g=g)
        graphs.append(graph)
        held.append((g, dh, dw, ws))
    for s in (15, 16, 17):
        for to, new in zip((h, w, y, dloss, dlse), case(T, V, D, seed=s)):
            to.copy_(new)
        lse.copy_(A.adahop_xent(h, w, y).lse)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for g, dh, dw, _ in held:
            want = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, piece=1024, g=g)
            assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])
            dh.zero_(), dw.zero_()
        torch.cuda.synchronize()
