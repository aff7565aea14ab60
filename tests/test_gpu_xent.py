"""Cross entropy over a vocabulary and its gradient against their definitions in
64 bits.

Tolerances, from the arithmetic (u = 2^-24, fp32's half step; products of bf16
values are exact in fp32):
  logit   |z - z*| <= Ez = (D + 2) u |scale| max_v sum_d |h w|: a sum of D terms in
          any order, the scale's rounding and the result's.
  exp     argument x = z - top: u |x| for its rounding, twice that again for the
          constant log2(e) and the product, one ulp (2 u) of the instruction;
          |x| e^x <= 0.37, so over a sum of terms <= 1 they weigh at most
          (2 + 3 * 0.37 * number of terms / sum) u; each term's own weight is
          bounded here by its value with X = max |x| instead: (2 + 3 X) u relative.
  lse     Ez + the sum's relative error, ((2 + 3 X) + V / 1024 + 64) u (16 terms a
          lane, 2 joins, V / 1024 + 6 joins of parts with an exponential each: two
          roundings a join are in the 64 and in X), + 4 u (|lse| + |top| + 1) for
          the logarithm and the last addition.
  loss    lse's + Ez + u |loss|.
  g       bf16's half step 2^-8 of |g|, and before it |dloss + dlse| |scale| p times
          (Ez + (4 + 3 X) u) + 4 u |dloss scale|.
  dh, dw  sum |dg| |w| + (n + 2) u sum |g| |w| over n terms, and the output's half
          step (bf16 2^-8, fp32 u).
"""
import math

import pytest
import torch

import mxfp4_precision_gemms_amd as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def say(*a):
    print(*a, flush=True)


def strided(t, pad, before=0):
    """t as rows of a larger buffer, the last of which ends with it."""
    if not pad:
        return t.to(DEV)
    rows, cols = t.shape
    flat = torch.full((before + (rows - 1) * (cols + pad) + cols,), float("nan"), dtype=t.dtype, device=DEV)
    v = flat[before:].as_strided((rows, cols), (cols + pad, 1))
    v.copy_(t)
    return v


def case(T, V, D, seed=0, wstd=None, ignored=0.2, pad_h=0, pad_w=0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, D, generator=g) * (wstd or 2 / math.sqrt(D))).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g)
    lean = 10 * torch.rand(T, 1, generator=g) / w[y].float().square().sum(1, keepdim=True).clamp(min=1e-6)
    h = (torch.randn(T, D, generator=g) + lean * w[y].float()).to(torch.bfloat16)
    out = torch.rand(T, generator=g) < ignored
    y = torch.where(out, torch.where(torch.rand(T, generator=g) < 0.5, -100, V), y)
    dloss = torch.rand(T, generator=g) + 0.5
    dlse = torch.randn(T, generator=g) * 0.1
    return strided(h, pad_h), strided(w, pad_w), y.to(DEV), dloss.to(DEV), dlse.to(DEV)


def logits(h, w, scale):
    h, w = h.double(), w.double()
    z = scale * (h @ w.t())
    ez = (h.shape[1] + 2) * U * abs(scale) * (h.abs() @ w.abs().t()).amax(1)
    return z, ez


def expected(h, w, y, scale):
    """(loss, lse) and how far each may be off."""
    z, ez = logits(h, w, scale)
    V = w.shape[0]
    lse = torch.logsumexp(z, 1)
    there = (y >= 0) & (y < V)
    loss = torch.where(there, lse - z.gather(1, y.clamp(0, V - 1)[:, None])[:, 0], torch.zeros_like(lse))
    top = z.amax(1)
    X = top - z.amin(1)
    el = ez + ((2 + 3 * X) + V / 1024 + 64) * U + 4 * U * (lse.abs() + top.abs() + 1)
    return loss, lse, torch.where(there, el + ez + U * loss.abs(), torch.zeros_like(el)), el


def check(name, got, want, tol):
    d = (got.double() - want).abs()
    say(f"  {name}: at most {float((d / tol.clamp(min=1e-300)).nan_to_num(0).amax()) if d.numel() else 0:.3f} "
        f"of the tolerance")
    assert bool((d <= tol).all()), name


def gradients(h, w, y, lse, dloss, dlse, scale, dt):
    z, ez = logits(h, w, scale)
    V = w.shape[0]
    there = (y >= 0) & (y < V)
    own = torch.where(there, dloss.double(), torch.zeros_like(dloss, dtype=torch.float64))
    every = own if dlse is None else own + dlse.double()
    x = z - lse.double()[:, None]
    p = x.exp()
    hot = torch.zeros_like(z)
    hot.scatter_(1, y.clamp(0, V - 1)[:, None], 1.0)
    g = scale * (every[:, None] * p - own[:, None] * hot)
    eg = abs(scale) * every.abs()[:, None] * p * (ez[:, None] + (4 + 3 * x.abs()) * U)
    eg = eg + 4 * U * abs(scale) * own[:, None].abs() * hot
    eg = eg * (1 + 2.0 ** -8) + 2.0 ** -8 * g.abs()
    hd, wd = h.double(), w.double()
    half = torch.finfo(dt).eps / 2
    dh, dw = g @ wd, g.t() @ hd
    eh = eg @ wd.abs() + (V + 2) * U * (g.abs() @ wd.abs())
    ew = eg.t() @ hd.abs() + (h.shape[0] + 2) * U * (g.abs().t() @ hd.abs())
    return dh, dw, eh * (1 + half) + half * dh.abs(), ew * (1 + half) + half * dw.abs()


# T, V, D: one of each, ragged tiles, D past one stage and inside a pair of
# stages, several rounds of tiles (more than 256), a long vocabulary
SIZES = [(1, 1, 8), (1, 300, 64), (2, 257, 72), (3, 5, 8), (17, 16, 128), (255, 256, 128), (257, 511, 136),
         (130, 1000, 200), (300, 2049, 520), (64, 70001, 64), (513, 25700, 72), (1025, 769, 1032)]


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("scale", [1.0, -0.7])
def test_forward(T, V, D, scale):
    say("xent", T, V, D, scale)
    h, w, y, _, _ = case(T, V, D, seed=T + V)
    got = A.adahop_xent(h, w, y, scale=scale)
    torch.cuda.synchronize()
    loss, lse, e_loss, e_lse = expected(h, w, y, scale)
    check("lse", got.lse, lse, e_lse)
    check("loss", got.loss, loss, e_loss)
    again = A.adahop_xent(h, w, y.to(torch.int32), scale=scale)
    assert torch.equal(again.loss, got.loss) and torch.equal(again.lse, got.lse)


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_backward(T, V, D, dt):
    say("xent_backward", T, V, D, dt)
    h, w, y, dloss, dlse = case(T, V, D, seed=T + V + 1)
    dlse = dlse if dt == torch.float32 else None
    scale = 0.8 if dt == torch.float32 else 1.0
    lse = torch.logsumexp(logits(h, w, scale)[0], 1).float()
    dh, dw = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, scale=scale, dh_dtype=dt, dw_dtype=dt)
    torch.cuda.synchronize()
    rh, rw, eh, ew = gradients(h, w, y, lse, dloss, dlse, scale, dt)
    check("dh", dh, rh, eh)
    check("dw", dw, rw, ew)


@pytest.mark.parametrize("T,V,D,piece", [(40, 1000, 72, 256), (300, 2049, 520, 512), (70, 4097, 64, 1),
                                         (513, 1300, 136, 1024), (9, 70001, 264, 20000)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_backward_in_pieces(T, V, D, piece, dt):
    say("pieces", T, V, D, piece, dt)
    h, w, y, dloss, dlse = case(T, V, D, seed=T + piece)
    lse = torch.logsumexp(logits(h, w, 1.0)[0], 1).float()
    dh, dw = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, dh_dtype=dt, dw_dtype=dt, piece=piece)
    rh, rw, eh, ew = gradients(h, w, y, lse, dloss, dlse, 1.0, dt)
    check("dh", dh, rh, eh)
    check("dw", dw, rw, ew)


@pytest.mark.parametrize("T,V,D,pad", [(5, 300, 72, 8), (300, 513, 136, 24), (257, 70001, 64, 8)])
def test_rows_apart(T, V, D, pad):
    """Rows of h, w, dh and dw with NaNs between them, whose memory ends with the
    last row; nothing between the outputs' rows changes."""
    say("rows apart", T, V, D, pad)
    h, w, y, dloss, dlse = case(T, V, D, seed=9, pad_h=pad, pad_w=2 * pad)
    loss, lse, e_loss, e_lse = expected(h, w, y, 1.0)
    got = A.adahop_xent(h, w, y)
    check("lse", got.lse, lse, e_lse)
    check("loss", got.loss, loss, e_loss)
    out = {}
    for k, n, dt in (("dh", T, torch.bfloat16), ("dw", V, torch.float32)):
        buf = torch.full((n, D + 3), -7.0, dtype=dt, device=DEV)
        out[k] = buf[:, 1:D + 1]
    dh, dw = A.adahop_xent_backward(h, w, y, got.lse, dloss, dlse, dh=out["dh"], dw=out["dw"], piece=256)
    rh, rw, eh, _ = gradients(h, w, y, got.lse, dloss, dlse, 1.0, torch.bfloat16)
    ew = gradients(h, w, y, got.lse, dloss, dlse, 1.0, torch.float32)[3]
    check("dh", dh, rh, eh)
    check("dw", dw, rw, ew)
    for v in (dh, dw):
        base = v._base
        assert bool((base[:, 0] == -7).all() and (base[:, D + 1:] == -7).all())


@pytest.mark.parametrize("which", ["dh", "dw"])
def test_one_gradient_alone(which):
    h, w, y, dloss, _ = case(70, 900, 136, seed=3)
    lse = A.adahop_xent(h, w, y).lse
    both = A.adahop_xent_backward(h, w, y, lse, dloss, piece=256)
    one = A.adahop_xent_backward(h, w, y, lse, dloss, piece=256, h_grad=which == "dh", w_grad=which == "dw")
    k = 0 if which == "dh" else 1
    assert one[1 - k] is None and torch.equal(one[k], both[k])


def test_no_rows():
    h = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones((33, 64), dtype=torch.bfloat16, device=DEV)
    y, e = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    got = A.adahop_xent(h, w, y)
    assert got.loss.shape == (0,) and got.lse.shape == (0,)
    for dt in (torch.bfloat16, torch.float32):
        dw = torch.full((33, 64), 5.0, dtype=dt, device=DEV)
        dh, dw = A.adahop_xent_backward(h, w, y, e, e, dw=dw)
        assert dh.shape == (0, 64) and bool((dw == 0).all())
    assert A.adahop_xent_backward(h, w, y, e, e, w_grad=False)[0].shape == (0, 64)


def test_every_row_left_out():
    h, w, y, dloss, _ = case(33, 600, 64, seed=4)
    for bad in (-1, 600, -100, 2 ** 40, -(2 ** 40)):
        y.fill_(bad)
        got = A.adahop_xent(h, w, y)
        loss, lse, _, e_lse = expected(h, w, y, 1.0)
        assert bool((got.loss == 0).all())
        check("lse", got.lse, lse, e_lse)
        for d in A.adahop_xent_backward(h, w, y, got.lse, dloss):
            assert bool((d == 0).all())


def test_infinities_and_nans():
    """Row 0 has a logit of +inf, row 1 of NaN, row 2 all of -inf; the others
    are as without them."""
    T, V, D = 70, 700, 64
    h, w, y, _, _ = case(T, V, D, seed=5, ignored=0.0)
    h[:, 0] = 0.0
    w[:, 0] = 0.0
    plain = A.adahop_xent(h[3:], w, y[3:])
    w[:, 0] = 1.0
    h[0, 0], h[2, 0] = float("inf"), float("-inf")
    h[1, 1] = float("nan")
    got = A.adahop_xent(h, w, y)
    z = h.float() @ w.float().t()
    want = torch.logsumexp(z, 1)
    say(got.lse[:3], want[:3], got.loss[:3])
    assert got.lse[0] == float("inf") and torch.isnan(got.lse[1]) and got.lse[2] == float("-inf")
    assert torch.isnan(got.loss[:3]).all()
    assert torch.equal(got.lse[3:], plain.lse) and torch.equal(got.loss[3:], plain.loss)


def test_large_logits():
    """Logits of +-1e4: no exponential overflows."""
    T, V, D = 65, 515, 64
    h, w, y, dloss, _ = case(T, V, D, seed=6, wstd=50.0)
    h = (h.float() * 30).to(torch.bfloat16)
    loss, lse, e_loss, e_lse = expected(h, w, y, 1.0)
    assert float(lse.abs().amax()) > 1e4
    got = A.adahop_xent(h, w, y)
    check("lse", got.lse, lse, e_lse)
    check("loss", got.loss, loss, e_loss)
    assert all(torch.isfinite(d).all() for d in A.adahop_xent_backward(h, w, y, got.lse, dloss))


def test_gradient_against_differences():
    """Along a random direction of h and of w, the central difference of the
    summed loss in 64 bits is the inner product with the gradient: both within
    the difference's own error (h^2 / 6 times the third derivative, below 1e-6
    here) and the gradient's tolerance."""
    T, V, D = 20, 90, 40
    h, w, y, dloss, dlse = case(T, V, D, seed=7)
    lse = A.adahop_xent(h, w, y).lse
    dh, dw = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, dh_dtype=torch.float32, dw_dtype=torch.float32)
    _, _, eh, ew = gradients(h, w, y, lse, dloss, dlse, 1.0, torch.float32)

    def total(hd, wd):
        z = hd @ wd.t()
        s = torch.logsumexp(z, 1)
        there = (y >= 0) & (y < V)
        own = torch.where(there, s - z.gather(1, y.clamp(0, V - 1)[:, None])[:, 0], 0 * s)
        return (own * dloss.double() + s * dlse.double()).sum()

    gen = torch.Generator().manual_seed(8)
    eps = 1e-4
    for grad, err, at in ((dh, eh, 0), (dw, ew, 1)):
        v = [torch.zeros(T, D, dtype=torch.float64, device=DEV), torch.zeros(V, D, dtype=torch.float64, device=DEV)]
        v[at] = torch.randn(grad.shape, generator=gen).double().to(DEV)
        up, down = (total(h.double() + s * v[0], w.double() + s * v[1]) for s in (eps, -eps))
        slope, got = (up - down) / (2 * eps), (grad.double() * v[at]).sum()
        assert abs(slope - got) <= (err * v[at].abs()).sum() + 1e-4 * (1 + abs(slope))


def test_workspace_of_the_callers():
    h, w, y, dloss, _ = case(70, 3000, 264, seed=10)
    want = A.adahop_xent(h, w, y)
    need = A.lib().adahop_xent_workspace_size(70, 3000)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    got = A.adahop_xent(h, w, y, ws=ws)
    assert torch.equal(got.loss, want.loss) and bool((ws[need:] == 0xA5).all())
    with pytest.raises(A.AdahopError):
        A.adahop_xent(h, w, y, ws=ws[:need - 1])
    for piece in (0, 512):
        a = A.XentBackwardArgs(70, 3000, 264, 16, 264, 16, 264, 16, 16, 16, None, 16, 264, 16, 264, piece, 1.0, 1)
        need = A.lib().adahop_xent_backward_args_workspace_size(a)
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        both = A.adahop_xent_backward(h, w, y, want.lse, dloss, piece=piece, ws=ws)
        assert bool((ws[need:] == 0xA5).all())
        for x, z in zip(both, A.adahop_xent_backward(h, w, y, want.lse, dloss, piece=piece)):
            assert torch.equal(x, z)
        with pytest.raises(A.AdahopError):
            A.adahop_xent_backward(h, w, y, want.lse, dloss, piece=piece, ws=ws[:need - 1])


def test_graph_and_streams():
    """Captured on a side stream and replayed on new inputs, two graphs with
    workspaces of their own, and a call on another stream beside them."""
    T, V, D = 200, 5000, 264
    h, w, y, dloss, _ = case(T, V, D, seed=11)
    fresh = [case(T, V, D, seed=s) for s in (12, 13, 14)]
    a = A.XentBackwardArgs(T, V, D, 16, D, 16, D, 16, 16, 16, None, 16, D, 16, D, 1024, 1.0, 1)
    sizes = A.lib().adahop_xent_workspace_size(T, V), A.lib().adahop_xent_backward_args_workspace_size(a)
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r = A.adahop_xent(h, w, y, ws=ws[0])
            A.adahop_xent_backward(h, w, y, r.lse, dloss, dh=dh, dw=dw, piece=1024, ws=ws[1])
        graphs.append((graph, r, dh, dw, ws))
    for nh, nw, ny, nd, _ in fresh:
        for to, new in ((h, nh), (w, nw), (y, ny), (dloss, nd)):
            to.copy_(new)
        want = A.adahop_xent(h, w, y)
        wh, ww = A.adahop_xent_backward(h, w, y, want.lse, dloss, piece=1024)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for (graph, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        beside = A.adahop_xent(h, w, y)
        torch.cuda.synchronize()
        assert torch.equal(beside.lse, want.lse)
        for _, r, dh, dw, _ in graphs:
            assert torch.equal(r.loss, want.loss) and torch.equal(r.lse, want.lse)
            assert torch.equal(dh, wh) and torch.equal(dw, ww)
            dh.zero_(), dw.zero_(), r.loss.zero_()
