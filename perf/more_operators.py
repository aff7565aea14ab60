"""Cases of the operators that end a training step and save its memory.

Softmax cross entropy over a large vocabulary from hidden states and output
weights, without the logits, and its gradient; and backward passes that read
activations kept in MXFP8 (E4M3 elements, one E8M0 scale per 32): of the linear
layer's activation, of the RMS norm, and of a linear layer's weight. `run`
computes them in elementary torch operations, or, with `own`, with the
package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _xent(T, V, D, scale=1.0, **more):
    return dict(op="xent", T=T, V=V, D=D, scale=scale, **more)


def _xent_grad(T, V, D, scale=1.0, zloss=False, **more):
    return dict(op="xent_grad", T=T, V=V, D=D, scale=scale, zloss=zloss, **more)


def _act_grad(m, n, act, gated=False, bias=False, remake=False, **more):
    return dict(op="act_grad", m=m, n=n, act=act, gated=gated, bias=bias, remake=remake, **more)


def _norm_grad(rows, cols, stream="bf16", dh=True, **more):
    return dict(op="norm_grad", rows=rows, cols=cols, stream=stream, dh=dh, **more)


def _weight_grad(T, Din, Dout, out="bf16", **more):
    return dict(op="weight_grad", T=T, Din=Din, Dout=Dout, out=out, **more)


def listed():
    return [
        # scoring one token of a small model
        _xent(1, 32000, 2048, name="xent_token"),
        # scoring a ragged batch, an odd vocabulary, logits at a temperature
        _xent(333, 50021, 2080, scale=0.8, name="xent_ragged"),
        # training: two sequences of 4096 tokens at a width of 4096, a large vocabulary
        _xent(8192, 131072, 4096, name="xent_train"),
        # fine-tuning a small head on a few tokens
        _xent_grad(37, 8191, 1032, name="xent_grad_few"),
        # a ragged micro-batch with the square of the normalizer in its loss
        _xent_grad(1531, 50021, 2048, zloss=True, name="xent_grad_ragged"),
        # training: two sequences of 4096 tokens, a large vocabulary
        _xent_grad(8192, 131072, 4096, name="xent_grad_train"),
        # training, 4 sequences: the gated activation of Llama3.1-8B, whose output is made again
        _act_grad(16384, 14336, "SILU", gated=True, remake=True, name="act_grad_gated"),
        # a ragged batch through an ordinary layer with bias
        _act_grad(2050, 8160, "GELU", bias=True, name="act_grad_bias"),
        # training, Llama3.2-1B's width, with the residual path's gradient
        _norm_grad(16384, 2048, name="norm_grad"),
        # a ragged micro-batch with the residual stream in 32 bits
        _norm_grad(3001, 4096, stream="f32", name="norm_grad_ragged_f32"),
        # training: the down-projection of Llama3.1-8B over 8 sequences of 4096 tokens
        _weight_grad(32768, 14336, 4096, name="weight_grad_train"),
        # a ragged micro-batch, kept in 32 bits to be added to
        _weight_grad(1531, 2080, 1032, out="f32", name="weight_grad_ragged_f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("xent", "xent", "xent_grad", "xent_grad", "act_grad", "norm_grad", "weight_grad"))
    if op in ("xent", "xent_grad"):
        D, V = 8 * _log(rng, 16, 1024), _log(rng, 1000, 131072)
        T = max(1, min(_log(rng, 1, 8192), 2 ** 42 // (V * D)))
        scale = rng.choice((1.0, 1.0, 0.8, 1.25))
        if op == "xent":
            return _xent(T, V, D, scale=scale)
        return _xent_grad(T, V, D, scale=scale, zloss=rng.random() < 0.4)
    if op == "act_grad":
        gated, n = rng.random() < 0.5, 32 * _log(rng, 2, 448)
        return _act_grad(min(_log(rng, 1, 16384), 16384 * 14336 // n), n,
                         rng.choice(("SILU", "GELU", "GELU_TANH", "RELU")), gated=gated,
                         bias=rng.random() < 0.5, remake=rng.random() < 0.5)
    if op == "norm_grad":
        cols = 32 * _log(rng, 2, 256)
        return _norm_grad(min(_log(rng, 1, 32768), 16384 * 2048 // cols), cols,
                          stream=rng.choice(("bf16", "f32")), dh=rng.random() < 0.8)
    Din, Dout = 32 * _log(rng, 2, 448), 8 * _log(rng, 8, 1024)
    T = max(1, min(_log(rng, 1, 32768), 32768 * 14336 * 4096 // (Din * Dout)))
    return _weight_grad(T, Din, Dout, out=rng.choice(("bf16", "bf16", "f32")))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    def activations(rows, cols):
        """Normal values, 1 % of the columns 30 times as large."""
        v = torch.randn(rows, cols, generator=gen, device=DEV)
        lines = torch.randint(0, cols, (max(1, cols // 100),), generator=gen, device=DEV)
        v[:, lines] *= 30.0
        return v

    s = {"case": case}
    if case["op"] in ("xent", "xent_grad"):
        T, V, D = case["T"], case["V"], case["D"]
        s["w"] = normal(V, D, std=2.0 / math.sqrt(D), dtype=torch.bfloat16)
        y = torch.randint(0, V, (T,), generator=gen, device=DEV)
        # hidden states that lean towards their token, some of them surely
        wy = s["w"][y].float()
        lean = 14.0 * uniform(T, 1) / wy.square().sum(1, keepdim=True)
        s["h"] = (normal(T, D) + lean * wy).to(torch.bfloat16)
        # a tenth of the rows is padding
        s["y"] = torch.where(uniform(T) < 0.1, torch.full_like(y, -100), y) if T > 1 else y
        if case["op"] == "xent_grad":
            s["lse"] = torch.logsumexp(case["scale"] * torch.matmul(s["h"].float(), s["w"].float().t()), 1)
            count = (s["y"] >= 0).sum().clamp(min=1)
            s["dloss"] = (0.5 + uniform(T)) / count
            s["dlse"] = 2e-4 * s["lse"] / count if case["zloss"] else None
    elif case["op"] == "act_grad":
        m, n = case["m"], case["n"]
        s["z"] = _pack_mxfp8(normal(m, 2 * n if case["gated"] else n, std=1.5))
        s["dout"] = normal(m, n, std=1e-3, dtype=torch.bfloat16)
    elif case["op"] == "norm_grad":
        rows, cols, stream = case["rows"], case["cols"], DTYPE[case["stream"]]
        h = activations(rows, cols)
        s["rstd"] = torch.rsqrt(h.double().square().mean(1) + 1e-5).float()
        s["h"] = _pack_mxfp8(h)
        s["gain"] = (1.0 + 0.1 * normal(cols)).to(torch.bfloat16)
        s["dy"] = normal(rows, cols, std=1e-3, dtype=torch.bfloat16)
        s["dh"] = normal(rows, cols, std=1e-3, dtype=stream) if case["dh"] else None
    else:
        s["x"] = _pack_mxfp8(activations(case["T"], case["Din"]))
        s["gy"] = normal(case["T"], case["Dout"], std=1e-3, dtype=torch.bfloat16)
    return s


def _power(byte):
    """2^(byte - 127) for bytes 1 .. 254, in 32 bits."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _pack_mxfp8(v):
    """(codes [rows, cols] and scales [rows, cols / 32], bytes) of a matrix in
    MXFP8: the least power of two that leaves a block's largest magnitude at
    448 or below."""
    b = v.view(v.shape[0], -1, 32)
    mant, exp = torch.frexp(b.abs().amax(2, keepdim=True))
    byte = torch.clamp(exp + 118 + (mant > 0.875).to(torch.int32), min=1)
    codes = (b / _power(byte)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(v.shape), byte.squeeze(2).to(torch.uint8)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, 32)
    return (v * _power(scales).unsqueeze(2)).view(codes.shape)


def _act(z, act):
    """(f(z), f'(z))."""
    if act == "RELU":
        return torch.clamp(z, min=0), (z > 0).to(z.dtype)
    if act == "SILU":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if act == "GELU":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain(s):
    c = s["case"]
    if c["op"] in ("xent", "xent_grad"):
        h, w, y = s["h"].float(), s["w"].float(), s["y"]
        z = c["scale"] * torch.matmul(h, w.t())
        there, at = y >= 0, y.clamp(min=0)[:, None]
        if c["op"] == "xent":
            top = z.amax(1)
            lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
            loss = torch.where(there, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
            return {"loss": loss, "lse": lse}
        dloss = torch.where(there, s["dloss"], torch.zeros_like(s["dloss"]))
        every = dloss if s["dlse"] is None else dloss + s["dlse"]
        g = every[:, None] * torch.exp(z - s["lse"][:, None])
        g.scatter_add_(1, at, -dloss[:, None])
        g = c["scale"] * g
        return {"dh": torch.matmul(g, w).to(torch.bfloat16), "dw": torch.matmul(g.t(), h).to(torch.bfloat16)}
    if c["op"] == "act_grad":
        n = c["n"]
        z, g = _values(*s["z"]), s["dout"].float()
        f, slope = _act(z[:, :n], c["act"])
        dz = g * slope
        if c["gated"]:
            dz, f = torch.cat((dz * z[:, n:], g * f), 1), f * z[:, n:]
        got = {"dz": dz.to(torch.bfloat16)}
        if c["bias"]:
            got["dbias"] = dz.sum(0)
        if c["remake"]:
            got["out"] = f.to(torch.bfloat16)
        return got
    if c["op"] == "norm_grad":
        n, g = _values(*s["h"]) * s["rstd"][:, None], s["dy"].float()
        dgain = (g * n).sum(0)
        g = g * s["gain"].float()
        dx = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(DTYPE[c["stream"]]), "dgain": dgain}
    return {"dw": torch.matmul(s["gy"].float().t(), _values(*s["x"])).to(DTYPE[c["out"]])}


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------
def _own(s):
    import mxfp4_precision_gemms_amd as A

    c = s["case"]
    if c["op"] == "xent":
        r = A.adahop_xent(s["h"], s["w"], s["y"], scale=c["scale"])
        return {"loss": r.loss, "lse": r.lse}
    if c["op"] == "xent_grad":
        dh, dw = A.adahop_xent_backward(s["h"], s["w"], s["y"], s["lse"], s["dloss"], dlse=s["dlse"],
                                        scale=c["scale"])
        return {"dh": dh, "dw": dw}
    if c["op"] == "act_grad":
        r = A.adahop_act_backward_mx8(s["dout"], s["z"], act=c["act"], gated=c["gated"],
                                      bias_grad=c["bias"], remake_out=c["remake"])
        got = {"dz": r.dz}
        if c["bias"]:
            got["dbias"] = r.dbias
        if c["remake"]:
            got["out"] = r.out
        return got
    if c["op"] == "norm_grad":
        dx, dgain = A.adahop_rmsnorm_backward_mx8(s["dy"], s["h"], s["gain"], s["rstd"], s["dh"],
                                                  dx_dtype=DTYPE[c["stream"]])
        return {"dx": dx, "dgain": dgain}
    return {"dw": A.adahop_gemm_wgrad_mx8(s["gy"], s["x"], out_dtype=DTYPE[c["out"]])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "xent":
        T, V, D = case["T"], case["V"], case["D"]
        return {"bytes": 2 * (T + V) * D + 16 * T, "flops": 2 * T * V * D + 4 * T * V}
    if case["op"] == "xent_grad":
        T, V, D = case["T"], case["V"], case["D"]
        # the logits again, then both products of their gradient
        return {"bytes": 4 * (T + V) * D + (20 if case["zloss"] else 16) * T, "flops": 6 * T * V * D + 4 * T * V}
    if case["op"] == "act_grad":
        e, parts = case["m"] * case["n"], 2 if case["gated"] else 1
        b = 2 * e + parts * e * 33 // 32 + 2 * parts * e + (2 * e if case["remake"] else 0)
        return {"bytes": b + (4 * parts * case["n"] if case["bias"] else 0), "flops": 20 * e}
    if case["op"] == "norm_grad":
        e, t = case["rows"] * case["cols"], 2 if case["stream"] == "bf16" else 4
        return {"bytes": e * (2 + t * (2 if case["dh"] else 1)) + e * 33 // 32 + 4 * case["rows"] + 6 * case["cols"],
                "flops": 12 * e}
    T, Din, Dout = case["T"], case["Din"], case["Dout"]
    return {"bytes": 2 * T * Dout + T * Din * 33 // 32 + Din * Dout * (2 if case["out"] == "bf16" else 4),
            "flops": 2 * T * Din * Dout}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)

    def matrix(codes, scales):
        i = codes.int()
        e, f = (i >> 3) & 15, (i & 7).double()
        v = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
        v = torch.where(i > 127, -v, v)
        return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)

    if case["op"] in ("xent", "xent_grad"):
        h, w = s["h"].double(), s["w"].double()
        logits = (h @ w.t()).mul_(case["scale"])
        rows = torch.nonzero(s["y"] >= 0)[:, 0]
        said = s["y"][rows]
        if case["op"] == "xent":
            lse = torch.logsumexp(logits, 1)
            loss = torch.zeros_like(lse)
            loss[rows] = lse[rows] - logits[rows, said]
            return {"loss": loss, "lse": lse}
        d = torch.zeros_like(s["lse"], dtype=torch.float64)
        d[rows] = s["dloss"].double()[rows]
        of_lse = d if s["dlse"] is None else d + s["dlse"].double()
        # the gradient of the logits: of the normalizer everywhere, of the token's own logit
        logits.sub_(s["lse"].double()[:, None]).exp_().mul_(of_lse[:, None])
        logits[rows, said] -= d[rows]
        logits.mul_(case["scale"])
        return {"dh": logits @ w, "dw": logits.t() @ h}
    if case["op"] == "act_grad":
        n = case["n"]
        z, g = matrix(*s["z"]), s["dout"].double()
        a = z[:, :n]
        if case["act"] == "RELU":
            f, slope = torch.where(a > 0, a, 0 * a), torch.where(a > 0, torch.ones_like(a), 0 * a)
        elif case["act"] == "SILU":
            e = torch.exp(-a)
            f, slope = a / (1 + e), (1 + e + a * e) / (1 + e) ** 2
        elif case["act"] == "GELU":
            cdf = 0.5 * torch.erfc(-a / 2 ** 0.5)
            f, slope = a * cdf, cdf + a * torch.exp(-a * a / 2) / (2 * math.pi) ** 0.5
        else:
            u = (8 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3)
            p = 1 / (1 + torch.exp(-u))
            f, slope = a * p, p + a * p * (1 - p) * (8 / math.pi) ** 0.5 * (1 + 0.134145 * a * a)
        dz = torch.cat((g * z[:, n:] * slope, g * f), 1) if case["gated"] else g * slope
        got = {"dz": dz}
        if case["bias"]:
            got["dbias"] = dz.sum(0)
        if case["remake"]:
            got["out"] = f * z[:, n:] if case["gated"] else f
        return got
    if case["op"] == "norm_grad":
        h, dy, gain = matrix(*s["h"]), s["dy"].double(), s["gain"].double()
        r = s["rstd"].double()[:, None]
        inner = (dy * gain * h).sum(1, keepdim=True)
        dx = r * dy * gain - h * inner * r ** 3 / case["cols"]
        dx = dx if s["dh"] is None else dx + s["dh"].double()
        return {"dx": dx, "dgain": (dy * h * r).sum(0)}
    return {"dw": s["gy"].double().t() @ matrix(*s["x"])}
