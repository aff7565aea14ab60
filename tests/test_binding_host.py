"""The binding's own refusals, on the host: a stand-in takes the library's
place and records what reaches it. No GPU, and nothing is launched."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A


class Standin:
    """Every entry point succeeds and is recorded; `size` is what each size
    that is asked for comes to."""

    def __init__(self):
        self.calls, self.args, self.size = [], {}, 0

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            self.args[name] = args
            return self.size if name.endswith("_size") else 0
        return call

    def launched(self):
        return [c for c in self.calls if not c.endswith("_size")]


@pytest.fixture
def standin(monkeypatch):
    s = Standin()
    monkeypatch.setattr(A, "lib", lambda: s)
    # a process that has a GPU, whose current stream is the default one
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
    return s


def mx_operands(device="cpu"):
    return [torch.zeros(s, dtype=torch.uint8, device=device) for s in ((4, 16), (4, 1), (8, 16), (8, 1))]


def test_stream_of_a_host_device():
    for device in ("cpu", "meta"):
        with pytest.raises(ValueError):
            A._stream(torch.device(device))


def test_stream_of_a_gpu(standin):
    assert A._stream(torch.device("cuda")) == 0 and A._stream(torch.device("cuda", 0)) == 0


def test_gemm_mx_of_host_tensors(standin):
    with pytest.raises(ValueError):
        A.adahop_gemm_mx(*mx_operands())
    assert standin.launched() == []


class OnGpu:
    """Says that it lies on GPU 0; as much of a tensor as the binding looks at."""

    def __init__(self, t):
        self.t, self.device = t, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("host", range(6))
def test_gemm_mx_with_one_host_tensor(standin, host):
    """Each operand, the output and the outlier term's tensors are looked at."""
    t = [OnGpu(x) if i != host else x for i, x in enumerate(
        mx_operands() + [torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)])]
    # (the outlier term's matrices are looked at where their address is taken)
    oe = None if host != 5 else {"route": "OE_LEFT", "k": 2, "idx": t[5], "a": (None, 1), "b": (None, 1)}
    with pytest.raises(ValueError):
        A.adahop_gemm_mx(*t[:4], oe=oe, out=t[4])
    assert standin.launched() == []


def test_gemm_mx_of_gpu_tensors(standin):
    t = [OnGpu(x) for x in mx_operands()]
    out = OnGpu(torch.zeros(4, 8, dtype=torch.bfloat16))
    assert A.adahop_gemm_mx(*t, out=out) is out
    assert standin.launched() == ["adahop_gemm_mx"]


# ---- the caller's workspace -------------------------------------------------
WORKSPACES = {
    "host": lambda: torch.zeros(256, dtype=torch.uint8),
    "one element repeated": lambda: OnGpu(torch.zeros(1, dtype=torch.uint8).expand(256)),
    "every second element": lambda: OnGpu(torch.zeros(512, dtype=torch.uint8)[::2]),
    "columns of a matrix": lambda: OnGpu(torch.zeros(16, 64, dtype=torch.uint8)[:, :16]),
}


@pytest.mark.parametrize("size", [0, 64])
@pytest.mark.parametrize("kind", list(WORKSPACES))
def test_workspace_refusals(standin, kind, size):
    standin.size = size
    a, b = ([OnGpu(torch.zeros(s, dtype=torch.uint8)) for s in ((r, 32), (r, 1))] for r in (4, 8))
    out = OnGpu(torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        A.adahop_linear_mx(a, b, out=out, ws=WORKSPACES[kind]())
    assert standin.launched() == []
    ws = OnGpu(torch.zeros(16, 4, dtype=torch.float32))          # any type, any shape
    assert A.adahop_linear_mx(a, b, out=out, ws=ws).out is out
    assert standin.launched() == ["adahop_linear_mx"]


def test_one_row_has_no_leading_dimension(standin):
    """A row of a matrix whose rows lie 104 bytes apart: the distance to the next
    row, which there is none, is not held against it."""
    a = [OnGpu(torch.zeros(3, 104, dtype=torch.uint8)[2:, :96]), OnGpu(torch.zeros(3, 7, dtype=torch.uint8)[2:, :3])]
    b = [OnGpu(torch.zeros(s, dtype=torch.uint8)) for s in ((8, 96), (8, 3))]
    out = OnGpu(torch.zeros(1, 8, dtype=torch.bfloat16))
    assert A.adahop_linear_mx(a, b, out=out).out is out
    got = standin.args["adahop_linear_mx"][0]._obj
    assert (got.ld_a_codes, got.ld_a_scales, got.ld_b_codes) == (96, 3, 96)
