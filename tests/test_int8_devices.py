"""Where the 8-bit helpers' tensors may lie: on the current CUDA device, and nowhere else.

Kernels that were given host addresses would fault, so nothing here may get as far as the
library: a stand-in for it says if a call did.  No GPU is needed (or used, where there is one).
"""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


class Reached(Exception):
    pass


class Library:
    """The library with its two calls that would enqueue work taken out."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        if name in ("cake_gg_i8_gemm", "cake_gg_i8_quant"):
            raise Reached(name)
        return getattr(self._lib, name)


@pytest.fixture(autouse=True)
def library(monkeypatch):
    gg_build.build()
    monkeypatch.setattr(gg, "_lib", Library(gg.load_library()))


def _cpu():
    import torch
    return dict(X=torch.zeros((4, 32), dtype=torch.bfloat16), W=torch.zeros((2, 16, 32), dtype=torch.int8),
                ws=torch.zeros((2, 16)), offsets=torch.tensor([0, 2, 4], dtype=torch.int32))


def test_products_of_host_tensors_are_refused():
    """Otherwise valid calls: dense and grouped, activations and 8-bit tokens, with what may be given."""
    import torch
    a = _cpu()
    q, s = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4)
    plan = gg.cake_gg_i8_plan(2, 4, 4, 16, 32)
    for call in (lambda: gg.int8_gemm(**a), lambda: gg.int8_gemm(a["X"], a["W"][0], a["ws"][0]),
                 lambda: gg.int8_gemm(**{**a, "X": q}, xs=s),
                 lambda: gg.int8_gemm(**a, rows=torch.zeros(5, dtype=torch.int32)),
                 lambda: gg.int8_gemm(**a, plan=plan, workspace=gg.make_workspace(plan, "cpu"), check=False,
                                      out=torch.zeros((4, 16), dtype=torch.bfloat16)),
                 lambda: gg.int8_gemm(**a, stream=1 << 20)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_quantising_host_tensors_is_refused():
    import torch
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    for more in ({}, dict(act="silu_mul"), dict(stream=1 << 20),
                 dict(out=torch.zeros((4, 32), dtype=torch.int8), scale=torch.zeros(4))):
        with pytest.raises(ValueError, match="CUDA"):
            gg.quantize_rows(x, **more)


class OnDevice:
    """A tensor as the helpers look at it, on a device that need not exist."""

    def __init__(self, shape, dtype, index=0):
        import torch
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")
        self.nbytes = 1 << 20

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20


def _fake(index):
    import torch
    return dict(X=OnDevice((4, 32), torch.bfloat16, index), W=OnDevice((2, 16, 32), torch.int8, index),
                ws=OnDevice((2, 16), torch.float32, index), offsets=OnDevice((3,), torch.int32, index),
                out=OnDevice((4, 16), torch.bfloat16, index), workspace=OnDevice((1 << 20,), torch.uint8, index),
                check=False, stream=1 << 20)


def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch):
    """The library launches on the current device, whatever the tensors'."""
    import torch
    monkeypatch.setattr(gg, "_current_device", lambda: 0, raising=False)
    with pytest.raises(Reached):
        gg.int8_gemm(**_fake(0))
    with pytest.raises(ValueError, match="cuda:1"):
        gg.int8_gemm(**_fake(1))
    with pytest.raises(ValueError, match="cuda:1"):
        gg.quantize_rows(OnDevice((4, 32), torch.bfloat16, 1), out=OnDevice((4, 32), torch.int8, 1),
                         scale=OnDevice((4,), torch.float32, 1), stream=1 << 20)


@pytest.mark.parametrize("index", [-1, 1])
def test_a_workspace_elsewhere_is_refused(index, monkeypatch):
    import torch
    monkeypatch.setattr(gg, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="workspace"):
        gg.int8_gemm(**{**_fake(0), "workspace": OnDevice((1 << 20,), torch.uint8, index)})
