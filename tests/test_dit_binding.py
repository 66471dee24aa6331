"""What the Python entry points of include/nvfp4_dit.h hand to the library, and
what their autograd functions do with it: the library's calls are replaced by
recorders, so no GPU is needed."""
import pytest
import torch

import nvfp4_w4a4_gemm_quantize_b200 as nv


class _Recorder:
    """Stands for the loaded library: every call is recorded and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(nv, "lib", lambda: r)
    monkeypatch.setattr(nv, "_on_device", lambda *tensors: None)
    monkeypatch.setattr(nv, "_stream", lambda stream: None)
    return r


def _weights(fmt, n=8, k=128):
    codes, sf = torch.zeros(n, k // 2, dtype=torch.uint8), torch.zeros(128 * (k // 16), dtype=torch.uint8)
    return nv.MXTensor(codes, sf, n, k) if fmt == "mx" else nv.NVFP4Tensor(codes, sf, torch.ones(1), n, k)


@pytest.mark.parametrize("fmt", ["nvfp4", "mx"])
@pytest.mark.parametrize("what,rows,stride", [("contiguous", 4, 128), ("wider rows", 4, 320), ("one row for all", 4, 0),
                                              ("one row", 1, 128), ("one row of stride 0", 1, 0), ("none", 0, 128)])
def test_gemv_passes_the_rows_own_stride(recorder, fmt, what, rows, stride):
    x = torch.zeros(4 * 320, dtype=torch.bfloat16).as_strided((rows, 128), (stride, 1))
    nv.gemv_w4a16(x, _weights(fmt))
    (name, args), = recorder.calls
    assert name == "nvfp4_gemv_w4a16" and args[0] == x.data_ptr() and args[7] == rows
    assert args[1] == (stride if rows > 1 else 128)


@pytest.mark.parametrize("stride", [8, 64, 120])
def test_gemv_refuses_rows_that_overlap(recorder, stride):
    x = torch.zeros(1024, dtype=torch.bfloat16).as_strided((4, 128), (stride, 1))
    with pytest.raises(ValueError, match="overlap"):
        nv.gemv_w4a16(x, _weights("nvfp4"))
    assert not recorder.calls
