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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", ["contiguous", "contiguous, off by one", "padded rows", "rows of 65", "one for all", "tokens shared",
                                  "head major", "empty"])
def test_gradients_get_rows_of_16_bytes(dtype, what):
    """Whatever a gradient's memory looks like, the backward calls get the same
    values with d contiguous and 16-byte steps, and the tensor itself where it
    has them already."""
    B, L, H, d = 2, 5, 3, 64
    n = B * L * H * d
    buf = torch.randn(4 * n, dtype=torch.float32).to(dtype)
    assert buf.data_ptr() % 16 == 0
    t, kept = {
        "contiguous": (buf[:n].view(B, L, H, d), True),
        "contiguous, off by one": (buf[1:n + 1].view(B, L, H, d), False),
        "padded rows": (buf.as_strided((B, L, H, d), (L * H * 72, H * 72, 72, 1)), True),
        "rows of 65": (buf.as_strided((B, L, H, d), (L * H * 65, H * 65, 65, 1)), False),
        "one for all": (buf[:1].view(1, 1, 1, 1).expand(B, L, H, d), False),
        "tokens shared": (buf[:d].view(1, 1, 1, d).expand(B, L, H, d), False),
        "head major": (buf[:n].view(B, H, L, d).transpose(1, 2), True),
        "empty": (buf[1:1].view(B, 0, H, d), None),
    }[what]
    r = nv._rows16(t)
    assert r.shape == t.shape and r.dtype == dtype and torch.equal(r, t)
    assert r.stride(3) == 1 and r.data_ptr() % 16 == 0
    step = 16 // t.element_size()
    assert all(s % step == 0 for s in r.stride()[:3])
    if kept is not None:
        assert (r is t) == kept
