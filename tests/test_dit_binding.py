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


def _turn(x, positions, axes, theta=10000.0, interleaved=True, inverse=False, **kw):
    """rotary() of neighbouring pairs in elementary operations."""
    angle = torch.cat([positions[:, a, None].double() * theta ** (-torch.arange(0, w, 2).double() / w)
                       for a, w in enumerate(axes) if w], 1)[:, None] * (-1 if inverse else 1)
    u, v = x.double()[..., 0::2], x.double()[..., 1::2]
    c, s = torch.cos(angle), torch.sin(angle)
    return torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2).to(x.dtype)


def test_rotary_can_be_differentiated_twice(monkeypatch):
    """The gradient under create_graph carries its graph: second derivatives are
    those of the elementary operations, also where the loss has other paths."""
    monkeypatch.setattr(nv, "rotary", lambda *a, **kw: _turn(*a, **kw).detach())
    g = torch.Generator().manual_seed(1)
    at = torch.arange(5)[:, None]
    x0, w0 = (torch.randn(2, 5, 3, 8, generator=g) for _ in range(2))

    def second(turn):
        x, w = x0.clone().requires_grad_(), w0.clone().requires_grad_()
        y = turn(x)
        (dx,) = torch.autograd.grad((y * w).pow(2).sum() + x.pow(3).sum(), x, create_graph=True)
        return (dx.detach(), *torch.autograd.grad(dx.pow(2).sum(), (x, w)))

    want = second(lambda x: _turn(x, at, (8,)))
    for how in (lambda x: nv.RotaryEmbedding.apply(x, at, (8,)), lambda x: nv.RotaryEmbedding.apply(x, at, (8,), 10000.0, True, False)):
        for a, b in zip(second(how), want):
            assert torch.allclose(a, b, rtol=1e-5, atol=1e-5 * float(b.abs().max()))
    # without create_graph: the plain call, no graph
    x = x0.clone().requires_grad_()
    (dx,) = torch.autograd.grad(nv.RotaryEmbedding.apply(x, at, (8,), 10000.0, True, True), x, w0)
    assert not dx.requires_grad and torch.allclose(dx, _turn(w0, at, (8,)), rtol=1e-5, atol=1e-5)


def _attention(q, k, v, kv_lens=None, scale=None, return_lse=False, **kw):
    """cross_attention() of one head per key head, all keys."""
    s = torch.einsum("blhd,bmhd->bhlm", q, k) * (q.shape[3] ** -0.5 if scale is None else scale)
    out = torch.einsum("bhlm,bmhd->blhd", torch.softmax(s, 3), v)
    return (out, torch.logsumexp(s, 3)) if return_lse else out


def _attention_backward(do, q, k, v, out, lse, kv_lens=None, scale=None, **kw):
    with torch.enable_grad():
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        return torch.autograd.grad(_attention(*leaves, None, scale), leaves, do.detach())


def test_attention_refuses_second_derivatives(monkeypatch):
    """First derivatives under create_graph are as without; a second one through
    the attention raises, instead of leaving its terms out beside other paths."""
    monkeypatch.setattr(nv, "cross_attention", lambda *a, **kw: tuple(t.detach() for t in _attention(*a, **kw)))
    monkeypatch.setattr(nv, "cross_attention_backward", _attention_backward)
    g = torch.Generator().manual_seed(2)
    leaves = [torch.randn(2, n, 3, 8, generator=g).requires_grad_() for n in (4, 6, 6)]
    want = torch.autograd.grad(nv.CrossAttention.apply(*leaves).sum(), leaves)
    assert not any(t.requires_grad for t in want)
    for loss in (lambda out: out.sum(), lambda out: out.pow(2).sum()):
        plain = torch.autograd.grad(loss(nv.CrossAttention.apply(*leaves)), leaves)
        grads = torch.autograd.grad(loss(nv.CrossAttention.apply(*leaves)), leaves, create_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(grads, plain))
        # each beside another path to q
        for i in range(3):
            with pytest.raises(RuntimeError, match="second derivative"):
                torch.autograd.grad(grads[i].pow(2).sum() + leaves[0].pow(2).sum(), leaves[0])
            grads = torch.autograd.grad(loss(nv.CrossAttention.apply(*leaves)), leaves, create_graph=True)


@pytest.mark.parametrize("create_graph", [False, True])
def test_attention_passes_its_status_to_both_passes(monkeypatch, create_graph):
    """dev_status of CrossAttention.apply is that of the forward and of the
    backward call; without one there is none."""
    seen = []

    def forward(q, k, v, kv_lens=None, scale=None, out=None, return_lse=False, dev_status=None, stream=None):
        seen.append(("forward", scale, dev_status))
        return torch.zeros_like(q), torch.zeros(1, 2, 4)

    def backward(do, q, k, v, out, lse, kv_lens=None, scale=None, workspace=None, dev_status=None, stream=None):
        assert workspace is None and stream is None
        seen.append(("backward", scale, dev_status))
        return torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)

    monkeypatch.setattr(nv, "cross_attention", forward)
    monkeypatch.setattr(nv, "cross_attention_backward", backward)
    q, k, v = (torch.zeros(1, n, 2, 8, requires_grad=True) for n in (4, 6, 6))
    status = torch.zeros(1, dtype=torch.int32)
    for args, want in (((None, 0.5, status), (0.5, status)), ((None, 0.5), (0.5, None)), ((), (None, None))):
        seen.clear()
        torch.autograd.grad(nv.CrossAttention.apply(q, k, v, *args).sum(), (q, k, v), create_graph=create_graph)
        assert [s[0] for s in seen] == ["forward", "backward"]
        assert all(s[1] == want[0] and s[2] is want[1] for s in seen)
