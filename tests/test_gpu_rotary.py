"""nvfp4_rotary against the formula in 64 bits.

The angle is formed and reduced in FP64: power, division by 2 pi and product
are off by at most 2.5 units of 2^-52 of it in the kernel and 1.5 here, together
2^-50 of the angle.  It is rounded to FP32 in half turns (2^-25 of them: 2^-25 pi radians), cos and sin
are off by at most 2 units in the last place (2^-23), the two products and
their sum round three times: each output by at most 10 * 2^-24 (|u| + |v|) plus
the FP64 part; a bf16 output rounds once more (2^-8 of the result)."""
import math

import pytest
import torch

import nvfp4_w4a4_gemm_quantize_b200 as nv

pytestmark = pytest.mark.gpu


def _reference(x, positions, axes, theta, interleaved, inverse=False):
    """(y, tolerance of its FP32 form) in FP64."""
    x = x.double()
    at = positions.double()
    if at.dim() == 2:
        at = at[None]
    angle = torch.cat([at[..., a, None] * theta ** (-torch.arange(0, w, 2, device=x.device).double() / w)
                       for a, w in enumerate(axes) if w], -1)[:, :, None]
    n = angle.shape[-1]
    c, s = torch.cos(angle), torch.sin(angle) * (-1 if inverse else 1)
    u, v = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    a, b = u * c - v * s, u * s + v * c
    t = (u.abs() + v.abs()) * (10 * 2.0 ** -24 + angle.abs() * 2.0 ** -50)
    y, tol = x.clone(), torch.zeros_like(x)
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a, b
        tol[..., 0:2 * n:2], tol[..., 1:2 * n:2] = t, t
    else:
        y[..., :n], y[..., n:2 * n] = a, b
        tol[..., :n], tol[..., n:2 * n] = t, t
    return y, tol


def _check(x, positions, axes, theta=10000.0, interleaved=True, inverse=False, **kw):
    y = nv.rotary(x, positions, axes, theta, interleaved, inverse, **kw)
    ref, tol = _reference(x, positions, axes, theta, interleaved, inverse)
    if x.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((y.double() - ref).abs() <= tol).all())
    return y


def _x(B, L, H, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, L, H, d, generator=g, device="cuda").to(dtype)


def _grid(t, y, x, start=0):
    at = torch.arange(t * y * x, device="cuda", dtype=torch.int32)
    return torch.stack([at // (y * x) + start, at // x % y, at % x], 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,H,d,axes", [(1, 24, 128, (44, 42, 42)), (2, 16, 72, (0, 36, 36)), (3, 1, 64, (16, 20, 20)),
                                        (2, 5, 80, (28, 26, 26)), (1, 3, 8, (2, 0, 0)), (1, 2, 256, (64, 96, 96)),
                                        (2, 7, 96, (6, 2, 10)), (1, 1, 40, (8, 16, 16))])
def test_rotary_head_layouts(cuda_ok, dtype, interleaved, B, H, d, axes):
    x, at = _x(B, 3 * 5 * 7, H, d, dtype, seed=d + H), _grid(3, 5, 7)
    y = _check(x, at, axes, interleaved=interleaved)
    back = _check(y, at, axes, interleaved=interleaved, inverse=True)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    # there and back: each way rounds by at most a half step of a pair's norm, and turning keeps the norm
    assert bool(((back.double() - x.double()).abs() <= 2.1 * (step + 24 * 2.0 ** -24) * 1.42 * x.double().abs().amax()).all())


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 257, 1000])
@pytest.mark.parametrize("n_axes", [1, 2, 4])
def test_rotary_lengths_and_axes(cuda_ok, L, n_axes):
    g = torch.Generator(device="cuda").manual_seed(L)
    at = torch.randint(0, 500, (L, n_axes), generator=g, device="cuda", dtype=torch.int32)
    axes = {1: (64,), 2: (32, 24), 4: (16, 0, 30, 18)}[n_axes]
    _check(_x(2, L, 3, 64, torch.bfloat16, L), at, axes, theta=500.0, interleaved=L % 2 == 0)


@pytest.mark.parametrize("dtype", [torch.int32, torch.float32])
@pytest.mark.parametrize("far", [0, 100003, 2 ** 31 - 200])
def test_rotary_far_negative_and_fractional_positions(cuda_ok, dtype, far):
    """Far positions keep their angle; positions of each sample; negative and
    (FP32) fractional ones."""
    if dtype == torch.float32 and far > 2 ** 24:
        far = 2.0 ** 30
    at = _grid(2, 4, 8).to(dtype)[None].repeat(3, 1, 1)
    at[0, :, 0] += far
    at[1, :, 1] -= far
    if dtype == torch.float32 and far == 0:
        at[2] = at[2] * 0.37
    for interleaved in (True, False):
        _check(_x(3, 64, 4, 64, torch.float32, 5), at, (16, 24, 24), interleaved=interleaved)


def test_rotary_views_in_and_out(cuda_ok):
    """A part of a fused projection, head-major buffers, a broadcast batch, in
    place; nothing outside the output's elements is written."""
    B, L, H, d = 2, 77, 6, 64
    qkv = torch.randn(B, L, 3, H, d, device="cuda").bfloat16()
    at, axes = _grid(1, 7, 11), (20, 22, 22)
    want = nv.rotary(qkv[:, :, 1].contiguous(), at, axes)
    assert torch.equal(_check(qkv[:, :, 1], at, axes), want)
    buf = torch.full((B, H, L + 1, d), 5.0, device="cuda", dtype=torch.bfloat16)
    nv.rotary(qkv[:, :, 1], at, axes, out=buf[:, :, :L].transpose(1, 2))
    assert torch.equal(buf[:, :, :L].transpose(1, 2), want) and bool((buf[:, :, L] == 5.0).all())
    one = torch.randn(1, L, 1, d, device="cuda").bfloat16()
    assert torch.equal(nv.rotary(one.expand(B, L, H, d), at, axes), nv.rotary(one.repeat(B, 1, H, 1), at, axes))
    for interleaved in (True, False):
        want = nv.rotary(qkv[:, :, 0], at, axes, interleaved=interleaved)
        rest = qkv[:, :, 1:].clone()
        mine = qkv.clone()
        nv.rotary(mine[:, :, 0], at, axes, interleaved=interleaved, out=mine[:, :, 0])
        assert torch.equal(mine[:, :, 0], want) and torch.equal(mine[:, :, 1:], rest)
    # positions with strides of their own
    wide = torch.zeros(L, 5, device="cuda", dtype=torch.int32)
    wide[:, 1:4] = at
    assert torch.equal(nv.rotary(qkv[:, :, 1], wide[:, 1:4], axes), nv.rotary(qkv[:, :, 1].contiguous(), at, axes))


def test_rotary_refuses_odd_strides_and_empty_is_empty(cuda_ok):
    x, at = torch.zeros(1, 4, 2, 68, device="cuda", dtype=torch.bfloat16), torch.zeros(4, 1, device="cuda", dtype=torch.int32)
    with pytest.raises(nv.NVFP4Error):
        nv.rotary(x[..., :64], at, (64,))                     # 136-byte head steps
    with pytest.raises(nv.NVFP4Error):
        nv.rotary(x, at, (64,))                               # d % 8
    with pytest.raises(nv.NVFP4Error):
        nv.rotary(x[..., 1:65], at, (64,))
    assert nv.rotary(x[:, :0, :, :64].contiguous(), at[:0], (64,)).shape == (1, 0, 2, 64)


def test_rotary_non_finite_values_stay_in_their_pair(cuda_ok):
    x = torch.ones(1, 8, 2, 64, device="cuda")
    at = torch.arange(8, device="cuda", dtype=torch.int32)[:, None]
    x[0, 3, 1, 10] = float("nan")
    y = nv.rotary(x, at, (64,))
    bad = y.isnan()
    assert bool(bad[0, 3, 1, 10:12].all()) and int(bad.sum()) == 2
    p = torch.arange(8, device="cuda", dtype=torch.float32)[:, None].repeat(1, 2)
    p[5, 1] = float("inf")
    y = nv.rotary(torch.ones(1, 8, 2, 64, device="cuda"), p, (32, 32))
    assert bool(y[0, 5, :, 32:].isnan().all()) and int(y.isnan().sum()) == 2 * 32


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_gradient(cuda_ok, interleaved):
    """Against the formula, and against differences: the map is linear, so
    <y(x + h) - y(x - h), g> = 2 <h, dx> exactly."""
    at, axes = _grid(2, 5, 6), (20, 22, 22)
    x = _x(2, 60, 4, 64, torch.float32, 1).requires_grad_()
    g = _x(2, 60, 4, 64, torch.float32, 2)
    y = nv.RotaryEmbedding.apply(x, at, axes, 10000.0, interleaved)
    (dx,) = torch.autograd.grad(y, x, g)
    ref, tol = _reference(g, at, axes, 10000.0, interleaved, inverse=True)
    assert bool(((dx.double() - ref).abs() <= tol).all())
    h = _x(2, 60, 4, 64, torch.float32, 3).double()
    up, _ = _reference(x.detach().double() + h, at, axes, 10000.0, interleaved)
    down, _ = _reference(x.detach().double() - h, at, axes, 10000.0, interleaved)
    diff = ((up - down) * g.double()).sum() / 2
    assert abs(float(diff - (h * dx.double()).sum())) <= float((tol * h.abs()).sum()) + 1e-9 * float((h * ref).abs().sum())
    # a gradient that arrives as a view with odd strides, and one from a sum (all strides zero)
    y = nv.RotaryEmbedding.apply(x, at, axes, 10000.0, interleaved)
    (dx,) = torch.autograd.grad(y.sum(), x)
    ref, tol = _reference(torch.ones_like(g), at, axes, 10000.0, interleaved, inverse=True)
    assert bool(((dx.double() - ref).abs() <= tol).all())
    y = nv.RotaryEmbedding.apply(x, at, axes, 10000.0, interleaved)
    wide = torch.zeros(2, 60, 4, 65, device="cuda")
    wide[..., 1:] = g
    (dx,) = torch.autograd.grad(y, x, wide[..., 1:])
    ref, tol = _reference(g, at, axes, 10000.0, interleaved, inverse=True)
    assert bool(((dx.double() - ref).abs() <= tol).all())


def test_rotary_offsets_past_32_bits(cuda_ok):
    """Samples and tokens more than 2^31 elements apart."""
    d, far = 64, 2 ** 31 + 8
    buf = torch.empty(far + 4096, device="cuda", dtype=torch.bfloat16)
    x = buf.as_strided((2, 4, 2, d), (far, 2 * d, d, 1))
    v = _x(2, 4, 2, d, torch.bfloat16, 8)
    x.copy_(v)
    at = torch.arange(4, device="cuda", dtype=torch.int32)[:, None]
    assert torch.equal(nv.rotary(x, at, (d,)), nv.rotary(v, at, (d,)))
    nv.rotary(x, at, (d,), out=x)
    assert torch.equal(x, nv.rotary(v, at, (d,)))


def test_rotary_on_another_stream_and_in_a_graph(cuda_ok):
    x, at, axes = _x(1, 90, 4, 64, torch.bfloat16, 9), _grid(1, 9, 10), (20, 22, 22)
    want = nv.rotary(x, at, axes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = nv.rotary(x, at, axes, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    xs = x.clone().requires_grad_()
    grad = _x(1, 90, 4, 64, torch.bfloat16, 10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(nv.RotaryEmbedding.apply(xs, at, axes), xs, grad)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = nv.RotaryEmbedding.apply(xs, at, axes)
        (dx,) = torch.autograd.grad(y, xs, grad)
    x2 = _x(1, 90, 4, 64, torch.bfloat16, 11)
    with torch.no_grad():
        xs.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, nv.rotary(x2, at, axes)) and torch.equal(dx, nv.rotary(grad, at, axes, inverse=True))
    assert math.isfinite(float(dx.float().sum()))
