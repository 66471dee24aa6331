"""The operators around the linear layers together, as a diffusion transformer
block uses them: conditioning by a 4-bit matrix-vector product, LayerNorm with
that modulation into the NVFP4 projections, rotary positions on queries and
keys, self attention, then attention to a text encoder's padded states; and the
training path of the last two.  The whole is compared with the same steps in 64
bits on the same quantized weights; the steps in between round to bf16 or to
NVFP4, so the check of the whole is on its norm, each operator's own test holds
its elements."""
import math

import pytest
import torch

import nvfp4_w4a4_gemm_quantize_b200 as nv
from nvfp4_w4a4_gemm_quantize_b200 import synth

pytestmark = pytest.mark.gpu

T, Y, X, H, D, TEXT = 4, 8, 8, 4, 128, 77
L, HID = T * Y * X, H * D
AXES = (44, 42, 42)


def _w(n, k, seed):
    return nv.quantize((synth.random_bf16((n, k), seed=seed).float() * k ** -0.5).bfloat16().cuda())


def _positions():
    at = torch.arange(L, device="cuda", dtype=torch.int32)
    return torch.stack([at // (Y * X), at // X % Y, at % X], 1)


def _turn64(x):
    at = _positions().double()
    angle = torch.cat([at[:, a, None] * 10000.0 ** (-torch.arange(0, w, 2, device="cuda").double() / w)
                       for a, w in enumerate(AXES)], 1)[:, None]
    c, s = torch.cos(angle), torch.sin(angle)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)


def _relative(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_block_forward(cuda_ok):
    B = 2
    x = synth.random_bf16((B * L, HID), seed=1).cuda()
    cond = synth.random_bf16((B, 256), seed=2).cuda()
    text = synth.random_bf16((B * TEXT, HID), seed=3).cuda()
    lens = torch.tensor([TEXT, 19], dtype=torch.int32, device="cuda")
    wm, wq, wk, wv, wxq, wxk, wxv = _w(2 * HID, 256, 4), *(_w(HID, HID, 5 + i) for i in range(6))
    bias = torch.cat([torch.ones(HID), torch.zeros(HID)]).cuda()

    # conditioning: scale and shift of every sample in FP32, read by the norm
    mod = nv.gemv_w4a16(cond, wm, bias=bias, out_dtype=torch.float32)
    gamma, beta = mod[:, :HID].contiguous(), mod[:, HID:].contiguous()
    h = nv.layernorm_quantize(x, gamma, beta, rows_per_group=L)
    q, k, v = (nv.gemm_w4a4(h, w).view(B, L, H, D) for w in (wq, wk, wv))
    # rotary straight into head-major rows, which the quantizer takes
    qr, kr = (torch.empty(B, H, L, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    nv.rotary(q, _positions(), AXES, out=qr.transpose(1, 2))
    nv.rotary(k, _positions(), AXES, out=kr.transpose(1, 2))
    rows = [nv.quantize(t.reshape(B * H * L, D)) for t in (qr, kr, v.transpose(1, 2).contiguous())]
    a = nv.attention(*rows, B * H).view(B, H, L, D).transpose(1, 2).reshape(B * L, HID)
    # cross attention to the text states
    xq = nv.gemm_w4a16(a, wxq).view(B, L, H, D)
    xk, xv = (nv.gemm_w4a16(text, w).view(B, TEXT, H, D) for w in (wxk, wxv))
    o = nv.cross_attention(xq, xk, xv, lens)

    def w64(w):
        return nv.dequantize(w, torch.float32).double()

    m64 = cond.double() @ w64(wm).T + bias
    n64 = torch.nn.functional.layer_norm(x.double(), (HID,), eps=1e-6).view(B, L, HID)
    n64 = (n64 * m64[:, None, :HID] + m64[:, None, HID:]).view(B * L, HID)
    q64, k64, v64 = ((n64 @ w64(w).T).view(B, L, H, D) for w in (wq, wk, wv))
    q64, k64 = (_turn64(t).transpose(1, 2) for t in (q64, k64))
    a64 = (torch.softmax(q64 @ k64.transpose(2, 3) / math.sqrt(D), 3) @ v64.transpose(1, 2)).transpose(1, 2).reshape(B * L, HID)
    xq64 = (a64 @ w64(wxq).T).view(B, L, H, D).transpose(1, 2)
    xk64, xv64 = ((text.double() @ w64(w).T).view(B, TEXT, H, D).transpose(1, 2) for w in (wxk, wxv))
    s64 = xq64 @ xk64.transpose(2, 3) / math.sqrt(D)
    s64[1, :, :, 19:] = -math.inf
    o64 = (torch.softmax(s64, 3) @ xv64).transpose(1, 2)
    # NVFP4 rounds a value by up to 2^-2 of it (E2M1's widest relative half step), 2^-3.5 in the mean square: the
    # projections' input, then queries, keys and values, carry that once each
    assert _relative(mod, m64) < 1e-5
    assert _relative(a, a64) < 4 * 2.0 ** -3.5
    assert _relative(o, o64) < 4 * 2.0 ** -3.5


def test_block_training(cuda_ok):
    """Rotary positions and cross attention under autograd, gradients against
    autograd in FP64 through the same graph."""
    B = 2
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(B, n, H, D, generator=g, device="cuda").bfloat16().requires_grad_() for n in (L, TEXT, TEXT))
    lens = torch.tensor([TEXT, 30], dtype=torch.int32, device="cuda")
    do = torch.randn(B, L, H, D, generator=g, device="cuda").bfloat16()
    o = nv.CrossAttention.apply(nv.RotaryEmbedding.apply(q, _positions(), AXES), k, v, lens)
    grads = torch.autograd.grad(o, (q, k, v), do)
    q6, k6, v6 = (t.detach().double().requires_grad_() for t in (q, k, v))
    s = _turn64(q6).transpose(1, 2) @ k6.permute(0, 2, 3, 1) / math.sqrt(D)
    s = s.masked_fill((torch.arange(TEXT, device="cuda") >= lens[:, None])[:, None, None], -math.inf)
    o6 = (torch.softmax(s, 3) @ v6.transpose(1, 2)).transpose(1, 2)
    want = torch.autograd.grad(o6, (q6, k6, v6), do.double())
    # at most six roundings to bf16 (2^-8 each) lie between the inputs and a gradient, and D inherits out's
    assert _relative(o, o6) < 6 * 2.0 ** -8
    for got, ref in zip(grads, want):
        assert _relative(got, ref) < 12 * 2.0 ** -8
