"""include/nvfp4_dit.h: every declared symbol is exported and bound, and bad
calls are rejected by the host-side checks before any launch (no GPU needed:
each call fails its checks, or has nothing to do, before touching the device)."""
import ctypes
import os
import re
import struct

import pytest
import torch

import nvfp4_w4a4_gemm_quantize_b200 as nv
from nvfp4_w4a4_gemm_quantize_b200 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, MISALIGNED, DEVICE, CUDA, TIMEOUT, WORKSPACE, NONFINITE = range(9)
A, B, C = 0x10000, 0x20000, 0x30000          # fake, 16-byte aligned device addresses (never dereferenced)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "nvfp4_dit.h")).read()
    names = sorted(set(re.findall(r"\b(nvfp4_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S))))
    assert names == ["nvfp4_cross_attention", "nvfp4_cross_attention_backward",
                     "nvfp4_cross_attention_backward_workspace_bytes", "nvfp4_gemv_w4a16", "nvfp4_rotary"]
    for n in names:
        assert hasattr(L, n) and n in _lib.SIGNATURES


def test_header_constants_match_the_binding():
    text = open(os.path.join(ROOT, "include", "nvfp4_dit.h")).read()
    for name, value in re.findall(r"(NVFP4_[A-Z0-9_]+) = (\d+)", text):
        assert getattr(nv, name) == int(value), name


def gemv(L, x=A, ld=256, codes=A, sf=A, scale=A, fmt=0, bias=None, M=1, N=64, K=256, y=A, dt=0):
    return L.nvfp4_gemv_w4a16(x, ld, codes, sf, scale, fmt, bias, M, N, K, y, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0, ld=0), INVALID), (dict(ld=128), INVALID),
    (dict(fmt=2), INVALID), (dict(dt=2), INVALID), (dict(M=17), SHAPE), (dict(K=96), SHAPE),
    (dict(K=192, fmt=1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(x=None), INVALID), (dict(codes=None), INVALID),
    (dict(sf=None), INVALID), (dict(scale=None), INVALID), (dict(y=None), INVALID), (dict(x=A + 2), MISALIGNED),
    (dict(codes=A + 8), MISALIGNED), (dict(sf=A + 4), MISALIGNED), (dict(y=A + 4), MISALIGNED),
    (dict(bias=A + 2), MISALIGNED), (dict(scale=A + 1), MISALIGNED), (dict(M=2, ld=260), MISALIGNED),
    (dict(M=0, x=None, y=None), OK)])
def test_gemv_rejects_bad_arguments(L, bad, want):
    assert gemv(L, **bad) == want


def heads(data=A, sb=1 << 20, sl=2048, sh=128):
    return struct.pack("Pqqq", data or 0, sb, sl, sh)            # nvfp4_heads


def rotary(L, x=heads(), pos=A, pt=0, pb=0, pl=3, axes=(44, 42, 42), theta=1e4, B=2, T=16, H=4, d=128, dt=0, flags=1,
           out=heads(B)):
    dims = (ctypes.c_int * max(1, len(axes)))(*axes)
    return L.nvfp4_rotary(x, pos, pt, pb, pl, dims, len(axes), theta, B, T, H, d, dt, flags, out, None)


@pytest.mark.parametrize("bad,want", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(d=0), INVALID), (dict(axes=()), INVALID),
    (dict(axes=(8,) * 5), INVALID), (dict(axes=(43, 42, 42)), INVALID), (dict(axes=(-2, 42, 42)), INVALID),
    (dict(axes=(0, 0, 0)), INVALID), (dict(axes=(64, 64, 2)), INVALID), (dict(dt=2), INVALID), (dict(pt=2), INVALID),
    (dict(flags=4), INVALID), (dict(theta=0.0), INVALID), (dict(theta=-1.0), INVALID), (dict(theta=INF), INVALID),
    (dict(theta=NAN), INVALID), (dict(d=132), SHAPE), (dict(d=264), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(H=1 << 20), SHAPE), (dict(pl=-3), INVALID), (dict(pb=-1), INVALID), (dict(pos=None), INVALID),
    (dict(pos=A + 2), MISALIGNED), (dict(x=heads(None)), INVALID), (dict(x=heads(A + 8)), MISALIGNED),
    (dict(x=heads(sl=-2048)), INVALID), (dict(x=heads(sl=64)), INVALID), (dict(x=heads(sh=132)), MISALIGNED),
    (dict(out=heads(B, sh=0)), INVALID), (dict(out=heads(B, sb=0)), INVALID), (dict(out=heads(B, sl=2052)), MISALIGNED),
    (dict(x=heads(sb=1 << 40)), INVALID), (dict(T=0, pos=None), OK), (dict(B=0, pos=None), OK)])
def test_rotary_rejects_bad_arguments(L, bad, want):
    assert rotary(L, **bad) == want


def forward(L, q=heads(), k=heads(), v=heads(), lens=None, scale=0.1, B=2, H=8, Hkv=4, Lq=16, Lk=16, d=128,
            out=heads(B), lse=None):
    return L.nvfp4_cross_attention(q, k, v, lens, scale, B, H, Hkv, Lq, Lk, d, out, lse, None, None)


SIZES = [
    (dict(B=-1), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(Lq=-1), INVALID), (dict(Lk=-1), INVALID),
    (dict(d=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=INF), INVALID),
    (dict(scale=NAN), INVALID), (dict(Hkv=3), INVALID), (dict(d=132), SHAPE), (dict(d=136), SHAPE), (dict(d=12), SHAPE),
    (dict(Lq=1 << 28), SHAPE), (dict(Lk=1 << 29), SHAPE), (dict(lens=A + 2), MISALIGNED), (dict(B=0), OK)]


@pytest.mark.parametrize("bad,want", SIZES + [
    (dict(q=heads(None)), INVALID), (dict(k=heads(None)), INVALID), (dict(v=heads(None)), INVALID),
    (dict(out=heads(None)), INVALID), (dict(lse=A + 2), MISALIGNED), (dict(q=heads(A + 2)), MISALIGNED),
    (dict(k=heads(sl=0)), INVALID), (dict(v=heads(sl=64)), INVALID), (dict(v=heads(sh=4)), MISALIGNED),
    (dict(out=heads(sh=64)), INVALID), (dict(Lq=0), OK)])
def test_cross_attention_rejects_bad_arguments(L, bad, want):
    assert forward(L, **bad) == want


def backward(L, do=heads(), q=heads(), k=heads(), v=heads(), o=heads(), lse=A, lens=None, scale=0.1, B=2, H=8, Hkv=4,
             Lq=16, Lk=16, d=128, dq=heads(), dk=heads(), dv=heads(), ws=A, wsb=1 << 30):
    return L.nvfp4_cross_attention_backward(do, q, k, v, o, lse, lens, scale, B, H, Hkv, Lq, Lk, d, dq, dk, dv, ws, wsb,
                                            None, None)


@pytest.mark.parametrize("bad,want", SIZES + [
    (dict(do=heads(None)), INVALID), (dict(o=heads(A + 4)), MISALIGNED), (dict(lse=None), INVALID),
    (dict(lse=A + 2), MISALIGNED), (dict(dq=heads(sh=0)), INVALID), (dict(dk=heads(sb=0)), INVALID),
    (dict(dv=heads(A + 8)), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE),
    (dict(ws=A + 4), MISALIGNED), (dict(Lq=0, Lk=0), OK)])
def test_cross_attention_backward_rejects_bad_arguments(L, bad, want):
    assert backward(L, **bad) == want


def test_workspace_size_of_bad_sizes_is_zero(L):
    f = L.nvfp4_cross_attention_backward_workspace_bytes
    assert f(2, 8, 4, 16, 16, 128) >= 2 * 8 * 16 * 4
    assert f(2, 8, 3, 16, 16, 128) == 0 and f(2, 8, 4, 16, 16, 12) == 0 and f(-1, 8, 4, 16, 16, 128) == 0


def test_python_entry_points_reject_what_they_cannot_take():
    q, k = torch.zeros(1, 4, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 6, 2, 64, dtype=torch.bfloat16)
    w = nv.NVFP4Tensor(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8), torch.ones(1), 8, 128)
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    at = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: nv.cross_attention(q.float(), k, k), lambda: nv.cross_attention(q, k, k[:, :5]),
                 lambda: nv.cross_attention(q, k[..., :32], k[..., :32]), lambda: nv.cross_attention(q[0], k, k),
                 lambda: nv.cross_attention(q, k, k, torch.zeros(1)), lambda: nv.cross_attention(q, k, k, out=q.float()),
                 lambda: nv.cross_attention(q, k, k, torch.zeros(2, dtype=torch.int32)),
                 lambda: nv.cross_attention_backward(q, q, k, k, q, torch.zeros(1, 4, 5)),
                 lambda: nv.cross_attention_backward(q[:, :3], q, k, k, q, torch.zeros(1, 4, 4)),
                 lambda: nv.rotary(q[0], at, (32, 32)), lambda: nv.rotary(q.half(), at, (32, 32)),
                 lambda: nv.rotary(q, at, (32, 16, 16)), lambda: nv.rotary(q, at.long(), (32, 32)),
                 lambda: nv.rotary(q, at[:3], (32, 32)), lambda: nv.rotary(q, at, (32, 32), out=q[:, :2]),
                 lambda: nv.rotary(q.transpose(2, 3), at, (32, 32)),
                 lambda: nv.gemv_w4a16(x.float(), w), lambda: nv.gemv_w4a16(x[:, :64], w),
                 lambda: nv.gemv_w4a16(torch.zeros(17, 128, dtype=torch.bfloat16), w),
                 lambda: nv.gemv_w4a16(x, w, bias=torch.zeros(7)), lambda: nv.gemv_w4a16(x, w, out=torch.zeros(2, 7)),
                 # CPU tensors
                 lambda: nv.cross_attention(q, k, k), lambda: nv.rotary(q, at, (32, 32)), lambda: nv.gemv_w4a16(x, w)):
        with pytest.raises(ValueError):
            call()
