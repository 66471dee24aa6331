"""Calls at the edges of what include/nvfp4_dit.h allows: operands that share
memory, values that are not finite, other streams and contexts."""
import ctypes
import threading

import pytest
import torch

import nvfp4_w4a4_gemm_quantize_b200 as nv
from nvfp4_w4a4_gemm_quantize_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mx"])
@pytest.mark.parametrize("M", [2, 3, 8, 16])
@pytest.mark.parametrize("N,K", [(131, 256), (300, 4224)])
def test_gemv_of_one_row_expanded(cuda_ok, fmt, M, N, K):
    """A conditioning row shared by the samples: the bits of its copies."""
    w = synth.random_bf16((N, K), seed=N, scale=0.02).cuda()
    w = nv.mx_quantize(w) if fmt == "mx" else nv.quantize(w)
    row = synth.random_bf16((1, K), seed=M).cuda()
    for x in (row.expand(M, K), row[0].expand(M, K)):
        assert x.stride(0) == 0
        for dtype in (torch.float32, torch.bfloat16):
            y = nv.gemv_w4a16(x, w, out_dtype=dtype)
            assert torch.equal(y, nv.gemv_w4a16(x.contiguous(), w, out_dtype=dtype))
            assert bool((y == y[:1]).all())


@pytest.mark.parametrize("Lq", [4, 200])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lk", [1, 14, 15, 16, 31, 128, 129, 300])
def test_row_of_minus_infinity_everywhere(cuda_ok, Lq, d, Lk):
    """exp(-infinity) over a sum of nothing else is 0 / 0: NaN in both kernels,
    lse = -infinity, NaN gradients; the other sample does not notice."""
    g = torch.Generator(device="cuda").manual_seed(Lk)
    q, k, v, do = (torch.randn(2, n, 2, d, generator=g, device="cuda").bfloat16() for n in (Lq, Lk, Lk, Lq))
    q[0, ..., 0] = q[0, ..., 0].abs() + 1
    base, base_lse = nv.cross_attention(q, k, v, return_lse=True)
    base_grads = nv.cross_attention_backward(do, q, k, v, base, base_lse)
    k[0, ..., 0] = -float("inf")
    out, lse = nv.cross_attention(q, k, v, return_lse=True)
    grads = nv.cross_attention_backward(do, q, k, v, out, lse)
    assert bool(out[0].isnan().all()) and bool((lse[0] == -float("inf")).all())
    assert all(bool(t[0].isnan().all()) for t in grads)
    assert torch.equal(out[1], base[1]) and torch.equal(lse[1], base_lse[1])
    assert all(torch.equal(t[1], b[1]) for t, b in zip(grads, base_grads))


@pytest.mark.parametrize("Lk", [15, 128, 300])
def test_rows_of_minus_infinity_among_others(cuda_ok, Lk):
    """Only the rows whose logits are all -infinity become NaN: keys of -infinity
    in one column meet queries that are 1 there, and queries that are -1 see
    +infinity, NaN too; a head without such a column keeps its bits."""
    g = torch.Generator(device="cuda").manual_seed(Lk)
    q, k, v = (torch.randn(1, n, 2, 64, generator=g, device="cuda").bfloat16() for n in (200, Lk, Lk))
    base = nv.cross_attention(q, k, v)
    q[:, :, 0, 0] = torch.where(torch.arange(200, device="cuda") % 3 == 0, -1.0, 1.0).bfloat16()
    k[:, :, 0, 0] = -float("inf")
    out, lse = nv.cross_attention(q, k, v, return_lse=True)
    assert bool(out[:, :, 0].isnan().all()) and torch.equal(out[:, :, 1], base[:, :, 1])
    up = torch.arange(200, device="cuda") % 3 == 0
    assert bool((lse[0, 0, ~up] == -float("inf")).all()) and bool(lse[0, 0, up].isnan().all())


@pytest.mark.parametrize("Lq", [3, 150])
def test_gradients_off_a_16_byte_boundary(cuda_ok, Lq):
    """A contiguous gradient that starts two bytes into its storage."""
    g = torch.Generator(device="cuda").manual_seed(Lq)
    q, k, v, do = (torch.randn(2, n, 2, 64, generator=g, device="cuda").bfloat16() for n in (Lq, 40, 40, Lq))
    off = torch.empty(do.numel() + 1, device="cuda", dtype=torch.bfloat16)[1:].view_as(do).copy_(do)
    assert off.is_contiguous() and off.data_ptr() % 16 == 2
    leaves = [t.requires_grad_() for t in (q, k, v)]
    want = torch.autograd.grad(nv.CrossAttention.apply(*leaves), leaves, do)
    got = torch.autograd.grad(nv.CrossAttention.apply(*leaves), leaves, off)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    at = torch.arange(Lq, device="cuda", dtype=torch.int32)[:, None]
    want = torch.autograd.grad(nv.RotaryEmbedding.apply(q, at, (64,)), q, do)[0]
    got = torch.autograd.grad(nv.RotaryEmbedding.apply(q, at, (64,)), q, off)[0]
    assert torch.equal(got, want)


def test_the_callers_context_stays_current(cuda_ok):
    """A thread with a context of its own still has it after a call (one that
    asks for the device and has nothing to launch)."""
    torch.zeros(1, device="cuda")
    cuda = ctypes.CDLL("libcuda.so.1")
    primary, mine, after = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    assert cuda.cuCtxGetCurrent(ctypes.byref(primary)) == 0 and primary.value
    assert cuda.cuCtxCreate_v2(ctypes.byref(mine), 0, 0) == 0               # becomes current here
    assert cuda.cuCtxSetCurrent(primary) == 0
    results = []

    def work():
        results.append(cuda.cuCtxSetCurrent(mine))
        results.append(nv.lib().nvfp4_dequantize(None, None, None, 0, 64, None, nv.NVFP4_DTYPE_BF16, None))
        results.append(cuda.cuCtxGetCurrent(ctypes.byref(after)))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert cuda.cuCtxDestroy_v2(mine) == 0
    assert cuda.cuCtxSetCurrent(primary) == 0
    assert results == [0, 0, 0] and after.value == mine.value


@pytest.mark.parametrize("M", [1, 5, 16])
@pytest.mark.parametrize("spread", [0, 100])
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_gemv_of_a_nan_scale(cuda_ok, M, spread, byte):
    """E4M3's NaN makes its feature NaN in every row of x, be x's values close
    together or 2^100 apart (which are decoded in different ways), as
    dequantize() has it; the other features keep their bits."""
    N, K = 200, 640
    w = nv.quantize(synth.random_bf16((N, K), seed=1, scale=0.02).cuda())
    x = synth.random_bf16((M, K), seed=2).cuda()
    x[:, 3] *= 2.0 ** -spread
    base = nv.gemv_w4a16(x, w, out_dtype=torch.float32)
    features = torch.tensor([0, 77, 130, 199])
    for i, n in enumerate(features.tolist()):
        c = 7 * i + 2                                       # one block of 16 along k
        w.sf[(n // 128 * (K // 64) + c // 4) * 512 + n % 32 * 16 + n % 128 // 32 * 4 + c % 4] = byte
    bad = torch.zeros(N, dtype=torch.bool)
    bad[features] = True
    values = nv.dequantize(w, torch.float32)
    assert torch.equal(values.isnan().any(1).cpu(), bad)
    y = nv.gemv_w4a16(x, w, out_dtype=torch.float32)
    assert bool(y[:, bad].isnan().all()) and torch.equal(y[:, ~bad], base[:, ~bad])


def _calls_on_a_stream():
    """name: (inputs' maker, call of them on a stream)"""
    def gemv():
        w = nv.quantize(synth.random_bf16((1280, 256), seed=3, scale=0.02).cuda())
        x = synth.random_bf16((4, 256), seed=4).cuda()
        return lambda s: [nv.gemv_w4a16(x, w, out_dtype=torch.float32, stream=s)]

    def rotary():
        x = torch.randn(1, 90, 4, 64, device="cuda").bfloat16()
        at = torch.arange(90, device="cuda", dtype=torch.int32)[:, None]
        return lambda s: [nv.rotary(x, at, (64,), stream=s)]

    def attention(Lq):
        q, k, v, do = (torch.randn(2, n, 4, 64, device="cuda").bfloat16() for n in (Lq, 300, 300, Lq))
        out, lse = nv.cross_attention(q, k, v, return_lse=True)
        return lambda s: [*nv.cross_attention(q, k, v, return_lse=True, stream=s),
                          *nv.cross_attention_backward(do, q, k, v, out, lse, stream=s)]

    return {"gemv": gemv, "rotary": rotary, "few queries": lambda: attention(3), "queries": lambda: attention(200)}


@pytest.mark.parametrize("name", ["gemv", "rotary", "few queries", "queries"])
@pytest.mark.parametrize("as_int", [False, True])
def test_a_call_on_another_stream_takes_no_memory_still_in_use(cuda_ok, name, as_int):
    """The current stream has freed blocks of just the outputs' sizes, which
    work that it has still to do will write: the call on the other stream, which
    does not wait for that, neither gets nor disturbs them."""
    call = _calls_on_a_stream()[name]()
    want = call(None)
    sizes = [t.numel() * t.element_size() for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    kept = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                       # about 50 ms
    for t in freed:
        t.fill_(0x5A)
    del t, freed
    got = call(side.cuda_stream if as_int else side)
    kept.copy_(torch.full_like(kept, 3))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((kept == 3).all())


def test_results_of_another_stream_outlive_their_use_here(cuda_ok):
    """A result that the current stream still reads is not recycled by the next
    call on the stream that made it."""
    x, at = torch.randn(1, 90, 4, 64, device="cuda"), torch.arange(90, device="cuda", dtype=torch.int32)[:, None]
    other = torch.randn(1, 90, 4, 64, device="cuda")
    want = nv.rotary(x, at, (64,))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = nv.rotary(x, at, (64,), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    copy = y.clone()                                     # queued behind the sleep
    del y
    for _ in range(4):
        nv.rotary(other, at, (64,), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_second_derivatives(cuda_ok):
    """Of rotary positions: z = sum x . turn(w), so its gradient of w is the
    turned-back x, whose product with a direction has that direction, turned, as
    its gradient of x.  Of attention: refused."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w, h = (torch.randn(2, 30, 4, 64, generator=g, device="cuda") for _ in range(3))
    at = torch.arange(30, device="cuda", dtype=torch.int32)[:, None]
    for interleaved in (True, False):
        xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()
        z = (xs * nv.RotaryEmbedding.apply(ws, at, (64,), 10000.0, interleaved)).sum()
        (dw,) = torch.autograd.grad(z, ws, create_graph=True)
        assert torch.equal(dw, nv.rotary(x, at, (64,), interleaved=interleaved, inverse=True))
        (dx,) = torch.autograd.grad((dw * h).sum(), xs)
        assert torch.equal(dx, nv.rotary(h, at, (64,), interleaved=interleaved))
    q, k, v = (torch.randn(1, n, 2, 64, generator=g, device="cuda").bfloat16().requires_grad_() for n in (20, 30, 30))
    plain = torch.autograd.grad(nv.CrossAttention.apply(q, k, v).sum(), (q, k, v))
    grads = torch.autograd.grad(nv.CrossAttention.apply(q, k, v).sum(), (q, k, v), create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(grads, plain))
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(grads[1].float().pow(2).sum() + q.float().pow(2).sum(), q)


def test_training_step_with_a_status(cuda_ok):
    """The status reaches both passes (it stays 0 where no wait ran out), and
    changes nothing else."""
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(2, n, 2, 64, generator=g, device="cuda").bfloat16().requires_grad_() for n in (150, 200, 200))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plain = nv.CrossAttention.apply(q, k, v)
    out = nv.CrossAttention.apply(q, k, v, None, None, status)
    grads = [torch.autograd.grad(o.sum(), (q, k, v)) for o in (plain, out)]
    assert torch.equal(out, plain) and all(torch.equal(a, b) for a, b in zip(*grads)) and int(status.item()) == 0
    with pytest.raises(ValueError):
        nv.CrossAttention.apply(q, k, v, None, None, status.cpu())


@pytest.mark.parametrize("Lq", [4, 200])
@pytest.mark.parametrize("low", [-float("inf"), -300.0])
def test_keys_that_weigh_nothing_beside_huge_values(cuda_ok, Lq, low):
    """Keys at logits of -infinity, or 200 and more below the row's others, have
    P below 2^-250: their values of 3e38 add less than 1e-36, and a gradient of
    3e38 leaves less than 1e-36 in theirs.  (A P that stops at 2^-126 would add
    3.5.)"""
    g = torch.Generator(device="cuda").manual_seed(Lq)
    q, k, v, do = (torch.randn(1, n, 2, 64, generator=g, device="cuda").bfloat16() for n in (Lq, 300, 300, Lq))
    q[..., 0] = 8.0
    k[..., 0] = 0.0
    gone = torch.arange(300, device="cuda") % 3 != 0
    base, base_lse = nv.cross_attention(q, k[:, ~gone].contiguous(), v[:, ~gone].contiguous(), return_lse=True)
    k[:, gone, :, 0] = low                                   # logits: 8 low / 8, the rest at most 30 or so
    v[:, gone] = 3e38
    out, lse = nv.cross_attention(q, k, v, return_lse=True)
    # the same sums in another order and other tiles: both within (h + h + 2^-16) of sum P |v| <= max |v|
    bound = 2.0 * (2 * 2.0 ** -8 + 2.0 ** -16) * float(v[:, ~gone].float().abs().max())
    assert float((out.float() - base.float()).abs().max()) <= bound
    assert float((lse - base_lse).abs().max()) <= 2.0 ** -16 * float(base_lse.abs().max() + 1)
    do[:, 0] = 3e38
    dv = nv.cross_attention_backward(do, q, k, v, out, lse)[2]
    assert float(dv[:, gone].float().abs().max()) <= 1e-36
