"""nvfp4_gemv_w4a16 against the oracle's element values in 64 bits.

Products x * w are exact in FP32 (8 + 6 significant bits).  A sum takes at most
K / 16 tensor-core steps one after the other plus the joins of its parts (fewer
than 40); a step's result, and what it drops when it aligns its terms, is off by
at most 2^-22 of the terms' magnitudes, so the sum by (K / 16 + 40) 2^-22
sum |x w|.  The scale, the bias and an FP32 output round three times (2^-24 of
|g acc| + |bias| each), a bf16 output once more (2^-8)."""
import numpy as np
import pytest
import torch

import oracle
import nvfp4_w4a4_gemm_quantize_b200 as nv
from nvfp4_w4a4_gemm_quantize_b200 import synth

pytestmark = pytest.mark.gpu


def _weights(N, K, fmt, seed, dist="normal"):
    w = synth.random_bf16((N, K), seed=seed, dist=dist, scale=0.02).cuda()
    return nv.mx_quantize(w) if fmt == "mx" else nv.quantize(w)


def _values(w):
    """Element values without the tensor scale, and the tensor scale, in FP64."""
    if isinstance(w, nv.MXTensor):
        return nv.mx_dequantize(w, torch.float32).double(), 1.0
    one = nv.NVFP4Tensor(w.codes, w.sf, torch.ones_like(w.scale), w.rows, w.k)
    return nv.dequantize(one, torch.float32).double(), float(w.scale.item())


def _check(x, w, bias=None, out_dtype=torch.float32, **kw):
    y = nv.gemv_w4a16(x, w, bias=bias, out_dtype=out_dtype, **kw)
    v, g = _values(w)
    acc = x.double() @ v.T
    b = bias.double() if bias is not None else torch.zeros(w.rows, dtype=torch.float64, device="cuda")
    ref = g * acc + b
    tol = g * (w.k / 16 + 40) * 2.0 ** -22 * (x.double().abs() @ v.abs().T) + 3 * 2.0 ** -24 * (ref.abs() + 2 * b.abs())
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert y.shape == ref.shape and bool(((y.double() - ref).abs() <= tol).all())
    return y


@pytest.mark.parametrize("fmt", ["nvfp4", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 127, 256), (2, 128, 640), (3, 129, 128), (5, 257, 1152), (7, 1337, 4224),
                                   (8, 64, 5120), (9, 1000, 384), (16, 33, 2560), (16, 1152, 4096)])
def test_gemv_sizes(cuda_ok, fmt, M, N, K):
    x = synth.random_bf16((M, K), seed=M + N, dist="student_t3").cuda()
    w = _weights(N, K, fmt, seed=N + K, dist="outlier")
    bias = torch.randn(N, generator=torch.Generator().manual_seed(N)).cuda()
    _check(x, w)
    _check(x, w, bias, torch.bfloat16)
    _check(x, w, bias, torch.float32)


@pytest.mark.parametrize("K", [64, 192, 320, 1088, 4160])
def test_gemv_half_chunk_along_k(cuda_ok, K):
    _check(synth.random_bf16((3, K), seed=K).cuda(), _weights(200, K, "nvfp4", seed=K + 1))


@pytest.mark.parametrize("fmt", ["nvfp4", "mx"])
@pytest.mark.parametrize("M", [1, 6, 16])
def test_gemv_exact_sums(cuda_ok, fmt, M):
    """Small integers times E2M1 values with power-of-two scales: every partial
    sum is a multiple of 1/8 below 2^18, so any order gives the same bits."""
    N, K = 300, 3200
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.integers(-4, 5, (M, K)).astype(np.float32)).cuda().bfloat16()
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2)).astype(np.uint8)).cuda()
    if fmt == "mx":
        w = nv.MXTensor.empty(N, K, "cuda")
        w.sf.copy_(torch.from_numpy(rng.integers(125, 129, w.sf.numel()).astype(np.uint8)))
    else:
        w = nv.NVFP4Tensor.empty(N, K, "cuda")
        w.sf.copy_(torch.from_numpy((8 * rng.integers(5, 9, w.sf.numel())).astype(np.uint8)))   # 2^-2 .. 2^1
        w.scale.fill_(1.0)
    w.codes.copy_(codes)
    v, _ = _values(w)
    assert torch.equal(nv.gemv_w4a16(x, w, out_dtype=torch.float32).double(), x.double() @ v.T)


def test_gemv_every_code_and_scale(cuda_ok):
    """x picks out one weight at a time: each E2M1 code under each finite E4M3
    scale, and under E8M0 scales across bf16's range, comes back exactly."""
    K = 256
    x = torch.zeros(16, K, device="cuda", dtype=torch.bfloat16)
    x[torch.arange(16), torch.arange(16) * 16 + torch.arange(16)] = 1.0     # row m: value m of block m
    for fmt, scales in (("nvfp4", range(127)), ("mx", range(2, 252, 2))):
        rows = list(scales)
        w = nv.MXTensor.empty(len(rows), K, "cuda") if fmt == "mx" else nv.NVFP4Tensor.empty(len(rows), K, "cuda")
        codes = torch.arange(16, device="cuda", dtype=torch.uint8)
        w.codes.copy_((codes[0::2] | codes[1::2] << 4).repeat(K // 16).expand(len(rows), K // 2))
        kb = K // (32 if fmt == "mx" else 16)
        r, c = torch.arange(len(rows))[:, None], torch.arange(kb)[None]
        at = (r // 128 * (kb // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
        sf = torch.zeros(w.sf.numel(), dtype=torch.uint8)
        sf[at.reshape(-1)] = torch.tensor(rows, dtype=torch.uint8)[:, None].expand(-1, kb).reshape(-1)
        w.sf.copy_(sf)
        if fmt == "nvfp4":
            w.scale.fill_(1.0)
        v, _ = _values(w)
        assert torch.equal(nv.gemv_w4a16(x, w, out_dtype=torch.float32).double(), x.double() @ v.T), fmt


def test_gemv_strided_rows_outputs_and_repeats(cuda_ok):
    w = _weights(520, 1152, "nvfp4", seed=5)
    buf = synth.random_bf16((4, 2 * 1152), seed=6).cuda()
    x = buf[:, 1152:]
    y = _check(x, w)
    out = torch.full((4, 520), float("nan"), device="cuda", dtype=torch.bfloat16)
    assert nv.gemv_w4a16(x, w, out=out) is out
    assert torch.equal(out, y.bfloat16())
    for _ in range(3):                                      # the same bits every time
        assert torch.equal(nv.gemv_w4a16(x, w, out_dtype=torch.float32), y)
    # one row of several rows' storage: its stride is not looked at (a single row is summed in an order of its own, so
    # its bits are those of a single row, not of the four)
    assert torch.equal(_check(x[2:3], w), nv.gemv_w4a16(x[2:3].clone(), w, out_dtype=torch.float32))
    assert nv.gemv_w4a16(x[:0], w).shape == (0, 520)


@pytest.mark.parametrize("fmt", ["nvfp4", "mx"])
def test_gemv_writes_nothing_past_its_outputs(cuda_ok, fmt):
    w = _weights(131, 256, fmt, seed=7)
    buf = torch.full((3 * 131 + 64,), 7.0, device="cuda")
    x = synth.random_bf16((3, 256), seed=8).cuda()
    nv.gemv_w4a16(x, w, out=buf[: 3 * 131].view(3, 131))
    assert bool((buf[3 * 131:] == 7.0).all())


def test_gemv_extreme_rows(cuda_ok):
    """Large and tiny rows side by side keep their own precision; a NaN stays in its row."""
    w = _weights(96, 512, "nvfp4", seed=9)
    x = synth.random_bf16((4, 512), seed=10).cuda()
    x[0] *= 2.0 ** 100
    x[1] *= 2.0 ** -100
    _check(x, w)
    x[3, 17] = float("nan")
    y = nv.gemv_w4a16(x, w, out_dtype=torch.float32)
    assert bool(y[3].isnan().all()) and not bool(y[:3].isnan().any())


def test_gemv_largest_layers(cuda_ok):
    """The weights-only layers (5120 -> 20480 and back), every row and column."""
    _check(synth.random_bf16((1, 5120), seed=11).cuda(), _weights(20480, 5120, "nvfp4", seed=12), out_dtype=torch.bfloat16)
    _check(synth.random_bf16((16, 20480), seed=13).cuda(), _weights(5120, 20480, "mx", seed=14), out_dtype=torch.bfloat16)


def test_gemv_matches_the_gemm(cuda_ok):
    x, w = synth.random_bf16((16, 1152), seed=15).cuda(), _weights(1152, 1152, "nvfp4", seed=16)
    a, b = nv.gemv_w4a16(x, w, out_dtype=torch.float32), nv.gemm_w4a16(x, w, out_dtype=torch.float32)
    v, g = _values(w)
    assert bool(((a - b).abs().double() <= 2 * g * (1152 / 16 + 40) * 2.0 ** -22 * (x.double().abs() @ v.abs().T)
                 + 2.0 ** -22 * a.abs().double()).all())


def test_gemv_on_another_stream_and_in_a_graph(cuda_ok):
    w = _weights(640, 1024, "nvfp4", seed=17)
    x = synth.random_bf16((2, 1024), seed=18).cuda()
    want = nv.gemv_w4a16(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = nv.gemv_w4a16(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = nv.gemv_w4a16(x, w)
    x2 = synth.random_bf16((2, 1024), seed=19).cuda()
    want2 = nv.gemv_w4a16(x2, w)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want2)


@pytest.mark.parametrize("fmt", ["nvfp4", "mx"])
@pytest.mark.parametrize("M", [1, 2, 8, 13])
@pytest.mark.parametrize("binades", [8, 30, 31, 32, 60])
def test_gemv_values_over_many_binades(cuda_ok, fmt, M, binades):
    """Rows of x whose values span a given number of binades (on either side of
    what FP16 holds exactly) at different magnitudes, zeros among them; E8M0
    scales over as many, up to where FP32 ends."""
    N, K = 140, 1152
    g = torch.Generator(device="cuda").manual_seed(binades + M)
    e = torch.randint(0, binades + 1, (M, K), generator=g, device="cuda").double() - binades
    e[:, 0], e[:, 1] = 0, -binades
    m = 1 + torch.randint(0, 128, (M, K), generator=g, device="cuda").double() / 128
    x = m * torch.exp2(e + 7 * torch.arange(M, device="cuda")[:, None].double() - 20)
    x = torch.where(torch.rand(M, K, generator=g, device="cuda") < 0.5, x, -x)
    x[:, 5::17] = 0.0
    x = x.bfloat16()
    w = _weights(N, K, fmt, seed=binades)
    if fmt == "mx":
        w.sf.copy_(torch.randint(127, 128 + binades, (w.sf.numel(),), generator=g, device="cuda").to(torch.uint8))
    _check(x, w)


@pytest.mark.parametrize("fmt,M,N,K", [("nvfp4", 16, 230016, 128), ("nvfp4", 8, 70, 20480), ("mx", 16, 64, 40960),
                                       ("mx", 1, 40, 65536), ("nvfp4", 1, 40, 65536), ("nvfp4", 11, 33, 30016)])
def test_gemv_more_than_shared_memory_holds(cuda_ok, fmt, M, N, K):
    """Output widths whose sums, and rows of x whose parts, a block takes in several passes."""
    _check(synth.random_bf16((M, K), seed=N).cuda(), _weights(N, K, fmt, seed=K))


def test_gemv_scales_at_the_ends_of_their_range(cuda_ok):
    """E8M0 scales of 2^100 beside small ones, in some units only."""
    N, K = 256, 640
    w = _weights(N, K, "mx", seed=3)
    sf = torch.randint(100, 130, (w.sf.numel(),), device="cuda", dtype=torch.uint8)
    sf[::97] = 227
    w.sf.copy_(sf)
    for M in (1, 5, 16):
        _check(synth.random_bf16((M, K), seed=M).cuda(), w)
