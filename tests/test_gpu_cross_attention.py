"""nvfp4_cross_attention and its backward pass against the formulas in 64 bits.

Bounds per element, from the inputs in FP64 (h = 2^-8, the half step of bf16):
  a logit: q k sums d exact products in FP32, at most d / 16 + 1 dependent steps
    off by 2^-22 of sum |q k| each; its exponential's argument is rounded and
    the hardware exponential is good to 2^-22: relative error of an
    unnormalised P at most e = scale (d / 16 + 1) 2^-22 sum |q k| + 2^-20
    + 2^-22 |logit| (the largest over a row's keys: the reference maximum and
    the sum have it too, so 3 e for P);
  sums over keys or queries: at most (their number / 16 + 40) dependent steps,
    f = that times 2^-22, relative to the sum of magnitudes;
  out: P rounded to bf16 (h), summed (f), rounded (h):
    (h + 3 e + f) P |v| + h |out|;
  lse: 2 e + 2^-22 |lse|;
  dv: (h + 3 e + f) P^T |grad| + h |dv|;
  dS: P scale (h |dP - D| + 3 e |dP - D| + 2^-18 (|grad| |v|) + error of D), D
    from the rounded out: sum |grad| * (error of out) + 2^-18 sum |grad out|
    (sums over d <= 128: at most 16 steps);
  dq, dk: the errors of dS times |k|, |q|, plus f |dS| |k| ..., plus h |dq|;
  in the gradients P = exp(scale q k - lse) comes out as zero where it is below
    the least normal number u = 2^-126 (the hardware exponential flushes it):
    at most u off, so u more in every P of dv, u scale |dP - D| more in dS."""
import math
import threading

import pytest
import torch

import nvfp4_w4a4_gemm_quantize_b200 as nv

pytestmark = pytest.mark.gpu

H8, F, U = 2.0 ** -8, 2.0 ** -18, 2.0 ** -126


def _inputs(B, Lq, Lk, H, Hkv, d, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn(B, n, h, d, generator=g, device="cuda").mul_(s).bfloat16()
                   for n, h, s in ((Lq, H, std), (Lk, Hkv, 1.0), (Lk, Hkv, 1.0), (Lq, H, 1.0)))
    return q, k, v, do


def _lens(lens, B, Lk):
    return [Lk] * B if lens is None else [min(max(n, 0), Lk) for n in lens]


def _reference(q, k, v, lens, scale, do=None):
    """FP64 values and bounds: {"out": (value, bound), ...}."""
    B, Lq, H, d = q.shape
    Lk, Hkv = k.shape[1:3]
    G = H // Hkv
    fk, fq = ((n / 16 + 40) * 2.0 ** -22 for n in (Lk, Lq * G))
    qd, kd, vd = (t.double().transpose(1, 2) for t in (q, k, v))            # [B, heads, tokens, d]
    kd, vd = (t.repeat_interleave(G, 1) for t in (kd, vd))
    keep = torch.arange(Lk, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]
    kd, vd = (torch.where(keep[:, None, :, None], t, 0.0) for t in (kd, vd))
    s = scale * qd @ kd.transpose(2, 3)
    e = (scale * (d / 16 + 1) * 2.0 ** -22 * (qd.abs() @ kd.abs().transpose(2, 3)) + 2.0 ** -20 + 2.0 ** -22 * s.abs())
    e = torch.where(keep[:, None, None], e, 0.0).amax(3, keepdim=True) if Lk else e.new_zeros(B, H, Lq, 1)
    s = s.masked_fill(~keep[:, None, None], -math.inf)
    lse = torch.logsumexp(s, 3) if Lk else s.new_full((B, H, Lq), -math.inf)
    p = torch.where(torch.isfinite(lse)[..., None], torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)[..., None]), 0.0)
    out = p @ vd
    tol = (H8 + 3 * e + fk) * (p @ vd.abs()) + H8 * out.abs()
    res = {"out": (out.transpose(1, 2), tol.transpose(1, 2)), "lse": (lse, 2 * e[..., 0] + 2.0 ** -22 * lse.abs())}
    if do is not None:
        g = do.double().transpose(1, 2)
        dp, D = g @ vd.transpose(2, 3), (g * out).sum(3, keepdim=True)
        eD = (g.abs() * tol).sum(3, keepdim=True) + F * (g * out).abs().sum(3, keepdim=True)
        ds = p * (dp - D) * scale
        eds = p * scale * ((H8 + 3 * e) * (dp - D).abs() + F * (g.abs() @ vd.abs().transpose(2, 3)) + eD)
        eds = eds + torch.where(keep[:, None, None], U * scale * (dp - D).abs(), 0.0)

        def shared(t):                       # [B, H, Lk, d] summed over the heads that share a key
            return t.reshape(B, Hkv, G, Lk, d).sum(2).transpose(1, 2)

        dq, dk, dv = ds @ kd, shared(ds.transpose(2, 3) @ qd), shared(p.transpose(2, 3) @ g)
        edq = eds @ kd.abs() + fk * (ds.abs() @ kd.abs()) + H8 * dq.abs()
        edk = shared(eds.transpose(2, 3) @ qd.abs() + fq * (ds.abs().transpose(2, 3) @ qd.abs())) + H8 * dk.abs()
        edv = shared((torch.where(keep[:, None, None], U, 0.0) + (H8 + 3 * e + fq) * p).transpose(2, 3) @ g.abs()) + H8 * dv.abs()
        res |= {"dq": (dq.transpose(1, 2), edq.transpose(1, 2)), "dk": (dk, edk), "dv": (dv, edv)}
    return res


def _within(got, want, what):
    ref, tol = want
    assert got.shape == ref.shape, what
    a, b = got.double(), ref.double()
    same = (a == b) | ((a - b).abs() <= tol * 1.001 + 1e-37)
    assert bool(same.all()), (what, float(((a - b).abs() / (tol + 1e-37))[~same].max()), int((~same).sum()))


def _device_lens(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


def _check(q, k, v, lens=None, scale=None, do=None):
    sc = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    n, dl = _lens(lens, q.shape[0], k.shape[1]), _device_lens(lens)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _reference(q, k, v, n, sc, do)
    out, lse = nv.cross_attention(q, k, v, dl, scale, return_lse=True, dev_status=st)
    _within(out, want["out"], "out")
    _within(lse, want["lse"], "lse")
    assert torch.equal(nv.cross_attention(q, k, v, dl, scale), out)         # without lse, and the same bits again
    grads = ()
    if do is not None:
        grads = nv.cross_attention_backward(do, q, k, v, out, lse, dl, scale, dev_status=st)
        for name, got in zip(("dq", "dk", "dv"), grads):
            _within(got, want[name], name)
        again = nv.cross_attention_backward(do, q, k, v, out, lse, dl, scale)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))
    assert int(st.item()) == 0
    return (out, lse, *grads)


@pytest.mark.parametrize("d", [8, 40, 64, 72, 96, 104, 128])
@pytest.mark.parametrize("Lq,Lk", [(130, 77), (257, 300)])
def test_head_widths(cuda_ok, d, Lq, Lk):
    q, k, v, do = _inputs(2, Lq, Lk, 3, 3, d, seed=d)
    _check(q, k, v, [Lk, Lk // 3], do=do)


@pytest.mark.parametrize("Lk", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513, 1100])
@pytest.mark.parametrize("d", [64, 128])
def test_key_lengths(cuda_ok, Lk, d):
    q, k, v, do = _inputs(1, 150, Lk, 2, 2, d, seed=Lk)
    _check(q, k, v, do=do)


@pytest.mark.parametrize("Lq", [1, 2, 3, 7, 8, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 255, 256, 257, 384, 385, 700])
@pytest.mark.parametrize("d", [72, 128])
def test_query_lengths(cuda_ok, Lq, d):
    q, k, v, do = _inputs(2, Lq, 140, 2, 2, d, seed=Lq)
    _check(q, k, v, [140, 33], do=do)


@pytest.mark.parametrize("lens", [[0, 0, 0], [0, 77, 5], [1, 0, 200], [-4, 201, 9999], [128, 129, 16], [200, 127, 144]])
@pytest.mark.parametrize("Lq", [3, 200])
def test_valid_lengths(cuda_ok, lens, Lq):
    """Empty samples give zeros and lse = -inf, lengths out of range are clamped."""
    q, k, v, do = _inputs(3, Lq, 200, 4, 2, 64, seed=7)
    out, lse, dq, dk, dv = _check(q, k, v, lens, do=do)
    for b, n in enumerate(_lens(lens, 3, 200)):
        if n == 0:
            assert not out[b].any() and bool((lse[b] == -math.inf).all()) and not dq[b].any()
        assert not dk[b, n:].any() and not dv[b, n:].any()


@pytest.mark.parametrize("lens", [[300, 5, 0, 129, 128], [1, 2, 128, 0, 0], [129, 300, 256, 257, 300], [0, 0, 0, 0, 127]])
def test_samples_of_one_and_more_key_tiles(cuda_ok, lens):
    """Samples whose states fill one tile of keys beside longer and empty ones."""
    q, k, v, do = _inputs(5, 150, 300, 4, 2, 72, seed=21)
    dq = _check(q, k, v, lens, do=do)[2]
    assert not any(dq[b].any() for b, n in enumerate(lens) if n == 0)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (6, 2), (8, 4), (16, 1), (20, 1)])
@pytest.mark.parametrize("Lq", [1, 4, 140])
def test_shared_heads(cuda_ok, H, Hkv, Lq):
    q, k, v, do = _inputs(2, Lq, 190, H, Hkv, 72, seed=H)
    _check(q, k, v, [190, 101], do=do)


@pytest.mark.parametrize("B,H,Lq,Lk,d", [(1, 1, 1, 1, 128), (1, 2, 1, 4097, 64), (8, 16, 1, 1500, 64), (3, 4, 5, 3000, 128),
                                         (40, 8, 1, 333, 96), (1, 1, 16, 20000, 128), (2, 3, 11, 700, 8)])
def test_few_queries(cuda_ok, B, H, Lq, Lk, d):
    q, k, v, _ = _inputs(B, Lq, Lk, H, H, d, seed=Lk)
    _check(q, k, v, [max(0, Lk - 97 * b) for b in range(B)])


@pytest.mark.parametrize("std", [0.0, 30.0])
@pytest.mark.parametrize("Lq", [2, 140])
def test_flat_and_sharp_rows(cuda_ok, std, Lq):
    """Equal logits, and rows that one key rules (logits in the hundreds)."""
    q, k, v, do = _inputs(1, Lq, 400, 2, 2, 128, seed=3, std=std)
    _check(q, k, v, do=do)


@pytest.mark.parametrize("Lq", [4, 300])
def test_rising_maxima_and_scales(cuda_ok, Lq):
    """Keys sorted by their logit, so that every tile moves the maximum, up and
    down; a scale of its own."""
    q, k, v, do = _inputs(1, Lq, 520, 1, 1, 64, seed=4)
    q = q[:, :1].expand(1, Lq, 1, 64).contiguous()
    for descending in (False, True):
        order = (k[0, :, 0].float() @ q[0, 0, 0].float()).argsort(descending=descending)
        _check(q, k[:, order].contiguous(), v, do=do)
    _check(q, k, v, scale=0.7, do=do)
    _check(q, k, v, scale=1e-3, do=do)


@pytest.mark.parametrize("Lq", [3, 150])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_states_past_the_length_are_not_read(cuda_ok, Lq, junk):
    q, k, v, do = _inputs(3, Lq, 300, 2, 2, 72, seed=5)
    lens = [131, 0, 288]
    base = _check(q, k, v, lens, do=do)
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = junk, junk
    dl = _device_lens(lens)
    out, lse = nv.cross_attention(q, k, v, dl, return_lse=True)
    got = (out, lse, *nv.cross_attention_backward(do, q, k, v, out, lse, dl))
    assert all(torch.equal(a, b) for a, b in zip(base, got))


@pytest.mark.parametrize("Lq", [4, 200])
@pytest.mark.parametrize("first", [1, 100, 128, 140, 270])
def test_keys_of_minus_infinity(cuda_ok, Lq, first):
    """Keys whose logits are -infinity weigh nothing, be they whole tiles."""
    q, k, v, _ = _inputs(1, Lq, 300, 2, 2, 64, seed=17)
    q[..., 0] = q[..., 0].abs() + 1
    want = _reference(q, k[:, first:], v[:, first:], [300 - first], 0.125)
    k[:, :first, :, 0] = -math.inf
    out, lse = nv.cross_attention(q, k, v, return_lse=True)
    _within(out, want["out"], "out")
    _within(lse, want["lse"], "lse")


@pytest.mark.parametrize("Lq", [4, 200])
def test_non_finite_query_stays_in_its_row(cuda_ok, Lq):
    q, k, v, _ = _inputs(2, Lq, 90, 2, 2, 64, seed=6)
    base = nv.cross_attention(q, k, v)
    q[1, 2, 1, 7] = float("nan")
    got = nv.cross_attention(q, k, v)
    assert bool(got[1, 2, 1].isnan().all())
    got[1, 2, 1] = base[1, 2, 1]
    assert torch.equal(got, base)


@pytest.mark.parametrize("Lq", [5, 200])
def test_views_broadcasts_and_neighbours(cuda_ok, Lq):
    """Parts of fused projections, head-major layouts, a batch that shares its
    states, an output view: the same bits as contiguous copies, and nothing
    outside the output's elements is written."""
    B, Lk, H, d = 2, 150, 4, 72
    g = torch.Generator(device="cuda").manual_seed(1)
    qx = torch.randn(B, Lq, 3, H, d, generator=g, device="cuda").bfloat16()[:, :, 1]
    kv = torch.randn(B, H, 2, Lk, d, generator=g, device="cuda").bfloat16()
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    do = torch.randn(B, H, Lq, d, generator=g, device="cuda").bfloat16().transpose(1, 2)
    lens = [150, 47]
    base = _check(*(t.contiguous() for t in (qx, k, v)), lens, do=do.contiguous())
    got = _check(qx, k, v, lens, do=do)
    assert all(torch.equal(a, b) for a, b in zip(base, got))
    buf = torch.full((B, Lq + 1, H + 1, d), 5.0, device="cuda", dtype=torch.bfloat16)
    nv.cross_attention(qx, k, v, _device_lens(lens), out=buf[:, :Lq, :H])
    assert torch.equal(buf[:, :Lq, :H], base[0]) and bool((buf[:, Lq] == 5.0).all()) and bool((buf[:, :, H] == 5.0).all())
    one_k, one_v = k[:1, :, :1], v[:1, :, :1]
    a = _check(qx, one_k.expand(B, Lk, H, d), one_v.expand(B, Lk, H, d), lens, do=do)
    b = _check(qx, one_k.repeat(B, 1, H, 1), one_v.repeat(B, 1, H, 1), lens, do=do)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_queries_and_no_keys(cuda_ok):
    q, k, v, do = _inputs(2, 5, 0, 2, 2, 64)
    out, lse = nv.cross_attention(q, k, v, return_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())
    dq, dk, dv = nv.cross_attention_backward(do, q, k, v, out, lse)
    assert not dq.any() and dk.shape == k.shape
    q, k, v, do = _inputs(2, 0, 9, 2, 2, 64)
    out, lse = nv.cross_attention(q, k, v, return_lse=True)
    dq, dk, dv = nv.cross_attention_backward(do, q, k, v, out, lse)
    assert out.shape == q.shape and not dk.any() and not dv.any() and dq.shape == q.shape


def _loss64(q, k, v, lens, scale, do):
    """sum(do * attention) in FP64, autograd-free."""
    return float((_reference(q, k, v, lens, scale)["out"][0] * do.double()).sum())


def test_gradient_against_differences(cuda_ok):
    """Central differences of the FP64 formula along random directions; the step
    1e-4 leaves an error of order 1e-8 of the third derivative."""
    B, Lq, Lk, H, Hkv, d = 2, 70, 50, 4, 2, 40
    q, k, v, do = _inputs(B, Lq, Lk, H, Hkv, d, seed=9)
    lens, scale = [50, 21], 1 / math.sqrt(d)
    grads = _check(q, k, v, lens, do=do)[2:]
    bounds = _reference(q, k, v, lens, scale, do)
    g = torch.Generator(device="cuda").manual_seed(2)
    for i, name in enumerate(("dq", "dk", "dv")):
        x = [t.double() for t in (q, k, v)]
        h = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-4 * h, x[i] - 1e-4 * h
        diff = (_loss64(*up, lens, scale, do) - _loss64(*down, lens, scale, do)) / 2e-4
        mine = float((grads[i].double() * h).sum())
        assert abs(diff - mine) <= float((bounds[name][1] * h.abs()).sum()) + 1e-4 * abs(diff)


def test_autograd_function(cuda_ok):
    """Gradients of views, of a broadcast and of a gradient that arrives with
    zero strides; kv_lens and scale pass through."""
    q0, k0, v0, _ = _inputs(2, 140, 90, 4, 4, 64, seed=11)
    lens = torch.tensor([90, 31], dtype=torch.int32, device="cuda")
    q = q0.clone().requires_grad_()
    k, v = k0[:1, :, :1].clone().requires_grad_(), v0[:1, :, :1].clone().requires_grad_()
    out = nv.CrossAttention.apply(q, k.expand(2, 90, 4, 64), v.expand(2, 90, 4, 64), lens, 0.2)
    dq, dk, dv = torch.autograd.grad(out.sum(), (q, k, v))
    ke, ve = k0[:1, :, :1].repeat(2, 1, 4, 1), v0[:1, :, :1].repeat(2, 1, 4, 1)
    want = _reference(q0, ke, ve, [90, 31], 0.2, torch.ones_like(q0))
    _within(out, want["out"], "out")
    _within(dq, want["dq"], "dq")
    for got, name in ((dk, "dk"), (dv, "dv")):
        ref, tol = (t.sum((0, 2), keepdim=True) for t in want[name])
        # the sum of eight bf16 gradients in bf16: at most eight more half steps of the terms' magnitudes
        tol = tol + 8 * H8 * want[name][0].abs().sum((0, 2), keepdim=True)
        _within(got, (ref, tol), name)


@pytest.mark.parametrize("Lq", [2, 200])
def test_offsets_past_32_bits(cuda_ok, Lq):
    """Samples and heads more than 2^31 elements apart."""
    far, d = 2 ** 31 + 64, 64
    buf = torch.empty(3 * far, device="cuda", dtype=torch.bfloat16)

    def spread(t, at):
        b, n, h, _ = t.shape
        s = buf[at:].as_strided((b, n, h, d), (far, d, 1 << 24, 1))
        s.copy_(t)
        return s

    q, k, v, do = _inputs(2, Lq, 100, 2, 2, d, seed=12)
    base = _check(q, k, v, [100, 60], do=do)
    got = _check(spread(q, 0), spread(k, 1 << 20), spread(v, 2 << 20), [100, 60], do=spread(do, 3 << 20))
    assert all(torch.equal(a, b) for a, b in zip(base, got))
    out = spread(torch.zeros_like(q), 4 << 20)
    nv.cross_attention(q, k, v, _device_lens([100, 60]), out=out)
    assert torch.equal(out, base[0])


@pytest.mark.parametrize("B,Lq,Lk,H,d,lens", [(2, 4096, 300, 16, 72, [300, 171]), (1, 8192, 512, 24, 128, None),
                                              (1, 3000, 2100, 3, 128, [2049])])
def test_block_sizes(cuda_ok, B, Lq, Lk, H, d, lens):
    """Image and video blocks: many work items a CTA, both passes."""
    q, k, v, do = _inputs(B, Lq, Lk, H, H, d, seed=13)
    _check(q, k, v, lens, do=do)


def test_calls_from_new_threads(cuda_ok):
    """The first CUDA call of a thread (as in an autograd worker)."""
    q, k, v, do = _inputs(1, 130, 40, 2, 2, 64, seed=16)
    out, lse = nv.cross_attention(q, k, v, return_lse=True)
    want = nv.cross_attention_backward(do, q, k, v, out, lse)
    got, buf = [], torch.empty_like(out)
    torch.cuda.synchronize()
    for call in (lambda: nv.cross_attention(q, k, v, out=buf),
                 lambda: got.extend(nv.cross_attention_backward(do, q, k, v, out, lse))):
        t = threading.Thread(target=call)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert torch.equal(buf, out) and len(got) == 3 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_threads_with_other_head_widths(cuda_ok):
    """Two threads on two streams, calls of different sizes of every kernel at
    the same time: each gets its own answers, none is refused."""
    jobs = [(_inputs(1, 130, 40, 2, 2, d, seed=d), _inputs(1, 3, 200, 2, 2, d, seed=d + 1)) for d in (64, 128)]
    w = [nv.quantize(torch.randn(256, k, device="cuda").bfloat16()) for k in (128, 4096)]
    x = [torch.randn(m, k, device="cuda").bfloat16() for m, k in ((1, 128), (16, 4096))]

    def run(i):
        res = []
        for q, k, v, do in jobs[i]:
            out, lse = nv.cross_attention(q, k, v, return_lse=True)
            res += [out, *nv.cross_attention_backward(do, q, k, v, out, lse)]
        return [*res, nv.gemv_w4a16(x[i], w[i])]

    want, got, errors = [run(0), run(1)], [None, None], []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    got[i] = run(i)
        except Exception as e:                       # noqa: BLE001 - reported by the test
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(torch.equal(a, b) for i in range(2) for a, b in zip(got[i], want[i]))


@pytest.mark.parametrize("Lq", [1, 300])
def test_two_streams_and_a_graph(cuda_ok, Lq):
    """Two calls at once on two streams; the training step captured and replayed
    with other inputs and lengths while an eager graph of the same tensors lives
    (the capture has leaves of its own, as CrossAttention asks)."""
    q, k, v, do = _inputs(2, Lq, 200, 4, 4, 64, seed=14)
    lens = torch.tensor([200, 64], dtype=torch.int32, device="cuda")
    want = nv.cross_attention(q, k, v, lens, return_lse=True)
    grads = nv.cross_attention_backward(do, q, k, v, *want, lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for s in streams * 3:
        o, l = nv.cross_attention(q, k, v, lens, return_lse=True, stream=s)
        got.append((o, l, nv.cross_attention_backward(do, q, k, v, o, l, lens, stream=s)))
    torch.cuda.synchronize()
    for o, l, gr in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1]) and all(torch.equal(a, b) for a, b in zip(gr, grads))

    tensors = [t.clone().requires_grad_() for t in (q, k, v)]
    eager = nv.CrossAttention.apply(*tensors, lens)                      # lives through the capture
    leaves = [t.detach().requires_grad_() for t in tensors]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(nv.CrossAttention.apply(*leaves, lens), leaves, do)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.CrossAttention.apply(*leaves, lens)
        gr = torch.autograd.grad(out, leaves, do)
    new = _inputs(2, Lq, 200, 4, 4, 64, seed=15)
    with torch.no_grad():
        for t, n in zip(leaves, new):
            t.copy_(n)
    do.copy_(new[3])
    lens.copy_(torch.tensor([17, 190], dtype=torch.int32))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    o, l = nv.cross_attention(*new[:3], lens, return_lse=True)
    again = nv.cross_attention_backward(new[3], *new[:3], o, l, lens)
    assert torch.equal(out, o) and all(torch.equal(a, b) for a, b in zip(gr, again))
    assert torch.equal(eager, want[0])
    del eager
