"""Cases of the operators around a diffusion transformer block's linear layers,
with their plain forms in elementary torch operations:

  gemv    Y[m, n] = g sum_k x[m, k] e2m1(w[n, k]) s[n, k / block] + bias[n] for a few rows m,
          the weights 4-bit in the library's two formats (NVFP4: E4M3 scales per 16 values and a
          tensor scale g; MX: E8M0 scales per 32 values, g = 1)
  rotary  rotary positions with several axes (time, height, width): every pair of a head's values
          turns by position[axis] theta^(-2 i / axis width); the backward pass turns back
  xattn   attention of queries to an encoder's states of another length, each sample with its own
          number of valid states; `train` also returns the gradients of q, k and v
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
MOST_GEMV = 20480 * 5120
MOST_ROTARY = 32768 * 24 * 128
MOST_SCORES = 32768 * 512 * 24


def listed():
    return [
        # adaLN modulation of one sample: shift, scale and gate of both halves of a 1152-wide block, in FP32 for the
        # norm kernel that reads them
        {"name": "gemv-modulation", "op": "gemv", "m": 1, "n": 6912, "k": 1152, "fmt": "nvfp4", "f32": True, "bias": True},
        # a conditioning row through the largest weights-only layer the library is measured on (5120 -> 20480)
        {"name": "gemv-fc1-one-row", "op": "gemv", "m": 1, "n": 20480, "k": 5120, "fmt": "nvfp4", "f32": False, "bias": False},
        # sixteen samples through the opposite layer (20480 -> 5120), MX weights
        {"name": "gemv-fc2-mx", "op": "gemv", "m": 16, "n": 5120, "k": 20480, "fmt": "mx", "f32": False, "bias": False},
        # odd sizes: three rows, an output width that no tile divides, a last half chunk along k
        {"name": "gemv-odd", "op": "gemv", "m": 3, "n": 1337, "k": 4160, "fmt": "nvfp4", "f32": True, "bias": False},
        # queries of the 16 x 32 x 64 video grid (24 heads of 128), a view into the fused projection, forward and backward
        {"name": "rotary-video-train", "op": "rotary", "b": 1, "grid": "16,32,64", "h": 24, "d": 128, "axes": "44,42,42",
         "pairs": True, "fused": True, "f32": False, "train": True, "start": 0},
        # image tokens of two samples, 16 heads of 72, split halves, height and width only
        {"name": "rotary-image", "op": "rotary", "b": 2, "grid": "1,61,67", "h": 16, "d": 72, "axes": "0,36,36",
         "pairs": False, "fused": True, "f32": False, "train": False, "start": 0},
        # one new frame of a long stream: few tokens at far positions, FP32, a part of the head unrotated
        {"name": "rotary-frame", "op": "rotary", "b": 1, "grid": "1,7,9", "h": 8, "d": 64, "axes": "16,20,20",
         "pairs": True, "fused": False, "f32": True, "train": False, "start": 100003},
        # 1024-pixel images and their captions of up to 300 text tokens: two samples, 16 heads of 72
        {"name": "xattn-image-text", "op": "xattn", "b": 2, "lq": 4096, "lk": 300, "h": 16, "hkv": 16, "d": 72,
         "lens": "300,171", "train": False},
        # the video grid's 32768 tokens and 512 text tokens, 24 heads of 128
        {"name": "xattn-video", "op": "xattn", "b": 1, "lq": 32768, "lk": 512, "h": 24, "hkv": 24, "d": 128, "lens": "",
         "train": False},
        # a training step of the same heads on two clips
        {"name": "xattn-video-train", "op": "xattn", "b": 2, "lq": 8192, "lk": 512, "h": 24, "hkv": 24, "d": 128,
         "lens": "512,389", "train": True},
        # shared key/value heads, odd lengths, one sample without any text
        {"name": "xattn-odd-train", "op": "xattn", "b": 3, "lq": 1237, "lk": 77, "h": 12, "hkv": 4, "d": 64,
         "lens": "77,0,13", "train": True},
        # one query token a sample over an encoder's 1500 states
        {"name": "xattn-one-token", "op": "xattn", "b": 8, "lq": 1, "lk": 1500, "h": 16, "hkv": 16, "d": 64,
         "lens": "1500,1500,1311,1500,750,1500,1099,1500", "train": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "rotary", "xattn", "xattn", "one"])
    if op == "gemv":
        fmt = rng.choice(["nvfp4", "nvfp4", "mx"])
        unit = 128 if fmt == "mx" else 64
        k = max(1, _log(rng, 256, 20480) // unit) * unit
        n = max(1, _log(rng, 64, min(24576, MOST_GEMV // k)))
        return {"op": "gemv", "m": _log(rng, 1, 16), "n": n, "k": k, "fmt": fmt, "f32": rng.random() < 0.5,
                "bias": rng.random() < 0.5}
    if op == "rotary":
        d = rng.choice([64, 72, 80, 96, 128])
        h = rng.randint(1, 32)
        b = rng.randint(1, 3)
        left = _log(rng, 4, max(4, MOST_ROTARY // (h * d * b)))
        t = rng.randint(1, max(1, min(24, left // 2)))
        y = max(1, int(math.sqrt(left / t)))
        x = max(1, left // (t * y))
        third = d // 3 // 2 * 2
        axes = rng.choice([(d - 2 * third, third, third), (0, d // 2, d // 2), (d // 4, d // 4, d // 4)])
        return {"op": "rotary", "b": b, "grid": "%d,%d,%d" % (t, y, x), "h": h, "d": d, "axes": "%d,%d,%d" % axes,
                "pairs": rng.random() < 0.5, "fused": rng.random() < 0.5, "f32": rng.random() < 0.3,
                "train": rng.random() < 0.5, "start": rng.choice([0, 0, _log(rng, 10, 200000)])}
    if op == "one":
        b, hkv = _log(rng, 1, 16), rng.choice([2, 4, 8, 16])
        g = rng.choice([1, 1, 2, 4])
        lk, d = _log(rng, 16, 4096), rng.choice([64, 72, 96, 128])
        return {"op": "xattn", "b": b, "lq": rng.choice([1, 1, 2, 4]), "lk": lk, "h": hkv * g, "hkv": hkv, "d": d,
                "lens": ",".join(str(rng.randint(0, lk)) for _ in range(b)), "train": False}
    b, hkv, d = rng.randint(1, 4), rng.choice([1, 2, 3, 4, 8, 12, 16]), rng.choice([40, 64, 72, 80, 96, 104, 128])
    g = rng.choice([1, 1, 2, 3])
    train = rng.random() < 0.5
    lk = _log(rng, 8, 2048)
    lq = _log(rng, 17, max(18, min(32768, MOST_SCORES // (b * hkv * g * lk * (4 if train else 1)))))
    lens = rng.choice(["", ",".join(str(rng.choice([lk, rng.randint(0, lk)])) for _ in range(b))])
    return {"op": "xattn", "b": b, "lq": lq, "lk": lk, "h": hkv * g, "hkv": hkv, "d": d, "lens": lens, "train": train}


def _ints(text):
    return [int(v) for v in text.split(",")] if text else []


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _quantized(w, fmt):
    """(codes, scale bytes in the tensor-core layout, tensor scale) of FP32 weights [n, k]."""
    n, k = w.shape
    block = 32 if fmt == "mx" else 16
    peak = w.reshape(n, k // block, block).abs().amax(2)
    if fmt == "mx":
        e = (torch.floor(torch.log2(peak.clamp(min=1e-37))) - 2).clamp(-127, 127)
        byte, s, g = (e + 127).to(torch.uint8), torch.exp2(e), torch.ones(1, device=w.device)
    else:
        g = (w.abs().amax() / 2688).reshape(1)
        sf = (peak / (6 * g)).clamp(max=448).to(torch.float8_e4m3fn)
        byte, s = sf.view(torch.uint8), sf.float() * g
    q = (w.reshape(n, k // block, block) / s.clamp(min=1e-37)[:, :, None]).reshape(n, k)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(q.abs(), mid).to(torch.uint8) | (q < 0).to(torch.uint8) * 8
    codes = code[:, 0::2] | code[:, 1::2] << 4
    rows, kb = -(-n // 128) * 128, k // block
    full = torch.zeros(rows, kb, dtype=torch.uint8, device=w.device)
    full[:n] = byte
    sf = full.reshape(rows // 128, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return codes.contiguous(), sf, g


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "gemv":
        s["x"] = _normal(g, case["m"], case["k"]).bfloat16()
        s["codes"], s["sf"], s["scale"] = _quantized(_normal(g, case["n"], case["k"], std=0.015), case["fmt"])
        s["bias"] = _normal(g, case["n"], std=0.1) if case["bias"] else None
        s["values"] = torch.tensor(E2M1, device="cuda")
    elif case["op"] == "rotary":
        b, h, d = case["b"], case["h"], case["d"]
        grid = _ints(case["grid"])
        tokens = grid[0] * grid[1] * grid[2]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        if case["fused"]:
            s["x"] = _normal(g, b, tokens, 3, h, d).to(dt)[:, :, 0]
        else:
            s["x"] = _normal(g, b, tokens, h, d).to(dt)
        s["dy"] = _normal(g, b, tokens, h, d).to(dt) if case["train"] else None
        at = torch.arange(tokens, device="cuda", dtype=torch.int32)
        s["positions"] = torch.stack([at // (grid[1] * grid[2]) + case["start"], at // grid[2] % grid[1], at % grid[2]], 1)
    else:
        b, h, hkv, d = case["b"], case["h"], case["hkv"], case["d"]
        s["q"] = _normal(g, b, case["lq"], h, d).bfloat16()
        kv = _normal(g, b, case["lk"], 2, hkv, d).bfloat16()
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        s["lens"] = torch.tensor(_ints(case["lens"]), dtype=torch.int32, device="cuda") if case["lens"] else None
        s["do"] = _normal(g, b, case["lq"], h, d).bfloat16() if case["train"] else None
    return s


# ----------------------------------------------------------------- plain forms (32 bits, rounded once)
def _weights(s):
    case = s["case"]
    n, k, block = case["n"], case["k"], 32 if case["fmt"] == "mx" else 16
    q = torch.stack([s["values"][(s["codes"] & 15).long()], s["values"][(s["codes"] >> 4).long()]], 2)
    byte = s["sf"].reshape(-1, k // block // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, k // block)[:n]
    sf = torch.exp2(byte.float() - 127) if case["fmt"] == "mx" else byte.contiguous().view(torch.float8_e4m3fn).float()
    return (q.reshape(n, k // block, block) * sf[:, :, None]).reshape(n, k)


def _gemv(s):
    y = s["x"].float() @ _weights(s).T * s["scale"]
    y = y + s["bias"] if s["bias"] is not None else y
    return y if s["case"]["f32"] else y.bfloat16()


def _angles(s):
    """FP64 angle of every token and rotated pair [tokens, pairs]."""
    at = s["positions"].double()
    return torch.cat([at[:, a, None] * 10000.0 ** (-torch.arange(0, w, 2, device="cuda").double() / w)
                      for a, w in enumerate(_ints(s["case"]["axes"])) if w], 1)


def _turn(x, angle, pairs):
    """x [b, tokens, h, d] with its first 2 * pairs values turned, in FP32, rounded to x's type."""
    n = angle.shape[1]
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    f = x.float()
    lo, hi = (f[..., 0:2 * n:2], f[..., 1:2 * n:2]) if pairs else (f[..., :n], f[..., n:2 * n])
    a, b = lo * c - hi * sn, lo * sn + hi * c
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, f[..., 2 * n:]], -1).to(x.dtype)


def _rotary(s):
    angle = _angles(s)
    y = _turn(s["x"], angle, s["case"]["pairs"])
    return (y, _turn(s["dy"], -angle, s["case"]["pairs"])) if s["case"]["train"] else y


def _xattn(s):
    case = s["case"]
    b, lq, lk, h, hkv, d = (case[n] for n in ("b", "lq", "lk", "h", "hkv", "d"))
    g, scale = h // hkv, 1.0 / math.sqrt(d)
    q = s["q"].float().reshape(b, lq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * lq, d)
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    p = q @ k.transpose(2, 3) * scale
    if s["lens"] is not None:
        gone = torch.arange(lk, device="cuda") >= s["lens"][:, None]
        p = p.masked_fill(gone[:, None, None], -math.inf)
    p = torch.exp(p - p.amax(3, keepdim=True).clamp(min=-1e30))
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    out = p @ v
    if not case["train"]:
        return _heads(out, case).bfloat16()
    do = s["do"].float().reshape(b, lq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * lq, d)
    dv = p.transpose(2, 3) @ do
    ds = p * (do @ v.transpose(2, 3) - (do * out).sum(3, keepdim=True)) * scale
    return (_heads(out, case).bfloat16(), _heads(ds @ k, case).bfloat16(),
            (ds.transpose(2, 3) @ q).transpose(1, 2).bfloat16(), dv.transpose(1, 2).bfloat16())


def _heads(t, case):
    """[b, hkv, group * lq, d] to [b, lq, h, d]."""
    b, lq, h, hkv, d = (case[n] for n in ("b", "lq", "h", "hkv", "d"))
    return t.reshape(b, hkv, h // hkv, lq, d).permute(0, 3, 1, 2, 4).reshape(b, lq, h, d)


# ----------------------------------------------------------------- the framework's operators
def _own_gemv(s):
    import nvfp4_w4a4_gemm_quantize_b200 as nv

    case = s["case"]
    if case["fmt"] == "mx":
        w = nv.MXTensor(s["codes"], s["sf"], case["n"], case["k"])
    else:
        w = nv.NVFP4Tensor(s["codes"], s["sf"], s["scale"], case["n"], case["k"])
    return nv.gemv_w4a16(s["x"], w, bias=s["bias"], out_dtype=torch.float32 if case["f32"] else torch.bfloat16)


def _own_rotary(s):
    import nvfp4_w4a4_gemm_quantize_b200 as nv

    case = s["case"]
    axes = tuple(_ints(case["axes"]))
    if not case["train"]:
        return nv.rotary(s["x"], s["positions"], axes, interleaved=case["pairs"])
    x = s["x"].detach().requires_grad_()
    y = nv.RotaryEmbedding.apply(x, s["positions"], axes, 10000.0, case["pairs"])
    (dx,) = torch.autograd.grad(y, x, s["dy"])
    return y.detach(), dx


def _own_xattn(s):
    import nvfp4_w4a4_gemm_quantize_b200 as nv

    if not s["case"]["train"]:
        return nv.cross_attention(s["q"], s["k"], s["v"], kv_lens=s["lens"])
    q, k, v = (s[n].detach().requires_grad_() for n in ("q", "k", "v"))
    out = nv.CrossAttention.apply(q, k, v, s["lens"])
    return (out.detach(), *torch.autograd.grad(out, (q, k, v), s["do"]))


def run(state):
    if own:
        return {"gemv": _own_gemv, "rotary": _own_rotary, "xattn": _own_xattn}[state["case"]["op"]](state)
    return {"gemv": _gemv, "rotary": _rotary, "xattn": _xattn}[state["case"]["op"]](state)


# ----------------------------------------------------------------- what each pass cannot do without
def work(case):
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        scales = k // 32 if case["fmt"] == "mx" else k // 16
        return {"bytes": n * (k // 2 + scales) + m * k * 2 + m * n * (4 if case["f32"] else 2) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if case["op"] == "rotary":
        grid = _ints(case["grid"])
        tokens = grid[0] * grid[1] * grid[2]
        values = case["b"] * tokens * case["h"] * case["d"]
        passes = 2 if case["train"] else 1
        return {"bytes": passes * (2 * values * (4 if case["f32"] else 2) + 12 * tokens), "flops": passes * 3 * values}
    b, lq, lk, h, hkv, d = (case[n] for n in ("b", "lq", "lk", "h", "hkv", "d"))
    states = sum(_ints(case["lens"])) if case["lens"] else b * lk
    rows, given, made = b * lq * h * d * 2, states * hkv * d * 4, b * lk * hkv * d * 4
    product = 2 * lq * states * h * d
    if not case["train"]:
        return {"bytes": 2 * rows + given, "flops": 2 * product}
    return {"bytes": 4 * rows + given + made, "flops": 7 * product}


# ----------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemv":
        n, k = case["n"], case["k"]
        kb = k // 32 if case["fmt"] == "mx" else k // 16
        code = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).reshape(n, k)
        e, m = (code >> 1 & 3).double(), (code & 1).double()
        w = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1)) * torch.where(code > 7, -1.0, 1.0)
        r, c = torch.arange(n, device="cuda")[:, None], torch.arange(kb, device="cuda")[None]
        byte = s["sf"][(r // 128 * (kb // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4].double()
        if case["fmt"] == "mx":
            sf = torch.exp2(byte - 127)
        else:
            be, bm = torch.floor(byte / 8), byte % 8
            sf = torch.where(be == 0, bm / 512, (1 + bm / 8) * torch.exp2(be - 7))
        y = (s["x"].double() @ (w * sf.repeat_interleave(k // kb, 1)).T) * s["scale"].double()
        return y + s["bias"].double() if s["bias"] is not None else y
    if case["op"] == "rotary":
        half = torch.cat([torch.exp(torch.arange(w // 2, device="cuda").double() * (-2 / w * math.log(10000.0)))
                          for w in _ints(case["axes"]) if w])
        axis = torch.cat([torch.full((w // 2,), a, device="cuda") for a, w in enumerate(_ints(case["axes"]))])
        phase = torch.polar(torch.ones_like(half), s["positions"].double()[:, axis] * half)[:, None]
        n = half.numel()
        first = torch.arange(n, device="cuda") * 2 if case["pairs"] else torch.arange(n, device="cuda")
        second = first + 1 if case["pairs"] else first + n

        def turned(x, phase):
            y = x.double()
            z = torch.complex(y[..., first], y[..., second]) * phase
            y[..., first], y[..., second] = z.real, z.imag
            return y

        y = turned(s["x"].clone(), phase)
        return (y, turned(s["dy"].clone(), phase.conj())) if case["train"] else y
    b, lq, lk, h, hkv, d = (case[n] for n in ("b", "lq", "lk", "h", "hkv", "d"))
    lens = _ints(case["lens"]) or [lk] * b
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    out, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
    for i in range(b):
        for j in range(h):
            at, n = j // (h // hkv), lens[i]
            if n == 0:
                continue
            p = torch.softmax(q[i, :, j] @ k[i, :n, at].T / math.sqrt(d), 1)
            out[i, :, j] = p @ v[i, :n, at]
            if case["train"]:
                do = s["do"][i, :, j].double()
                dp = do @ v[i, :n, at].T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                dq[i, :, j] = ds @ k[i, :n, at]
                dk[i, :n, at] += ds.T @ q[i, :, j]
                dv[i, :n, at] += p.T @ do
    return (out, dq, dk, dv) if case["train"] else out
