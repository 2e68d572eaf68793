"""The operators of a linear layer in 8-bit floating point, and the calls that
are timed on them: the product of block-scaled operands, the RMS norm (with
the residual's addition) whose output is quantised, its backward pass, and the
quantiser.

Every 8-bit matrix goes with one FP32 scale per block: 128 consecutive
elements along the product's inner dimension times 1 or 128 along the other.
With F the largest value of the 8-bit type,

    a = max |x| over the block,   s = max(a / F, 2^-126),   q = fp8(x / s)
    C = op(qA sA) op(qB sB)
    h = x + r,   t = 1 / sqrt(mean h^2 + eps),   y = h t w
    g = dy w,    dx = t (g - h t^2 mean(g h)) + dh,   dw = sum over rows of dy h t
"""
import math

import torch

own = False

B = 128
EPS = 1e-6
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOAT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # serving: one token through a square projection; the weights' bytes and the launch count
        {"name": "product 1 token", "op": "product", "m": 1, "n": 4096, "k": 4096, "ta": 0, "tb": 1,
         "ga": 1, "gb": 128, "fa": "e4m3", "fb": "e4m3", "out": "bf16"},
        # serving: a batch of decoded tokens through a widening projection
        {"name": "product 24 tokens", "op": "product", "m": 24, "n": 8192, "k": 4096, "ta": 0, "tb": 1,
         "ga": 1, "gb": 128, "fa": "e4m3", "fb": "e4m3", "out": "bf16"},
        # sizes that no tile divides (the library's own ragged product)
        {"name": "product ragged", "op": "product", "m": 1000, "n": 1013, "k": 997, "ta": 0, "tb": 1,
         "ga": 1, "gb": 128, "fa": "e4m3", "fb": "e4m3", "out": "f32"},
        # a short prompt: fewer tiles than the GPU has SMs
        {"name": "product 512 tokens", "op": "product", "m": 512, "n": 4096, "k": 8192, "ta": 0, "tb": 1,
         "ga": 1, "gb": 128, "fa": "e4m3", "fb": "e4m3", "out": "bf16"},
        # training: the gradient of a layer's input, the weights read along their rows
        {"name": "product input gradient", "op": "product", "m": 4096, "n": 4096, "k": 8192, "ta": 0, "tb": 0,
         "ga": 1, "gb": 128, "fa": "e5m2", "fb": "e4m3", "out": "bf16"},
        # training: the gradient of a layer's weights, both operands scaled along the tokens
        {"name": "product weight gradient", "op": "product", "m": 4096, "n": 8192, "k": 4096, "ta": 1, "tb": 0,
         "ga": 1, "gb": 1, "fa": "e4m3", "fb": "e4m3", "out": "f32"},
        # the largest: a long prompt through a wide projection
        {"name": "product 8192 tokens", "op": "product", "m": 8192, "n": 8192, "k": 8192, "ta": 0, "tb": 1,
         "ga": 1, "gb": 128, "fa": "e4m3", "fb": "e4m3", "out": "bf16"},
        # serving: the norm before a projection, one token
        {"name": "norm 1 token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "f": "e4m3", "train": False},
        # training: the norm of a long batch, with what its backward pass needs
        {"name": "norm 8192 tokens", "op": "norm", "rows": 8192, "cols": 8192, "type": "bf16", "f": "e4m3",
         "train": True},
        # training: its backward pass, an odd number of tokens
        {"name": "norm gradient", "op": "norm gradient", "rows": 4095, "cols": 8192, "type": "bf16"},
        # weights into 128 x 128 blocks, after an optimizer step
        {"name": "quantise weights", "op": "quantise", "rows": 4096, "cols": 8192, "type": "f32", "f": "e4m3",
         "block": "tile"},
        # training: an output gradient for both of its products, an odd number of tokens
        {"name": "quantise gradient", "op": "quantise", "rows": 4095, "cols": 4104, "type": "bf16", "f": "e5m2",
         "block": "both"},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm: as it falls, or a multiple of 128, 16 or 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice([1, 1, 8, 16, 128])
    return max(lo, min(hi, cdiv(v, step) * step if v > step else v))


def draw(rng):
    op = rng.choice(["product", "product", "product", "norm", "norm gradient", "quantise"])
    if op == "product":
        # forward, input gradient, weight gradient
        ta, tb, ga, gb = rng.choice([(0, 1, 1, 128), (0, 1, 1, 128), (0, 0, 1, 128), (1, 0, 1, 1)])
        return {"op": op, "m": _size(rng, 1, 8192), "n": _size(rng, 64, 8192), "k": _size(rng, 64, 8192), "ta": ta,
                "tb": tb, "ga": ga, "gb": gb, "fa": rng.choice(["e4m3", "e4m3", "e5m2"]), "fb": "e4m3",
                "out": rng.choice(["bf16", "bf16", "f16", "f32"])}
    c = {"op": op, "rows": _size(rng, 1, 8192), "cols": _size(rng, 16, 8192),
         "type": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "norm":
        c |= {"f": rng.choice(["e4m3", "e5m2"]), "train": rng.choice([False, True])}
    elif op == "quantise":
        c |= {"f": rng.choice(["e4m3", "e5m2"]), "block": rng.choice(["row", "column", "tile", "both"])}
    return c


# ---------------------------------------------------------------- inputs
def _activations(rows, cols, g):
    """Unit activations with a few channels far larger than the rest; one token in 64 is padding (all zeros)."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 20.0, 1.0)
    if rows > 1:
        x *= (torch.rand(rows, 1, generator=g, device="cuda") >= 1 / 64).float()
    return x


def _operand(rows, cols, br, bc, f, g, weight):
    """An 8-bit matrix whose rows start on 16-byte boundaries, and its scales."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * 0.02 if weight else _activations(rows, cols, g)
    q, s = _quantise(x, br, bc, f)
    del x
    pitch = cdiv(cols, 16) * 16
    buf = torch.zeros(rows, pitch, dtype=torch.uint8, device="cuda")
    buf[:, :cols] = q.view(torch.uint8)
    return buf.view(F8[f])[:, :cols], s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        a = _operand(*((k, m, B, c["ga"]) if c["ta"] else (m, k, c["ga"], B)), c["fa"], g, False)
        b = _operand(*((n, k, c["gb"], B) if c["tb"] else (k, n, B, c["gb"])), c["fb"], g, c["gb"] == B)
        return {"c": c, "a": a, "b": b}
    t = FLOAT[c["type"]]
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "quantise":
        x = torch.randn(rows, cols, generator=g, device="cuda") * 0.02 if c["block"] == "tile" else \
            _activations(rows, cols, g)
        return {"c": c, "x": x.to(t)}
    w = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(t)
    if c["op"] == "norm":
        return {"c": c, "x": torch.randn(rows, cols, generator=g, device="cuda").to(t),
                "r": _activations(rows, cols, g).to(t), "w": w}
    h = _activations(rows, cols, g).to(t)
    return {"c": c, "h": h, "w": w, "dy": (torch.randn(rows, cols, generator=g, device="cuda") * 0.01).to(t),
            "dh": (torch.randn(rows, cols, generator=g, device="cuda") * 0.01).to(t),
            "t": torch.rsqrt(h.float().square().mean(1) + EPS)}


# ---------------------------------------------------------------- the plain forms
def _spread(s, br, bc, rows, cols):
    """One scale per element."""
    if br > 1:
        s = s.repeat_interleave(br, 0)[:rows]
    if bc > 1:
        s = s.repeat_interleave(bc, 1)[:, :cols]
    return s


def _quantise(x, br, bc, f):
    rows, cols = x.shape
    x = x.float()
    p = torch.nn.functional.pad(x, (0, -cols % bc, 0, -rows % br))
    a = p.abs().view(cdiv(rows, br), br, cdiv(cols, bc), bc).amax((1, 3))
    s = (a / FMAX[f]).clamp_min(2.0 ** -126)
    return (x / _spread(s, br, bc, rows, cols)).to(F8[f]), s


def _plain_product(c, a, b):
    def full(q, s, outer, trans):
        br, bc = (B, outer) if trans else (outer, B)
        return q.float() * _spread(s, br, bc, *q.shape)
    x = full(*a, c["ga"], c["ta"])
    y = full(*b, c["gb"], not c["tb"])
    return ((x.t() if c["ta"] else x) @ (y.t() if c["tb"] else y)).to(FLOAT[c["out"]])


def _plain_norm(c, x, r, w):
    h = x.float() + r.float()
    t = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * t[:, None] * w.float()
    q, s = _quantise(y, 1, B, c["f"])
    out = {"q": q, "s": s, "h": h.to(x.dtype)}
    if c["train"]:
        out |= {"y": y.to(x.dtype), "t": t}
    return out


def _plain_norm_gradient(dy, h, w, t, dh):
    h32, dy32, t = h.float(), dy.float(), t[:, None]
    g = dy32 * w.float()
    dx = t * (g - h32 * t.square() * (g * h32).mean(1, keepdim=True)) + dh.float()
    return {"dx": dx.to(h.dtype), "dw": (dy32 * h32 * t).sum(0).to(w.dtype)}


def _blocks(c):
    return {"row": [(1, B)], "column": [(B, 1)], "tile": [(B, B)], "both": [(1, B), (B, 1)]}[c["block"]]


def run(state):
    s, c = state, state["c"]
    if own:
        import dense_fp32_matrix_10_gb300 as sg
        if c["op"] == "product":
            return sg.gemm_fp8(*s["a"], *s["b"], transA=bool(c["ta"]), transB=bool(c["tb"]),
                               out_dtype=FLOAT[c["out"]])
        if c["op"] == "norm":
            o = sg.rms_norm_fp8(s["x"], s["w"], residual=s["r"], eps=EPS, dtype=F8[c["f"]], training=c["train"])
            out = {"q": o.q, "s": o.scale, "h": o.h}
            return out | {"y": o.y, "t": o.rstd} if c["train"] else out
        if c["op"] == "norm gradient":
            dx, dw = sg.rms_norm_backward(s["dy"], s["h"], s["w"], s["t"], dh=s["dh"])
            return {"dx": dx, "dw": dw}
        if c["block"] == "both":
            return sg.quantize_fp8_both(s["x"], dtype=F8[c["f"]])
        return sg.quantize_fp8(s["x"], block=_blocks(c)[0], dtype=F8[c["f"]])
    if c["op"] == "product":
        return _plain_product(c, s["a"], s["b"])
    if c["op"] == "norm":
        return _plain_norm(c, s["x"], s["r"], s["w"])
    if c["op"] == "norm gradient":
        return _plain_norm_gradient(s["dy"], s["h"], s["w"], s["t"], s["dh"])
    return tuple(v for br, bc in _blocks(c) for v in _quantise(s["x"], br, bc, c["f"]))


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        scales = (cdiv(m, c["ga"]) + cdiv(n, c["gb"])) * cdiv(k, B)
        return {"bytes": m * k + n * k + 4 * scales + m * n * SIZE[c["out"]], "flops": 2 * m * n * k}
    rows, cols, size = c["rows"], c["cols"], SIZE[c["type"]]
    n = rows * cols
    if c["op"] == "norm":
        stored = 3 + (1 if c["train"] else 0)
        return {"bytes": n * (stored * size + 1) + cols * size + 4 * rows * (cdiv(cols, B) + int(c["train"])),
                "flops": 8 * n}
    if c["op"] == "norm gradient":
        return {"bytes": 4 * n * size + 2 * cols * size + 4 * rows, "flops": 11 * n}
    scales = sum(cdiv(rows, br) * cdiv(cols, bc) for br, bc in _blocks(c))
    return {"bytes": n * (size + len(_blocks(c))) + 4 * scales, "flops": 3 * n * len(_blocks(c))}


# ---------------------------------------------------------------- the definitions in 64 bits
def _to_f8_64(v, f):
    """v rounded to the nearest value of the 8-bit type, ties to even, in 64 bits (no overflow)."""
    mantissa, least = (3, -6) if f == "e4m3" else (2, -14)
    e = (torch.frexp(v)[1] - 1).clamp_min(least) - mantissa
    step = torch.ldexp(torch.ones_like(v), e)
    return torch.round(v / step) * step


def _quantise_64(x, br, bc, f):
    rows, cols = x.shape
    R, C = cdiv(rows, br), cdiv(cols, bc)
    p = x.new_zeros(R * br, C * bc)
    p[:rows, :cols] = x
    p = p.reshape(R, br, C, bc)
    s = torch.maximum(p.abs().amax(3).amax(1) / FMAX[f], torch.full((R, C), 2.0 ** -126, dtype=x.dtype,
                                                                     device=x.device))
    q = _to_f8_64(p / s[:, None, :, None], f).reshape(R * br, C * bc)[:rows, :cols]
    return q.contiguous(), s


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        (qa, sa), (qb, sb) = s["a"], s["b"]
        out = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        qa, sa = (qa, sa) if not c["ta"] else (qa.t(), sa.t())      # m x k
        qb, sb = (qb, sb) if c["tb"] else (qb.t(), sb.t())          # n x k
        ia = torch.arange(m, device="cuda") // c["ga"]
        ib = torch.arange(n, device="cuda") // c["gb"]
        for b in range(0, cdiv(k, B), 16):                          # 2048 of the inner dimension at a time
            ks = torch.arange(b * B, min(k, (b + 16) * B), device="cuda") // B
            part = slice(b * B, min(k, (b + 16) * B))
            out += (qa[:, part].double() * sa.double()[ia][:, ks]) @ \
                (qb[:, part].double() * sb.double()[ib][:, ks]).t()
        return out
    if c["op"] == "quantise":
        x = s["x"].double()
        return tuple(v for br, bc in _blocks(c) for v in _quantise_64(x, br, bc, c["f"]))
    if c["op"] == "norm":
        h = s["x"].double() + s["r"].double()
        t = 1 / torch.sqrt((h * h).sum(1) / c["cols"] + EPS)
        y = s["w"].double() * h * t.unsqueeze(1)
        q, sc = _quantise_64(y, 1, B, c["f"])
        return {"q": q, "s": sc, "h": h, "y": y, "t": t} if c["train"] else {"q": q, "s": sc, "h": h}
    h, dy, t = s["h"].double(), s["dy"].double(), s["t"].double().unsqueeze(1)
    n = h * t                                                       # the normalised row
    g = dy * s["w"].double()
    dx = t * (g - n * ((g * n).sum(1, keepdim=True) / c["cols"])) + s["dh"].double()
    return {"dx": dx, "dw": (dy * n).sum(0)}
