"""The operators of a gated block in 8-bit floating point around its products, and the calls that are timed on them:
the norms behind and in front of a block with its gate and the scaled residual, the block's gated unit, the gradients
of both, which read what the forward pass kept in 8 bits, and the change of kept rows into a weight gradient's operand.

An 8-bit matrix goes with one FP32 scale per block: 128 consecutive elements along the inner dimension of the product
that reads it. With F the largest value of the 8-bit type,

    e = max |v| over the block,   s = max(e / F, 2^-126),   q = fp8(v / s)

Norms, a row at a time, of a block's output a and the residual stream x (gate: one row for every so many of a's):

    ta = 1 / sqrt(mean a^2 + eps),   h = rho x + gate (a ta wa)
    t  = 1 / sqrt(mean h^2 + eps),   y = h t w
    H  = t (dy w - h t^2 mean(dy w h)) + dh,   dx = rho H,   v = H gate wa,   da = ta (v - a ta^2 mean(v a))
    dw = sum dy h t,   dwa = sum H gate a ta,   dgate = wa times the sum of H a ta over its rows

Gated unit:

    y = u g / (1 + exp(-g)),   du = dy g p,   dg = dy u p (1 + g (1 - p))   with p = 1 / (1 + exp(-g))
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
    """gates: 0 none, 1 a learned row for all, more: one for each sequence. keep: the type of what the forward pass
    keeps for the backward pass ("" nothing, "float" the tensors themselves)."""
    return [
        # serving: between two blocks, one token
        {"name": "norms 1 token", "op": "norms", "rows": 1, "cols": 4096, "type": "bf16", "f": "e4m3", "gates": 0,
         "rho": 1.0, "keep": ""},
        # training: a long batch, block output and residual stream kept in 8 bits
        {"name": "norms 8192 tokens", "op": "norms", "rows": 8192, "cols": 8192, "type": "bf16", "f": "e4m3",
         "gates": 1, "rho": 1.0, "keep": "e4m3"},
        # training: eight sequences with a gate each, an odd number of tokens, nothing quantised but the operand
        {"name": "norms 8 sequences", "op": "norms", "rows": 8 * 509, "cols": 4104, "type": "f16", "f": "e4m3",
         "gates": 8, "rho": 0.5, "keep": "float"},
        # training: the gradient through both norms from what was kept in 8 bits
        {"name": "norms gradient kept", "op": "norms gradient", "rows": 4095, "cols": 8192, "type": "bf16",
         "gates": 1, "rho": 1.0, "keep": "e4m3"},
        # training: a gate per sequence, the tensors themselves kept
        {"name": "norms gradient 8 sequences", "op": "norms gradient", "rows": 8 * 512, "cols": 4096, "type": "bf16",
         "gates": 8, "rho": 0.5, "keep": "float"},
        # sizes that no block divides, full precision
        {"name": "norms gradient ragged", "op": "norms gradient", "rows": 1000, "cols": 1013, "type": "f32",
         "gates": 0, "rho": 1.0, "keep": "float"},
        # serving: the unit between two products, one token
        {"name": "unit 1 token", "op": "unit", "rows": 1, "cols": 8192, "type": "bf16", "f": "e4m3", "keep": ""},
        # training: a long batch, both inputs kept in 8 bits
        {"name": "unit 8192 tokens", "op": "unit", "rows": 8192, "cols": 8192, "type": "bf16", "f": "e4m3",
         "keep": "e4m3"},
        # training: operands for the gradients of both projections, an odd number of tokens
        {"name": "unit gradient kept", "op": "unit gradient", "rows": 4095, "cols": 8192, "type": "bf16", "f": "e5m2",
         "keep": "e4m3"},
        # a short sequence, sizes that no block divides, the tensors themselves kept
        {"name": "unit gradient ragged", "op": "unit gradient", "rows": 1000, "cols": 1013, "type": "f32",
         "f": "e4m3", "keep": "float"},
        # training: a projection's kept input for its weight gradient, a short sequence
        {"name": "turn 512 tokens", "op": "turn", "rows": 512, "cols": 4096, "f": "e4m3", "to": "e4m3"},
        # the same, a long batch
        {"name": "turn 8192 tokens", "op": "turn", "rows": 8192, "cols": 8192, "f": "e4m3", "to": "e4m3"},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm: as it falls, or a multiple of 128, 16 or 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice([1, 1, 8, 16, 128])
    return max(lo, min(hi, cdiv(v, step) * step if v > step else v))


def draw(rng):
    op = rng.choice(["norms", "norms", "norms gradient", "norms gradient", "unit", "unit gradient", "turn"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = 4096 if kind == "f32" else 8192
    c = {"op": op, "rows": _size(rng, 1, most), "cols": _size(rng, 16, 8192)}
    if op == "turn":
        return c | {"f": rng.choice(["e4m3", "e5m2"]), "to": rng.choice(["e4m3", "e4m3", "e5m2"])}
    c["type"] = kind
    if op != "norms gradient":
        c["f"] = rng.choice(["e4m3", "e4m3", "e5m2"])
    c["keep"] = rng.choice(["float", "e4m3", "e4m3", "e5m2"] if "gradient" in op else ["", "float", "e4m3", "e5m2"])
    if op == "unit" and c["keep"] == "float":
        c["keep"] = ""
    if op in ("norms", "norms gradient"):
        c["rho"] = rng.choice([1.0, 1.0, 0.5])
        c["gates"] = rng.choice([0, 1, 1, 2])
        if c["gates"] == 2:   # sequences of one length; of one token, too
            c["gates"] = _size(rng, 1, c["rows"])
            c["rows"] = c["gates"] * max(1, c["rows"] // c["gates"])
    return c


# ---------------------------------------------------------------- inputs
def _activations(rows, cols, g, live):
    """Unit activations with a few channels far larger than the rest, and none in the rows of padding."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 20.0, 1.0)
    return x * live


def _aligned(q):
    """The same 8-bit matrix with rows that start on 16-byte boundaries, as the quantisers leave it."""
    buf = torch.zeros(q.shape[0], cdiv(q.shape[1], 16) * 16, dtype=torch.uint8, device="cuda")
    buf[:, :q.shape[1]] = q.view(torch.uint8)
    return buf.view(q.dtype)[:, :q.shape[1]]


def _kept(x, keep):
    """What the forward pass kept of x: itself, or its 8-bit rows and their scales."""
    if keep == "float":
        return x
    q, s = _quantise(x, 1, B, keep)
    return _aligned(q), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, rows, cols = case, case["rows"], case["cols"]
    live = (torch.rand(rows, 1, generator=g, device="cuda") >= (1 / 64 if rows > 1 else 0)).float()
    if c["op"] == "turn":
        q, s = _quantise(_activations(rows, cols, g, live), 1, B, c["f"])
        return {"c": c, "q": _aligned(q), "s": s}
    t = FLOAT[c["type"]]
    if c["op"] in ("unit", "unit gradient"):
        z = _activations(rows, 2 * cols, g, live).to(t)        # one product gives both halves
        gate, up = z[:, :cols], z[:, cols:]
        if c["op"] == "unit":
            return {"c": c, "gate": gate, "up": up}
        dy = (torch.randn(rows, cols, generator=g, device="cuda") * 0.01 * live).to(t)
        return {"c": c, "gate": _kept(gate, c["keep"]), "up": _kept(up, c["keep"]), "dy": dy}
    st = {"c": c, "wa": (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(t),
          "w": (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(t), "gate": None}
    if c["gates"] == 1:
        st["gate"] = 0.3 + 0.1 * torch.randn(cols, generator=g, device="cuda")      # learned, in full precision
    elif c["gates"] > 1:
        st["gate"] = (0.5 * torch.randn(c["gates"], cols, generator=g, device="cuda")).to(t)
    a = (torch.randn(rows, cols, generator=g, device="cuda") * 3 * live).to(t)
    x = _activations(rows, cols, g, live).to(t)
    if c["op"] == "norms":
        return st | {"a": a, "x": x}
    grad = lambda: (torch.randn(rows, cols, generator=g, device="cuda") * 0.01 * live).to(t)   # noqa: E731
    ta, th = (torch.rsqrt(v.float().square().mean(1) + EPS) for v in (a, x))
    return st | {"a": _kept(a, c["keep"]), "h": _kept(x, c["keep"]), "ta": ta, "t": th, "dy": grad(), "dh": grad()}


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
    e = p.abs().view(cdiv(rows, br), br, cdiv(cols, bc), bc).amax((1, 3))
    s = (e / FMAX[f]).clamp_min(2.0 ** -126)
    return (x / _spread(s, br, bc, rows, cols)).to(F8[f]), s


def _values(x):
    """A kept matrix as FP32 values."""
    return x.float() if torch.is_tensor(x) else x[0].float() * _spread(x[1], 1, B, *x[0].shape)


def _gate_rows(gate, rows):
    """The gate of every row (or 1)."""
    if gate is None:
        return 1.0
    gate = gate.float()
    return gate if gate.dim() == 1 else gate.repeat_interleave(rows // gate.shape[0], 0)


def _plain_norms(c, a, x, wa, w, gate):
    a32 = a.float()
    ta = torch.rsqrt(a32.square().mean(1) + EPS)
    h = c["rho"] * x.float() + _gate_rows(gate, c["rows"]) * (a32 * ta[:, None] * wa.float())
    t = torch.rsqrt(h.square().mean(1) + EPS)
    q, s = _quantise(h * t[:, None] * w.float(), 1, B, c["f"])
    out = {"q": q, "s": s, "h": h.to(a.dtype)}
    if c["keep"]:
        out |= {"ta": ta, "t": t}
    if c["keep"] in F8:
        out |= {"a8": _quantise(a32, 1, B, c["keep"]), "h8": _quantise(h, 1, B, c["keep"])}
    return out


def _plain_norms_gradient(c, s):
    dy, wa, w = s["dy"].float(), s["wa"].float(), s["w"].float()
    a, h, ta, t = _values(s["a"]), _values(s["h"]), s["ta"][:, None], s["t"][:, None]
    gate = _gate_rows(s["gate"], c["rows"])
    g = dy * w
    H = t * (g - h * t.square() * (g * h).mean(1, keepdim=True)) + s["dh"].float()
    v = H * (gate * wa)
    da = ta * (v - a * ta.square() * (v * a).mean(1, keepdim=True))
    n = H * (a * ta)
    out = {"da": da.to(s["dy"].dtype), "dx": (c["rho"] * H).to(s["dy"].dtype),
           "dwa": (n * gate).sum(0).to(s["wa"].dtype), "dw": (dy * h * t).sum(0).to(s["w"].dtype)}
    if c["gates"]:
        sums = n.view(c["gates"], -1, c["cols"]).sum(1) * wa
        out["dgate"] = sums.to(s["gate"].dtype).view(s["gate"].shape)
    return out


def _plain_unit(c, gate, up):
    g, u = gate.float(), up.float()
    q, s = _quantise(g / (1 + torch.exp(-g)) * u, 1, B, c["f"])
    out = {"q": q, "s": s}
    return out | {"gate8": _quantise(g, 1, B, c["keep"]), "up8": _quantise(u, 1, B, c["keep"])} if c["keep"] else out


def _plain_unit_gradient(c, dy, gate, up):
    dy, g, u = dy.float(), _values(gate), _values(up)
    p = 1 / (1 + torch.exp(-g))
    pad = (0, -c["cols"] % B)                       # each half of [dg | du] fills whole blocks
    dz = torch.cat([torch.nn.functional.pad(d, pad) for d in (dy * u * (p * (1 + g * (1 - p))), dy * (g * p))], 1)
    return *_quantise(dz, 1, B, c["f"]), *_quantise(dz, B, 1, c["f"]), *_quantise(g * p * u, B, 1, "e4m3")


def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if own:
        import dense_fp32_matrix_10_gb300 as sg
        if op == "norms":
            o = sg.sandwich_norm_fp8(s["a"], s["x"], s["wa"], s["w"], gate=s["gate"], residual_scale=c["rho"], eps=EPS,
                                     dtype=F8[c["f"]], training=bool(c["keep"]), checkpoint=F8.get(c["keep"]))
            out = {"q": o.q, "s": o.scale, "h": o.h}
            if c["keep"]:
                out |= {"ta": o.post_rstd, "t": o.rstd}
            return out | {"a8": o.a8, "h8": o.h8} if c["keep"] in F8 else out
        if op == "norms gradient":
            o = sg.sandwich_norm_backward(s["dy"], s["a"], s["h"], s["wa"], s["w"], s["ta"], s["t"], gate=s["gate"],
                                          residual_scale=c["rho"], dh=s["dh"])
            out = {"da": o.da, "dx": o.dx, "dwa": o.dpost_weight, "dw": o.dweight}
            return out | {"dgate": o.dgate} if c["gates"] else out
        if op == "unit":
            o = sg.swiglu_fp8(s["gate"], s["up"], dtype=F8[c["f"]], checkpoint=F8.get(c["keep"]))
            out = {"q": o.q, "s": o.scale}
            return out | {"gate8": o.gate8, "up8": o.up8} if c["keep"] else out
        if op == "unit gradient":
            return tuple(sg.swiglu_backward_fp8(s["dy"], s["gate"], s["up"], dtype=F8[c["f"]]))
        return sg.requantize_fp8(s["q"], s["s"], dtype=F8[c["to"]])
    if op == "norms":
        return _plain_norms(c, s["a"], s["x"], s["wa"], s["w"], s["gate"])
    if op == "norms gradient":
        return _plain_norms_gradient(c, s)
    if op == "unit":
        return _plain_unit(c, s["gate"], s["up"])
    if op == "unit gradient":
        return _plain_unit_gradient(c, s["dy"], s["gate"], s["up"])
    return _quantise(_values((s["q"], s["s"])), B, 1, c["to"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, rows, cols = case, case["rows"], case["cols"]
    n = rows * cols
    row, col = 4 * rows * cdiv(cols, B), 4 * cdiv(rows, B) * cols        # one set of scales
    if c["op"] == "turn":
        return {"bytes": 2 * n + row + col, "flops": 4 * n}
    size, keep8 = SIZE[c["type"]], c["keep"] in F8
    if c["op"] == "unit":
        return {"bytes": n * (2 * size + 1) + row + (2 * (n + row) if keep8 else 0), "flops": 10 * n}
    kept = n + row if keep8 else n * size                                # a matrix that the forward pass kept
    if c["op"] == "unit gradient":
        wide = cdiv(cols, B) * B                                         # dg and du, each both ways; y one way
        dz = 4 * rows * wide + 2 * row + 2 * 4 * cdiv(rows, B) * wide
        return {"bytes": n * size + 2 * kept + dz + n + col, "flops": 30 * n}
    gate = (cols * 4 if c["gates"] == 1 else c["gates"] * cols * size)
    if c["op"] == "norms":
        stats = 8 * rows if c["keep"] else 0
        return {"bytes": n * (3 * size + 1) + row + (2 * (n + row) if keep8 else 0) + 2 * cols * size + gate + stats,
                "flops": 14 * n}
    return {"bytes": n * 4 * size + 2 * kept + 4 * cols * size + 2 * gate + 8 * rows, "flops": 30 * n}


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


def _value_64(kept):
    """A kept matrix in 64 bits: every scale beside the 128 elements that it is for."""
    if torch.is_tensor(kept):
        return kept.double()
    q, s = kept
    at = torch.arange(q.shape[1], device="cuda") // B
    return q.double() * s.double()[:, at]


def exact(case, seed):
    s, c = prepare(case, seed), case
    rows, cols, op = c["rows"], c["cols"], c["op"]
    if op == "turn":
        return _quantise_64(_value_64((s["q"], s["s"])), B, 1, c["to"])
    if op in ("unit", "unit gradient"):
        g, u = _value_64(s["gate"]), _value_64(s["up"])
        silu = g * torch.sigmoid(g)
        if op == "unit":
            q, sc = _quantise_64(silu * u, 1, B, c["f"])
            out = {"q": q, "s": sc}
            return out | {"gate8": _quantise_64(g, 1, B, c["keep"]), "up8": _quantise_64(u, 1, B, c["keep"])} \
                if c["keep"] else out
        dy, wide = s["dy"].double(), cdiv(cols, B) * B
        slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)             # of g sigmoid(g)
        dz = torch.zeros(rows, 2 * wide, dtype=torch.float64, device="cuda")
        dz[:, :cols] = slope * u * dy
        dz[:, wide:wide + cols] = silu * dy
        return *_quantise_64(dz, 1, B, c["f"]), *_quantise_64(dz, B, 1, c["f"]), *_quantise_64(silu * u, B, 1, "e4m3")
    wa, w = s["wa"].double(), s["w"].double()
    seq = torch.arange(rows, device="cuda") // (rows // max(1, c["gates"]))
    gate = torch.ones(rows, cols, dtype=torch.float64, device="cuda") if s["gate"] is None else \
        s["gate"].double().view(c["gates"], cols)[seq]
    if op == "norms":
        a, x = s["a"].double(), s["x"].double()
        ta = 1 / torch.sqrt((a * a).sum(1) / cols + EPS)
        h = gate * (wa * (a * ta.unsqueeze(1))) + x * c["rho"]
        t = 1 / torch.sqrt((h * h).sum(1) / cols + EPS)
        q, sc = _quantise_64(w * (h * t.unsqueeze(1)), 1, B, c["f"])
        out = {"q": q, "s": sc, "h": h}
        if c["keep"]:
            out |= {"ta": ta, "t": t}
        if c["keep"] in F8:
            out |= {"a8": _quantise_64(a, 1, B, c["keep"]), "h8": _quantise_64(h, 1, B, c["keep"])}
        return out
    ta, t = s["ta"].double().unsqueeze(1), s["t"].double().unsqueeze(1)
    na, nh = _value_64(s["a"]) * ta, _value_64(s["h"]) * t              # the normalised rows
    dy = s["dy"].double()

    def through(d, n, scale):                                           # the gradient of a norm's input
        return scale * (d - n * ((d * n).sum(1, keepdim=True) / cols))

    H = s["dh"].double() + through(dy * w, nh, t)
    out = {"da": through(wa * gate * H, na, ta), "dx": H * c["rho"], "dwa": (gate * na * H).sum(0),
           "dw": (nh * dy).sum(0)}
    if c["gates"]:
        per = torch.zeros(c["gates"], cols, dtype=torch.float64, device="cuda").index_add_(0, seq, na * H) * wa
        out["dgate"] = per.view(s["gate"].shape)
    return out
