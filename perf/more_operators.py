"""Cases of the operators between a training step's products, with their plain forms.

  norm   RMS norm of a residual stream with the addition of a branch, forward and gradient; the result also in
         8-bit floating point (E4M3) with a power-of-two scale for each 128 values, along rows and columns
  gate   the gated activation silu(gate) * up, forward and gradient, with the same 8-bit outputs
  clip   the norm over many gradients together, and the gradients scaled down to a largest norm

`own` false: elementary torch operations in 32 bits (sums of squares in 64), rounded once at the end.
`own` true: the package's entry points. 8-bit results are a pair (codes as the E4M3 values they stand for,
scales as the powers of two they stand for)."""
import math

import torch

own = False

FP8_MAX = 448.0             # largest E4M3 value
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases --
# norm: stream = type of the residual stream, branch = type of what is added to it (and of dy); axis = the 8-bit
# outputs; y = whether the bf16 result is written too. gate: joined = gate and up are the halves of one matrix.
# clip: sizes come from `model`, `width` and `layers` (see _shapes).
def listed():
    return [
        # one token's norm in front of an 8-bit layer: the smallest call, where the launch counts
        dict(name="norm 1x4096", op="norm", grad=False, rows=1, cols=4096, stream="bf16", branch="bf16", axis="rows", y=False),
        # a layer's norm over a step's 8192 tokens: codes for the forward product and, transposed, for the weight gradient
        dict(name="norm 8192x4096", op="norm", grad=False, rows=8192, cols=4096, stream="bf16", branch="bf16", axis="both", y=False),
        # a ragged batch with an odd feature size, the stream kept in FP32, y for a layer in bf16 as well
        dict(name="norm 1111x2001 f32", op="norm", grad=False, rows=1111, cols=2001, stream="f32", branch="bf16", axis="both", y=True),
        # the norm's gradient over a step's tokens, with the gradient that arrives along the stream
        dict(name="norm grad 8192x4096", op="norm", grad=True, rows=8192, cols=4096, stream="bf16", branch="bf16"),
        # its ragged FP32 counterpart
        dict(name="norm grad 1111x2001 f32", op="norm", grad=True, rows=1111, cols=2001, stream="f32", branch="bf16"),
        # a small model's gated activation, rows only, as an evaluation makes it
        dict(name="gate 256x512", op="gate", grad=False, rows=256, cols=512, dtype="bf16", joined=False, axis="rows", a=False),
        # a layer's activation over 8192 tokens, from a fused gate-and-up product, for the down product and its weight gradient
        dict(name="gate 8192x14336", op="gate", grad=False, rows=8192, cols=14336, dtype="bf16", joined=True, axis="both", a=False),
        # the gradient of that, as the operands of one fused product's dgrad and wgrad
        dict(name="gate grad 8192x14336", op="gate", grad=True, rows=8192, cols=14336, dtype="bf16", joined=True, axis="both", a=False),
        # a ragged batch of separate products in FP32, gradients in bf16 and in 8 bits
        dict(name="gate grad 1111x2001 f32", op="gate", grad=True, rows=1111, cols=2001, dtype="f32", joined=False, axis="both", a=True),
        # the gradients of a small model: 19 tensors of up to 512 x 1024 values
        dict(name="clip small", op="clip", model="layers", layers=2, width=512, hidden=1024, dtype="f32", out="f32"),
        # one layer of an 8-billion-parameter model: FP32 sums in, bf16 gradients out
        dict(name="clip layer", op="clip", model="layers", layers=1, width=4096, hidden=14336, dtype="f32", out="bf16"),
        # many tensors of odd sizes, back to back in one bf16 bucket: norms' gains, biases, adapters
        dict(name="clip 300 tensors", op="clip", model="bucket", tensors=300, width=40000, dtype="bf16", out="bf16"),
    ]


def _size(rng, lo, hi):
    """Spread over the logarithm; half of the sizes are multiples of 64 where they are large enough."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def _draw(rng):
    op = rng.choice(["norm", "gate", "clip"])
    if op == "clip":
        t, o = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
        if rng.random() < 0.5:
            return dict(op=op, model="bucket", tensors=_size(rng, 1, 1000), width=_size(rng, 30, 100000), dtype=t, out=o)
        return dict(op=op, model="layers", layers=rng.randint(1, 4), width=_size(rng, 64, 4096), hidden=_size(rng, 64, 14336), dtype=t, out=o)
    rows, cols, grad, axis = _size(rng, 1, 16384), _size(rng, 32, 16384), rng.random() < 0.4, rng.choice(["none", "rows", "both"])
    if op == "norm":
        stream, branch = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        c = dict(op=op, grad=grad, rows=rows, cols=cols, stream=stream, branch=branch)
        return c if grad else dict(c, axis=axis, y=axis == "none" or rng.random() < 0.3)
    return dict(op=op, grad=grad, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]), axis=axis,
                joined=cols % 128 == 0 and rng.random() < 0.7, a=axis == "none" or rng.random() < 0.3)


def draw(rng):
    while True:
        c = _draw(rng)
        if work(c)["bytes"] <= 1.2e9:       # the largest listed ones' cost
            return c


def _shapes(c):
    """The numbers of values of a clip case's tensors."""
    if c["model"] == "layers":
        # per layer: fused query, key and value; output; fused gate and up; down; two gains. Then the last norm's gain
        w, h = c["width"], c["hidden"]
        return [n for _ in range(c["layers"]) for n in (w * w, w * (w // 4), w * (w // 4), w * w, 2 * h * w, h * w, w, w, w)] + [w]
    # from one value to `width` of them, the same list for everybody
    n, w = c["tensors"], c["width"]
    return [max(1, int(w ** ((7 * i % n + 1) / n))) + 3 * (i % 5) for i in range(n)]


# ------------------------------------------------------------------------------- the inputs --
def _heavy(g, rows, cols, scale):
    """Student-t with three degrees of freedom: what gradients look like."""
    n = torch.randn(rows, cols, generator=g, device="cuda")
    chi = torch.zeros_like(n)
    for _ in range(3):
        chi += torch.randn(rows, cols, generator=g, device="cuda").square_()
    return n.div_(chi.div_(3.0).sqrt_()).mul_(scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        R, C = case["rows"], case["cols"]
        S, B = TYPES[case["stream"]], TYPES[case["branch"]]
        # a stream grows over the layers, and a thousandth of its channels is 50 times larger
        stream = (3.0 * rnd(R, C) * torch.where(torch.rand(C, generator=g, device="cuda") < 1e-3, 50.0, 1.0)).to(S)
        w = (1.0 + 0.2 * rnd(C)).to(torch.bfloat16)
        if not case["grad"]:
            return dict(case=case, x=rnd(R, C).to(B), r=stream, w=w)
        rstd = (stream.double().square().mean(dim=1) + EPS).rsqrt().float()      # the forward call's
        return dict(case=case, dy=_heavy(g, R, C, 1e-3).to(B), dres=_heavy(g, R, C, 1e-3).to(S), h=stream, rstd=rstd, w=w)
    if case["op"] == "gate":
        R, C, t = case["rows"], case["cols"], TYPES[case["dtype"]]
        if case["joined"]:
            gu = (1.5 * rnd(R, 2 * C)).to(t)
            s = dict(case=case, gate=gu[:, :C], up=gu[:, C:])
        else:
            s = dict(case=case, gate=(1.5 * rnd(R, C)).to(t), up=(1.5 * rnd(R, C)).to(t))
        return dict(s, da=_heavy(g, R, C, 1e-3).to(t)) if case["grad"] else s
    sizes = _shapes(case)
    flat = _heavy(g, 1, sum(sizes), 1e-3)[0].to(TYPES[case["dtype"]])
    out = torch.empty(flat.shape, dtype=TYPES[case["out"]], device="cuda")
    # about half of the norm these gradients have (1.7e-3 sqrt(n) in the mean): they are clipped, as in a
    # run's first steps
    return dict(case=case, grads=list(flat.split(sizes)), out=out, outs=list(out.split(sizes)), max_norm=8e-4 * math.sqrt(sum(sizes)))


# ------------------------------------------------------------------------------- the passes --
def _codes(v):
    """E4M3 codes [R, round_up(L, 128)] (as values; zeros behind L) and scales [R, ceil(L / 128)] of v[R, L] in 1 x 128
    blocks along its rows: divided by the smallest power of two that brings the block's maximum to at most 448."""
    b = torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).view(v.shape[0], -1, 128)
    amax = b.abs().amax(dim=2, keepdim=True)
    frac, exp = torch.frexp(amax)                       # amax = frac 2^exp, frac in [0.5, 1)
    e = torch.where(amax > 0, exp - 9 + (frac > 0.875).int(), -127).clamp(min=-127)   # 448 = 0.875 2^9
    q = (b * torch.exp2(-e.float())).to(torch.float8_e4m3fn).view(v.shape[0], -1)
    return q, (e[:, :, 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _eight(v, axis):
    """The 8-bit outputs of a matrix: along its rows, and along its columns."""
    o = {} if axis == "none" else dict(rows=_codes(v))
    return dict(o, columns=_codes(v.t().contiguous())) if axis == "both" else o


def _plain_norm(s):
    c, w = s["case"], s["w"].float()
    if not c["grad"]:
        h = (s["x"].float() + s["r"].float()).to(s["r"].dtype)
        rstd = (h.double().square().mean(dim=1) + EPS).rsqrt().float()
        y = h.float() * rstd[:, None] * w
        return dict(_eight(y, c["axis"]), h=h, rstd=rstd, **(dict(y=y.to(torch.bfloat16)) if c["y"] else {}))
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    n = h * rstd
    u = dy * w
    dh = rstd * (u - n * (u * n).mean(dim=1, keepdim=True)) + s["dres"].float()
    return dict(dh=dh.to(s["h"].dtype), dw=(dy * n).sum(dim=0))


def _halves(dg, du, c):
    """The 8-bit outputs of the two gradients: of one matrix where they are halves of it, or one by one."""
    if c["joined"]:
        return _eight(torch.cat([dg, du], dim=1), c["axis"])
    return dict(gate=_eight(dg, c["axis"]), up=_eight(du, c["axis"]))


def _plain_gate(s):
    c, g, u = s["case"], s["gate"].float(), s["up"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    if not c["grad"]:
        a = g * sig * u
        return dict(_eight(a, c["axis"]), **(dict(a=a.to(torch.bfloat16)) if c["a"] else {}))
    da = s["da"].float()
    dg, du = da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig
    return dict(_halves(dg, du, c), **(dict(dgate=dg.to(torch.bfloat16), dup=du.to(torch.bfloat16)) if c["a"] else {}))


def _plain_clip(s):
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    s["out"].copy_(torch.cat([g.float() * scale for g in s["grads"]]))
    return dict(norm=norm.float(), out=s["out"])


def _pair(q, s, length):
    """What the bytes of codes and scales stand for."""
    return q.view(torch.float8_e4m3fn), s[:, :(length + 127) // 128].view(torch.float8_e8m0fnu)


def _own(s):
    import mxfp4_block_scaled_h16_amd as mx
    c = s["case"]
    if c["op"] == "clip":
        return dict(norm=mx.grad_clip(s["grads"], s["max_norm"], out=s["outs"]), out=s["out"])
    R, C = c["rows"], c["cols"]
    axis = {"none": None, "rows": 1, "both": "both"}[c.get("axis", "none")]
    eight = lambda o, C: {**(dict(rows=_pair(o.q1, o.s1, C)) if axis else {}),   # noqa: E731
                          **(dict(columns=_pair(o.q0, o.s0, R)) if axis == "both" else {})}
    if c["op"] == "norm":
        if c["grad"]:
            o = mx.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["w"], dres=s["dres"])
            return dict(dh=o.dh, dw=o.dweight)
        o = mx.rmsnorm_forward(s["x"], s["w"], residual=s["r"], eps=EPS, axis=axis, y_dtype=torch.bfloat16 if c["y"] else None)
        return dict(eight(o, C), h=o.h, rstd=o.rstd, **(dict(y=o.y) if c["y"] else {}))
    dtype = torch.bfloat16 if c["a"] else None
    if not c["grad"]:
        o = mx.swiglu_forward(s["gate"], s["up"], axis=axis, out_dtype=dtype)
        return dict(eight(o, C), **(dict(a=o.a) if c["a"] else {}))
    o = mx.swiglu_backward(s["da"], s["gate"], s["up"], axis=axis, out_dtype=dtype, joined=c["joined"])
    wide = dict(dgate=o.dgate, dup=o.dup) if c["a"] else {}
    return dict(eight(o, 2 * C), **wide) if c["joined"] else dict(gate=eight(o.gate, C), up=eight(o.up, C), **wide)


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "gate": _plain_gate, "clip": _plain_clip}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- its floor --
def work(case):
    bytes_of = {"bf16": 2, "f32": 4}
    if case["op"] == "clip":
        n = sum(_shapes(case))
        return {"bytes": n * (bytes_of[case["dtype"]] + bytes_of[case["out"]]), "flops": 3 * n}
    R, C = case["rows"], case["cols"]
    eight = {"none": 0, "rows": 1, "both": 2}[case.get("axis", "none")]
    if case["op"] == "norm":
        S, B = bytes_of[case["stream"]], bytes_of[case["branch"]]
        if case["grad"]:
            return {"bytes": R * C * (B + 3 * S) + 4 * R + 6 * C, "flops": 10 * R * C}
        return {"bytes": R * C * (B + 2 * S + eight + (2 if case["y"] else 0)) + 4 * R + 2 * C, "flops": 5 * R * C}
    t = bytes_of[case["dtype"]]
    wide = 2 if case["a"] else 0
    if case["grad"]:
        return {"bytes": R * C * (3 * t + 2 * (eight + wide)), "flops": 12 * R * C}
    return {"bytes": R * C * (2 * t + eight + wide), "flops": 6 * R * C}


# ------------------------------------------------------------------------------- in 64 bits --
def _scaled_64(v):
    """v[R, L] (64 bits) over its blocks' scales, not rounded, and the scales."""
    R, L = v.shape
    nb = (L + 127) // 128
    wide = torch.zeros(R, nb * 128, dtype=torch.float64, device=v.device)
    wide[:, :L] = v
    top = wide.abs().reshape(R, nb, 128).max(dim=2).values
    scale = torch.exp2(torch.ceil(torch.log2(top / FP8_MAX)).clamp(min=-127.0))      # top = 0: 2^-127
    # the logarithm may be a rounding off at a power of two: the smallest scale that fits is meant
    scale = torch.where(top > FP8_MAX * scale, 2.0 * scale, scale)
    scale = torch.where((top <= FP8_MAX * scale / 2) & (scale > 2.0 ** -127), scale / 2, scale)
    return wide.div_(scale.repeat_interleave(128, dim=1)), scale


def _eight_64(v, axis):
    both = (("rows", False), ("columns", True))[:{"none": 0, "rows": 1, "both": 2}[axis]]
    return {name: _scaled_64(v.t() if turn else v) for name, turn in both}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        g = torch.cat(s["grads"]).double()
        norm = torch.linalg.vector_norm(g)
        return dict(norm=norm, out=g * min(1.0, s["max_norm"] / (float(norm) + 1e-6)))
    if case["op"] == "norm":
        w = s["w"].double()
        if not case["grad"]:
            total = s["x"].double() + s["r"].double()
            h = total.to(s["r"].dtype).double()          # the norm is that of the stream as it is kept
            rstd = 1.0 / torch.sqrt(torch.linalg.vecdot(h, h) / case["cols"] + EPS)
            y = torch.einsum("rc,r,c->rc", h, rstd, w)
            return dict(_eight_64(y, case["axis"]), h=total, rstd=rstd, **(dict(y=y) if case["y"] else {}))
        dy, h, rstd = s["dy"].double(), s["h"].double(), s["rstd"].double()
        inner = torch.linalg.vecdot(dy * w, h)
        dh = s["dres"].double() + (dy * w) * rstd[:, None] - h * (rstd.pow(3) * inner / case["cols"])[:, None]
        return dict(dh=dh, dw=torch.mv((dy * h).t(), rstd))
    g, u = s["gate"].double(), s["up"].double()
    sig = torch.sigmoid(g)
    if not case["grad"]:
        a = torch.mul(g, sig).mul_(u)
        return dict(_eight_64(a, case["axis"]), **(dict(a=a) if case["a"] else {}))
    da = s["da"].double()
    dg, du = da * u * (sig + g * sig * torch.sigmoid(-g)), da * (g * sig)
    wide = dict(dgate=dg, dup=du) if case["a"] else {}
    if not case["joined"]:
        return dict(gate=_eight_64(dg, case["axis"]), up=_eight_64(du, case["axis"]), **wide)
    return dict(_eight_64(torch.cat([dg, du], dim=1), case["axis"]), **wide)
