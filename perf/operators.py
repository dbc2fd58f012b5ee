"""Cases of three operators of a training step, with their plain forms.

  fp8_linear   one product of a linear layer in 8-bit floating point (E4M3), a power-of-two scale
               for each block of 128: Fprop Y = X W^T, Dgrad dX = dY W, Wgrad dW = dY^T X
  xent         softmax cross entropy of a linear head over a large vocabulary, and its gradients
  orthogonalize  the Newton-Schulz orthogonalisation of a weight gradient

`own` false: elementary torch operations in 32 bits, rounded once at the end. `own` true: the
package's entry points."""
import math

import torch

own = False

FP8_MAX = 448.0             # largest E4M3 value
NS_COEFFS = (3.4445, -4.7750, 2.0315)
IGNORE = -100


# ------------------------------------------------------------------------------- the cases --
def listed():
    return [
        # the smallest product, where the launches count: 256 tokens, 512 -> 256
        dict(name="fp8 fprop 256x512x256", op="fp8_linear", which="fprop", M=256, K=512, N=256),
        # the QKV projection of a layer at 8192 tokens
        dict(name="fp8 fprop 8192x4096x6144", op="fp8_linear", which="fprop", M=8192, K=4096, N=6144),
        # a ragged batch through odd feature sizes: nothing is a multiple of a block
        dict(name="fp8 dgrad 1111x1000x2001", op="fp8_linear", which="dgrad", M=1111, K=1000, N=2001),
        # the down projection's weight gradient over a step's 8192 tokens
        dict(name="fp8 wgrad 8192x14336x4096", op="fp8_linear", which="wgrad", M=8192, K=14336, N=4096),
        # a small model's head, one short sequence
        dict(name="xent 128x512x1000", op="xent", T=128, K=512, V=1000, train=True),
        # evaluation: the loss alone, over a medium vocabulary with an odd size
        dict(name="xent eval 2048x2048x50257", op="xent", T=2048, K=2048, V=50257, train=False),
        # a ragged batch of tokens of a medium model, with its gradients
        dict(name="xent 1537x1024x50257", op="xent", T=1537, K=1024, V=50257, train=True),
        # a large head: 4096 features, vocabulary of 128256, a step's 8192 tokens
        dict(name="xent 8192x4096x128256", op="xent", T=8192, K=4096, V=128256, train=True),
        # the smallest update: one small projection
        dict(name="orthogonalize 256x512", op="orthogonalize", B=1, m=256, n=512, dtype="f32"),
        # the key and value projections' updates together
        dict(name="orthogonalize 2x1024x4096", op="orthogonalize", B=2, m=1024, n=4096, dtype="f32"),
        # the output projection's update from a bf16 gradient
        dict(name="orthogonalize 4096x4096 bf16", op="orthogonalize", B=1, m=4096, n=4096, dtype="bf16"),
        # the gate projection's update: more rows than columns
        dict(name="orthogonalize 14336x4096", op="orthogonalize", B=1, m=14336, n=4096, dtype="f32"),
    ]


def _size(rng, lo, hi):
    """Spread over the logarithm; half of the sizes are multiples of 64 where they are large enough."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["fp8_linear", "xent", "orthogonalize"])
    while True:
        if op == "fp8_linear":
            c = dict(op=op, which=rng.choice(["fprop", "dgrad", "wgrad"]), M=_size(rng, 1, 16384), K=_size(rng, 32, 14336),
                     N=_size(rng, 32, 14336))
            if c["M"] * c["K"] * c["N"] <= 8192 * 14336 * 4096:
                return c
        elif op == "xent":
            c = dict(op=op, T=_size(rng, 1, 16384), K=_size(rng, 64, 8192), V=_size(rng, 100, 160000), train=rng.random() < 0.75)
            if c["T"] * c["K"] * c["V"] <= 8192 * 4096 * 128256 // 2 and c["T"] * c["V"] <= 1 << 30:
                return c
        else:
            c = dict(op=op, B=rng.choice([1, 1, 1, 2, 3, 4, 8]), m=_size(rng, 16, 14336), n=_size(rng, 16, 14336),
                     dtype=rng.choice(["f32", "bf16"]))
            s = min(c["m"], c["n"])
            if c["B"] * s * s * (s + max(c["m"], c["n"])) <= 4096 * 4096 * (4096 + 14336):
                return c


# ------------------------------------------------------------------------------- the inputs --
def _heavy(g, rows, cols, scale):
    """Student-t with three degrees of freedom: what gradients look like."""
    n = torch.randn(rows, cols, generator=g, device="cuda")
    chi = sum(torch.randn(rows, cols, generator=g, device="cuda").square_() for _ in range(3))
    return n.div_(chi.div_(3.0).sqrt_()).mul_(scale)


def _activations(g, rows, cols):
    """Normal, with a thousandth of the channels 50 times larger."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return x * torch.where(torch.rand(cols, generator=g, device="cuda") < 1e-3, 50.0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    bf16 = torch.bfloat16
    if case["op"] == "fp8_linear":
        M, K, N = case["M"], case["K"], case["N"]
        x = _activations(g, M, K).to(bf16)
        w = (0.02 * torch.randn(N, K, generator=g, device="cuda")).to(bf16)
        dy = _heavy(g, M, N, 1e-3).to(bf16)
        a, b = {"fprop": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[case["which"]]
        return dict(case=case, a=a, b=b)
    if case["op"] == "xent":
        T, K, V = case["T"], case["K"], case["V"]
        w = (0.02 * torch.randn(V, K, generator=g, device="cuda")).to(bf16)
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        # tokens from hopeless to certain: the target's logit is lifted by 0 to 12
        lift = 12.0 * torch.rand(T, 1, generator=g, device="cuda") / (0.02 * K)
        x = (torch.randn(T, K, generator=g, device="cuda") + lift * w[target].float() / 0.02).to(bf16)
        # a tenth of the positions is padding; the gradient is that of the mean over the others
        pad = torch.rand(T, generator=g, device="cuda") < 0.1
        target = torch.where(pad, IGNORE, target)
        dloss = torch.full((T,), 1.0, device="cuda") / (~pad).sum().clamp(min=1)
        return dict(case=case, x=x, w=w, target=target, dloss=dloss)
    B, m, n = case["B"], case["m"], case["n"]
    # a gradient: a few strong directions over a heavy-tailed rest
    r = max(1, min(m, n) // 32)
    grad = torch.stack([_heavy(g, m, n, 1e-3) + 2e-3 * torch.randn(m, r, generator=g, device="cuda")
                        @ torch.randn(r, n, generator=g, device="cuda") / math.sqrt(r) for _ in range(B)])
    grad = grad if B > 1 else grad[0]
    return dict(case=case, g=grad if case["dtype"] == "f32" else grad.to(bf16))


# ------------------------------------------------------------------------------- the passes --
def _blocks(v, tile):
    """The 8-bit values, as the numbers they stand for, of v in blocks of 128 along its last axis (tile: of
    128 x 128): divided by the smallest power of two that brings the block's maximum to at most 448."""
    R, L = v.shape
    v = torch.nn.functional.pad(v.float(), (0, -L % 128, 0, -R % 128 if tile else 0))
    b = v.view(v.shape[0] // 128, 128, -1, 128) if tile else v.view(v.shape[0], 1, -1, 128)
    amax = b.abs().amax(dim=(1, 3), keepdim=True)
    frac, exp = torch.frexp(amax)                       # amax = frac 2^exp, frac in [0.5, 1)
    e = torch.where(amax > 0, exp - 9 + (frac > 0.875).int(), -127).clamp(min=-127)   # 448 = 0.875 2^9
    q = (b * torch.exp2(-e.float())).to(torch.float8_e4m3fn).float()      # exact but for the cast
    return (q * torch.exp2(e.float())).view(v.shape[0], -1)[:R, :L]


def _plain_fp8(s):
    a, b, which = s["a"], s["b"], s["case"]["which"]
    if which == "fprop":
        y = _blocks(a, False) @ _blocks(b, True).t()
    elif which == "dgrad":
        y = _blocks(a, False) @ _blocks(b, True)
    else:
        y = _blocks(a.t(), False) @ _blocks(b.t(), False).t()
    return y.to(torch.bfloat16)


def _plain_xent(s):
    x, w, target = s["x"].float(), s["w"].float(), s["target"]
    valid = target != IGNORE
    at = torch.where(valid, target, 0)[:, None]
    z = x @ w.t()
    top = z.amax(dim=1, keepdim=True)
    lse = top + (z - top).exp().sum(dim=1, keepdim=True).log()
    loss = torch.where(valid, (lse - z.gather(1, at))[:, 0], 0.0)
    if not s["case"]["train"]:
        return dict(loss=loss, lse=lse[:, 0])
    d = torch.where(valid, s["dloss"], 0.0)[:, None]
    p = (z - lse).exp() * d
    p.scatter_add_(1, at, -d)
    return dict(loss=loss, lse=lse[:, 0], dx=(p @ w).to(torch.bfloat16), dw=(p.t() @ x).to(torch.bfloat16))


def _steps(x, a, b, c, k):
    """k Newton-Schulz steps X <- a X + (b A + c A A) X, A = X X^T."""
    if k == 0:
        return x
    A = x @ x.transpose(-1, -2)
    return _steps(a * x + (b * A + c * (A @ A)) @ x, a, b, c, k - 1)


def _plain_orthogonalize(s):
    x = s["g"].float()
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + 1e-7)
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-1, -2) if tall else x
    x = _steps(x, *NS_COEFFS, 5)
    return (x.transpose(-1, -2) if tall else x).to(torch.bfloat16)


def _own(s):
    import mxfp4_block_scaled_h16_amd as mx
    op = s["case"]["op"]
    if op == "fp8_linear":
        call = {"fprop": mx.fp8_linear_fprop, "dgrad": mx.fp8_linear_dgrad, "wgrad": mx.fp8_linear_wgrad}[s["case"]["which"]]
        return call(s["a"], s["b"], out_dtype=torch.bfloat16)
    if op == "xent":
        loss, lse = mx.linear_xent_forward(s["x"], s["w"], s["target"], ignore_index=IGNORE)
        if not s["case"]["train"]:
            return dict(loss=loss, lse=lse)
        dx, dw = mx.linear_xent_backward(s["dloss"], s["x"], s["w"], s["target"], lse, ignore_index=IGNORE)
        return dict(loss=loss, lse=lse, dx=dx, dw=dw)
    return mx.orthogonalize(s["g"], steps=5, coefficients=NS_COEFFS, out_dtype=torch.bfloat16)


def run(state):
    if own:
        return _own(state)
    return {"fp8_linear": _plain_fp8, "xent": _plain_xent, "orthogonalize": _plain_orthogonalize}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- its floor --
def work(case):
    if case["op"] == "fp8_linear":
        M, K, N = case["M"], case["K"], case["N"]
        ins, outs = {"fprop": (M * K + N * K, M * N), "dgrad": (M * N + N * K, M * K), "wgrad": (M * N + M * K, N * K)}[case["which"]]
        return {"bytes": 2 * ins + 2 * outs, "flops": 2 * M * K * N}
    if case["op"] == "xent":
        T, K, V = case["T"], case["K"], case["V"]
        ins = 2 * (T * K + V * K) + 8 * T
        if not case["train"]:
            return {"bytes": ins + 8 * T, "flops": 2 * T * K * V}
        return {"bytes": ins + 4 * T + 8 * T + 2 * (T * K + V * K), "flops": 6 * T * K * V}
    B, m, n = case["B"], case["m"], case["n"]
    s, l = min(m, n), max(m, n)
    # a step: the two symmetric products by half, the third whole
    return {"bytes": B * m * n * ((4 if case["dtype"] == "f32" else 2) + 2), "flops": B * 5 * (s * s * l + s * s * s + 2 * s * s * l)}


# ------------------------------------------------------------------------------- in 64 bits --
def _e4m3_64(y):
    """y, at most 448 in magnitude, to the nearest of the E4M3 values, ties to the even one: four significant
    bits, and steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(y)
    step = torch.exp2((e.double() - 4.0).clamp(min=-9.0))
    return torch.round(y / step) * step                 # torch.round: halves to even


def _quantized_64(v, height):
    """v in blocks of `height` rows x 128 columns (the rows' and columns' ends cut short), block by block maximum."""
    v = v.double()
    R, L = v.shape
    rows, cols = torch.arange(R, device=v.device) // height, torch.arange(L, device=v.device) // 128
    part = torch.full((R, int(cols[-1]) + 1), 0.0, dtype=torch.float64, device=v.device)
    part.scatter_reduce_(1, cols.expand(R, L), v.abs(), "amax")
    top = torch.full((int(rows[-1]) + 1, part.shape[1]), 0.0, dtype=torch.float64, device=v.device)
    top.scatter_reduce_(0, rows[:, None].expand(R, part.shape[1]), part, "amax")
    scale = torch.exp2(torch.ceil(torch.log2(top / FP8_MAX)).clamp(min=-127.0))      # top = 0: 2^-127
    # the logarithm may be a rounding off at a power of two: the smallest scale that fits is meant
    scale = torch.where(top > FP8_MAX * scale, 2.0 * scale, scale)
    scale = torch.where((top <= FP8_MAX * scale / 2) & (scale > 2.0 ** -127), scale / 2, scale)[rows][:, cols]
    return _e4m3_64(v / scale) * scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "fp8_linear":
        if case["which"] == "wgrad":
            a, b = _quantized_64(s["a"].t().contiguous(), 1), _quantized_64(s["b"].t().contiguous(), 1)
            return a @ b.t()
        a, b = _quantized_64(s["a"], 1), _quantized_64(s["b"], 128)
        return a @ (b.t() if case["which"] == "fprop" else b)
    if case["op"] == "xent":
        x, w, t = s["x"].double(), s["w"].double(), s["target"]
        z = torch.mm(x, w.t())
        lse = torch.logsumexp(z, dim=1)
        keep = t.ne(IGNORE)
        rows = torch.nonzero(keep)[:, 0]
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - z[rows, t[rows]]
        if not case["train"]:
            return dict(loss=loss, lse=lse)
        z.sub_(lse[:, None]).exp_()                      # the probabilities
        z[rows, t[rows]] -= 1.0
        z.mul_((s["dloss"].double() * keep)[:, None])
        return dict(loss=loss, lse=lse, dx=torch.mm(z, w), dw=torch.mm(z.t(), x))
    a, b, c = NS_COEFFS
    outs = []
    for g in s["g"].double().reshape(case["B"], case["m"], case["n"]):
        x = g / (torch.linalg.norm(g) + 1e-7)
        flip = case["m"] > case["n"]
        if flip:
            x = x.t().contiguous()
        for _ in range(5):
            gram = torch.mm(x, x.t())
            x = torch.addmm(x, torch.addmm(gram, gram, gram, beta=b, alpha=c), x, beta=a)
        outs.append(x.t() if flip else x)
    return torch.stack(outs).reshape(s["g"].shape)
