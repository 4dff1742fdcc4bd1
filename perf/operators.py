"""The row operators of a sparse feed-forward block, as they are measured.

The block that follows a submanifold convolution in a sparse transformer stage
works on the [N, C] feature rows alone:

    x  ->  layer norm  ->  gated feed-forward (both projections, activation and
    product)  ->  1x1x1 convolution (down projection)  ->  dropout + residual

Measured here are layer norm, the gated feed-forward product and dropout, each
with its backward pass, on the row counts and channels of this repository's
workloads (424 voxels of a 16^3 grid, 26,214 of 64^3, 209,715 of 128^3, 55,100
of the 64^3 shells, 4,749,279 of the two 512^3 scenes; 64 to 1024 channels) and
on odd sizes around them.

Definitions (per row x, all sums over the row's channels):

    layer norm   y = (x - mean) / sqrt(var + eps) * gamma + beta
    gated        out = act(x @ W[0] + b[0]) * (x @ W[1] + b[1])
    dropout      out = residual + keep * x / (1 - p)

dropout's keep bits come from the Philox-4x32-10 counter generator (Salmon,
Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
elements 8 g .. 8 g + 7 take the eight 16-bit halves, low half first, of the
four words of counter (g mod 2^32, g >> 32, offset mod 2^32, offset >> 32)
under the key (seed mod 2^32, seed >> 32).  With t = round(p * 65536) an
element is kept when its 16 bits are >= t, and scaled by 65536 / (65536 - t).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, back, n, c, dtype, affine=True):
    return {"name": name, "op": "norm_backward" if back else "norm", "n": n, "c": c,
            "dtype": dtype, "affine": affine}


def _gated(name, back, n, c, hidden, dtype, act, bias):
    return {"name": name, "op": "gated_backward" if back else "gated", "n": n, "c": c,
            "hidden": hidden, "dtype": dtype, "act": act, "bias": bias}


def _dropout(name, n, c, dtype, p, residual):
    return {"name": name, "op": "dropout", "n": n, "c": c, "dtype": dtype, "p": p,
            "residual": residual}


def listed():
    return [
        # the smallest scene, one normalisation in the middle of a network: latency
        _norm("norm_tiny16", False, 424, 128, "bf16"),
        # two full 512^3 scenes, 64 channels: 1.2 GB through memory
        _norm("norm_shells512", False, 4749279, 64, "bf16"),
        # the training step's pass back through a 128-channel stage
        _norm("norm_bwd_uniform128", True, 209715, 128, "f16"),
        # odd channels (concatenated skip features), fp32 training
        _norm("norm_bwd_odd", True, 26213, 515, "f32"),
        # the smallest scene through the wide projections: latency
        _gated("gated_tiny16", False, 424, 128, 512, "bf16", "silu", True),
        # the channel-heavy stage, inference
        _gated("gated_resblock64", False, 55100, 512, 2048, "bf16", "silu", True),
        # channels off every power of two, fp16
        _gated("gated_odd", False, 26213, 100, 387, "f16", "gelu", True),
        # fp32 inference
        _gated("gated_f32", False, 26214, 128, 512, "f32", "silu", False),
        # the channel-heavy stage, training
        _gated("gated_bwd_resblock64", True, 55100, 512, 2048, "bf16", "silu", True),
        # a narrow stage, training
        _gated("gated_bwd_uniform64", True, 26214, 64, 256, "f16", "gelu", True),
        # the block's closing sum: dropout of the branch plus the skip connection
        _dropout("dropout_residual", 209715, 512, "bf16", 0.1, True),
        # its backward pass on odd rows: the same mask on the gradient
        _dropout("dropout_odd", 26213, 515, "f32", 0.25, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "gated", "gated", "gated_backward", "gated_backward",
                     "dropout"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    step = rng.choice([1, 8, 64])  # any channel count, vector-sized ones, tile-sized ones
    if op.startswith("gated"):
        c = step * _log(rng, max(1, 16 // step), max(1, 1024 // step))
        hidden = step * _log(rng, max(1, 16 // step), max(1, 2048 // step))
        most = 55100 * 512 * 2048 // (16 if dtype == "f32" else 1)
        n = _log(rng, 1, max(1, min(300000, most // (c * hidden), 55100 * 2560 // (c + hidden))))
        return {"op": op, "n": n, "c": c, "hidden": hidden, "dtype": dtype,
                "act": rng.choice(["silu", "gelu", "relu", "none"]), "bias": rng.random() < 0.5}
    c = step * _log(rng, max(1, 8 // step), max(1, 2048 // step))
    most = 4749279 * 64 // (4 if dtype == "f32" or op != "norm" else 1)
    n = _log(rng, 1, max(1, min(4749279, most // c)))
    if op == "dropout":
        return {"op": op, "n": n, "c": c, "dtype": dtype, "p": rng.choice([0.05, 0.1, 0.25, 0.5]),
                "residual": rng.random() < 0.5}
    return {"op": op, "n": n, "c": c, "dtype": dtype, "affine": rng.random() < 0.75}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(case, seed):
    """Everything that is drawn, in order: used by prepare() and by exact()."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, n, c, op = DTYPES[case["dtype"]], case["n"], case["c"], case["op"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * scale

    s = {"x": normal(n, c)}
    if op.startswith("norm"):
        # channels of unequal spread around a row offset, as after a residual sum
        s["x"] = s["x"] * (0.5 + torch.rand(c, generator=g, device=DEV)) + normal(n, 1, scale=0.5)
        if case["affine"]:
            s["gamma"] = 1.0 + normal(c, scale=0.1)
            s["beta"] = normal(c, scale=0.1)
        if op == "norm_backward":
            s["grad_out"] = normal(n, c).to(dt)
    elif op.startswith("gated"):
        h = case["hidden"]
        s["W"] = normal(2, c, h, scale=c ** -0.5).to(dt)
        s["bias"] = normal(2, h, scale=0.1).to(dt) if case["bias"] else None
        if op == "gated_backward":
            s["grad_out"] = normal(n, h).to(dt)
    elif case["residual"]:
        s["residual"] = normal(n, c).to(dt)
    s["x"] = s["x"].to(dt)
    if op == "dropout":
        # a training program's seed, and the number of the call under it
        s["seed"] = (0x9E3779B97F4A7C15 * (seed + 1)) % (1 << 63)
        s["offset"] = 1 + seed % 7
    return s


def prepare(case, seed):
    s = _rows(case, seed)
    s["case"] = dict(case)
    if own and case["op"].startswith("gated"):
        # the index that a program holds for its voxels
        from submanifold_sparse_convolution_coord_b200.binding import SubMIndex
        i = torch.arange(case["n"], device=DEV)
        coords = torch.stack([i // 2 ** 21, i // 2 ** 14 % 128, i // 128 % 128, i % 128], 1)
        s["index"] = SubMIndex(coords.to(torch.int32))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    return (_run_own if own else _run_plain)(case["op"], case, s)


def _run_own(op, case, s):
    from submanifold_sparse_convolution_coord_b200 import binding as smc
    if op == "norm":
        return smc.smc_layer_norm(s["x"], s.get("gamma"), s.get("beta"), EPS)
    if op == "norm_backward":
        dx, dgamma, dbeta = smc.smc_layer_norm_backward(s["x"], s.get("gamma"), s["grad_out"], EPS)
        return {"grad_in": dx, "grad_gamma": dgamma, "grad_beta": dbeta}
    if op == "gated":
        return s["index"].gated_forward(s["x"], s["W"], bias=s["bias"], activation=case["act"])
    if op == "gated_backward":
        dx, dw, db = s["index"].gated_backward(s["x"], s["W"], s["grad_out"], bias=s["bias"],
                                               activation=case["act"])
        return {"grad_in": dx, "grad_W": dw, "grad_bias": db}
    return smc.smc_dropout(s["x"], case["p"], s["seed"], s["offset"], residual=s.get("residual"))


def _run_plain(op, case, s):
    dt = DTYPES[case["dtype"]]
    x = s["x"].float()
    if op.startswith("norm"):
        xc = x - x.mean(1, keepdim=True)
        rstd = torch.rsqrt(xc.square().mean(1, keepdim=True) + EPS)
        xhat = xc * rstd
        if op == "norm":
            return (xhat * s["gamma"] + s["beta"] if case["affine"] else xhat).to(dt)
        dy = s["grad_out"].float()
        dxhat = dy * s["gamma"] if case["affine"] else dy
        dx = rstd * (dxhat - dxhat.mean(1, keepdim=True)
                     - xhat * (dxhat * xhat).mean(1, keepdim=True))
        return {"grad_in": dx.to(dt), "grad_gamma": (dy * xhat).sum(0) if case["affine"] else None,
                "grad_beta": dy.sum(0) if case["affine"] else None}
    if op.startswith("gated"):
        W = s["W"].float()
        g, u = x @ W[0], x @ W[1]
        if s["bias"] is not None:
            g, u = g + s["bias"][0].float(), u + s["bias"][1].float()
        a, da = _activation(case["act"], g)
        if op == "gated":
            return (a * u).to(dt)
        dh = s["grad_out"].float()
        dg, du = dh * u * da, dh * a
        return {"grad_in": (dg @ W[0].T + du @ W[1].T).to(dt),
                "grad_W": torch.stack([x.T @ dg, x.T @ du]).to(dt),
                "grad_bias": None if s["bias"] is None else torch.stack([dg.sum(0), du.sum(0)]).to(dt)}
    keep, scale = _keep_bits(x.numel(), case["p"], s["seed"], s["offset"])
    out = torch.where(keep.view_as(x), x * scale, 0.0)
    return (out + s["residual"].float() if case["residual"] else out).to(dt)


def _activation(name, g):
    """act(g) and its derivative."""
    if name == "none":
        return g, torch.ones_like(g)
    if name == "relu":
        return torch.clamp(g, min=0), (g > 0).float()
    if name == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    cdf = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _keep_bits(count, p, seed, offset):
    """dropout's keep decisions, from the definition, in 64-bit integers."""
    m32 = 0xFFFFFFFF
    i = torch.arange((count + 7) // 8, device=DEV)
    c0, c1 = i & m32, i >> 32
    c2, c3 = torch.full_like(i, offset & m32), torch.full_like(i, offset >> 32)
    k0, k1 = seed & m32, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits; the high word is taken unsigned
        c0, c1, c2, c3 = (b >> 32 & m32) ^ c1 ^ k0, b & m32, (a >> 32 & m32) ^ c3 ^ k1, a & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    bits = torch.stack([w for v in (c0, c1, c2, c3) for w in (v & 0xFFFF, v >> 16)], 1)
    t = round(p * 65536)
    return bits.view(-1)[:count] >= t, 65536 / (65536 - t) if t < 65536 else 0.0


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e, n, c, op = BYTES[case["dtype"]], case["n"], case["c"], case["op"]
    if op == "norm":  # rows in, rows out, gamma and beta
        return {"bytes": 2 * n * c * e + (8 * c if case["affine"] else 0), "flops": 8 * n * c}
    if op == "norm_backward":  # rows and gradients in, gradients out, gamma in, its and beta's out
        return {"bytes": 3 * n * c * e + (12 * c if case["affine"] else 0), "flops": 14 * n * c}
    if op == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * n * c * e, "flops": 2 * n * c}
    h = case["hidden"]
    weights = (2 * c * h + (2 * h if case["bias"] else 0)) * e
    if op == "gated":  # two products
        return {"bytes": n * (c + h) * e + weights, "flops": 4 * n * c * h}
    # the pre-activations again, the rows' gradient and the weights': three times two products
    return {"bytes": n * (2 * c + h) * e + 2 * weights, "flops": 12 * n * c * h}


# ---------------------------------------------------------------------------
# in 64 bits, from torch's own functions and their derivatives
# ---------------------------------------------------------------------------
def exact(case, seed):
    s, op = _rows(case, seed), case["op"]
    f = torch.nn.functional
    wide = {k: v.double().requires_grad_() for k, v in s.items() if isinstance(v, torch.Tensor)}
    x = wide["x"]
    if op.startswith("norm"):
        y = f.layer_norm(x, (case["c"],), wide.get("gamma"), wide.get("beta"), EPS)
        if op == "norm":
            return y.detach()
        want = [x] + ([wide["gamma"], wide["beta"]] if case["affine"] else [])
        got = torch.autograd.grad(y, want, wide["grad_out"].detach())
        return dict(zip(("grad_in", "grad_gamma", "grad_beta"), list(got) + [None] * (3 - len(got))))
    if op.startswith("gated"):
        act = {"silu": f.silu, "gelu": f.gelu, "relu": f.relu, "none": lambda v: v}[case["act"]]
        b = wide.get("bias")
        g, u = (f.linear(x, wide["W"][k].T, None if b is None else b[k]) for k in (0, 1))
        y = act(g) * u
        if op == "gated":
            return y.detach()
        want = [x, wide["W"]] + ([] if b is None else [b])
        got = torch.autograd.grad(y, want, wide["grad_out"].detach())
        return dict(zip(("grad_in", "grad_W", "grad_bias"), list(got) + [None] * (3 - len(got))))
    x = x.detach()
    t = round(case["p"] * 65536)
    words = _philox_words(torch.arange(-(-x.numel() // 8), device=DEV), s["seed"], s["offset"])
    out = torch.zeros(words.shape[0] * 8, dtype=torch.float64, device=DEV)
    for j in range(8):
        half = words[:, j // 2] // (65536 if j % 2 else 1) % 65536
        out[j::8] = (half >= t).double() * (65536 / (65536 - t))
    out = out[:x.numel()].view_as(x) * x
    return out + wide["residual"].detach() if case["residual"] else out


def _philox_words(group, seed, offset):
    """The four words of each group, with the 64-bit products taken in 16-bit limbs."""
    def product(v, m):
        lo, hi = (v % 65536) * m, (v // 65536) * m  # each below 2^48
        mid = lo // 65536 + hi
        return mid // 65536, (mid % 65536) * 65536 + lo % 65536
    word = [group % 2 ** 32, group // 2 ** 32, torch.full_like(group, offset % 2 ** 32),
            torch.full_like(group, offset // 2 ** 32)]
    for r in range(10):
        key = [(seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        (h0, l0), (h1, l1) = product(word[0], 0xD2511F53), product(word[2], 0xCD9E8D57)
        word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
    return torch.stack(word, 1)
