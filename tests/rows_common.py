"""Plain float64 implementations of the row operators (layer norm, gated
feed-forward, dropout) and the error bounds their kernels are held to.

The bounds follow the arithmetic, with e32 = 2^-24 (fp32) and u = half a step
of the result's type:

* a sum of m terms in fp32, in any order: at most m * 2 e32 * (sum of their
  absolute values); the factor 2 allows for the tensor core's accumulation,
  which truncates instead of rounding;
* an fp32 evaluation of an activation or its slope at v: at most
  2^-20 (1 + |v|) absolute for a value bounded by (1 + |v|): an exponential's
  argument carries |v| e32 relative error, and the quotient and products
  around it a few e32 more;
* one rounding to the result's type: u * |value|, and 2^-25 below fp16's
  normal range (half a subnormal step).
"""
import math

import torch

E32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rounding(ref, dtype):
    return UNIT[dtype] * ref.abs() + TINY[dtype]


def assert_close(got, ref, bound, what=""):
    """|got - ref| <= bound element by element; NaN and infinity in the same places."""
    got = got.double().cpu()
    ref, bound = ref.cpu(), bound.cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: non-finite values differ"
    err = torch.where(fine, (got - ref).abs(), torch.zeros_like(ref))
    bound = torch.where(fine, bound, torch.ones_like(ref))
    bad = err > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst error / "
                           f"bound {float((err / bound.clamp_min(1e-300)).max()):.3g}")


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def norm(x, gamma, beta, eps):
    x = x.double()
    xc = x - x.mean(1, keepdim=True)
    y = xc / torch.sqrt((xc * xc).mean(1, keepdim=True) + eps)
    if gamma is not None:
        y = y * gamma.double()
    return y if beta is None else y + beta.double()


def norm_grads(x, gamma, dy, eps):
    x, dy = x.double(), dy.double()
    xc = x - x.mean(1, keepdim=True)
    r = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + eps)
    xh = xc * r
    g = dy if gamma is None else dy * gamma.double()
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# A row sum is split over at least 4 threads, each adding at most 64 terms (c <=
# 16384: c / 256), then joined by at most 8 more additions.
SUM_TERMS = 72


def _norm_parts(x, eps):
    """xhat, 1/sqrt(var + eps) and the error of a computed xhat."""
    x = x.double()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    var = (xc * xc).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    dmean = SUM_TERMS * E32 * x.abs().mean(1, keepdim=True) + E32 * mean.abs()
    dxc = dmean + E32 * (x.abs() + mean.abs())      # of one x - mean
    dev = xc.abs()
    dvar = (2 * dev * dxc + dxc * dxc).mean(1, keepdim=True) + (SUM_TERMS + 4) * E32 * var
    # half the relative error of var + eps, at the smallest value it may have
    # taken; 4 more roundings in the inverse root
    low = torch.clamp(var + eps - dvar, min=0.5 * eps)
    dr = r * torch.clamp(0.5 * dvar / low, max=1e3) + 4 * E32 * r
    dxh = dxc * (r + dr) + dev * dr + 2 * E32 * dev * r
    return xc * r, r, dxh, dr


def norm_bound(x, gamma, beta, eps, dtype):
    ref = norm(x, gamma, beta, eps)
    xh, _, dxh, _ = _norm_parts(x, eps)
    g = 1.0 if gamma is None else gamma.double().abs()
    b = 0.0 if beta is None else beta.double().abs()
    return rounding(ref, dtype) + (dxh + 2 * E32 * xh.abs()) * g * 1.01 + 2 * E32 * b


def norm_grads_bound(x, gamma, dy, eps, dtype):
    dx, dgamma, dbeta = norm_grads(x, gamma, dy, eps)
    xh, r, dxh, dr = _norm_parts(x, eps)
    dy = dy.double()
    g = dy if gamma is None else dy * gamma.double()
    n = x.shape[0]
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dm1 = (SUM_TERMS + 2) * E32 * g.abs().mean(1, keepdim=True)
    dm2 = (g.abs() * dxh).mean(1, keepdim=True) + \
        (SUM_TERMS + 4) * E32 * (g * xh).abs().mean(1, keepdim=True)
    inner = g.abs() + m1.abs() + (xh * m2).abs()
    dinner = dm1 + dxh * (m2.abs() + dm2) + xh.abs() * dm2 + 4 * E32 * inner
    bdx = rounding(dx, dtype) + 1.01 * (r * dinner + dr * inner + E32 * r * inner)
    bgamma = (dy.abs() * dxh).sum(0) + (n + 4) * E32 * (dy * xh).abs().sum(0)
    bbeta = (n + 4) * E32 * dy.abs().sum(0)
    return bdx, bgamma + 1e-30, bbeta + 1e-30


# ---------------------------------------------------------------------------
# gated feed-forward
# ---------------------------------------------------------------------------
ACTS = ("none", "relu", "silu", "gelu")
# largest slope, and largest change of the slope, of each activation
LIP = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13}
LIP2 = {"none": 0.0, "relu": 0.0, "silu": 0.5, "gelu": 0.8}


def act(name, v):
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        return v.clamp(min=0), (v > 0).to(v.dtype)
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    cdf = 0.5 * torch.erfc(-v / math.sqrt(2))
    return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)


class Gated:
    """The gated product and its gradients in float64, with their bounds."""

    def __init__(self, x, W, bias, activation, dh=None, terms=lambda m: 2 * (m + 2)):
        """terms(m): how many roundings of 2^-24 a sum of m products may carry."""
        self.dtype, self.act = x.dtype, activation
        x, W = x.double(), W.double()
        b = torch.zeros(2, W.shape[2], dtype=torch.float64, device=x.device) if bias is None else \
            bias.double()
        g, u = x @ W[0] + b[0], x @ W[1] + b[1]
        c = x.shape[1]
        acc = terms(c) * E32
        dg, du = (acc * (x.abs() @ W[k].abs() + b[k].abs()) for k in (0, 1))
        a, s = act(activation, g)
        ev = 2.0 ** -20 * (1 + g.abs())  # of the activation or its slope
        da = LIP[activation] * dg + (0 if activation in ("none", "relu") else ev)
        self.out = a * u
        self.out_bound = rounding(self.out, self.dtype) + \
            1.01 * (da * (u.abs() + du) + a.abs() * du + 2 * E32 * (a * u).abs())
        if dh is None:
            return
        dh = dh.double()
        ds = LIP2[activation] * dg + (0 if activation in ("none", "relu") else ev)
        if activation == "relu":
            ds = ds + (g.abs() <= dg).double()  # the side of the kink is not known
        G, U = dh * u * s, dh * a
        eg = dh.abs() * (ds * (u.abs() + du) + s.abs() * du) + 3 * E32 * G.abs() + \
            rounding(G, self.dtype)
        eu = dh.abs() * da + 2 * E32 * U.abs() + rounding(U, self.dtype)
        n, h = dh.shape
        self.dx = G @ W[0].T + U @ W[1].T
        self.dx_bound = rounding(self.dx, self.dtype) + 1.01 * (
            eg @ W[0].abs().T + eu @ W[1].abs().T +
            terms(2 * h) * E32 * (G.abs() @ W[0].abs().T + U.abs() @ W[1].abs().T))
        xa = x.abs().T
        self.dW = torch.stack([x.T @ G, x.T @ U])
        self.dW_bound = rounding(self.dW, self.dtype) + 1.01 * torch.stack(
            [xa @ e + terms(n) * E32 * (xa @ v.abs()) for e, v in ((eg, G), (eu, U))])
        self.db = torch.stack([G.sum(0), U.sum(0)])
        self.db_bound = rounding(self.db, self.dtype) + 1.01 * torch.stack(
            [e.sum(0) + terms(n) * E32 * v.abs().sum(0) for e, v in ((eg, G), (eu, U))])


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
def philox(c, k):
    """Philox-4x32-10 on Python integers: counter of 4 words, key of 2."""
    m = 0xFFFFFFFF
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def keep_bits(first, count, seed, offset):
    """The 16 random bits of elements first .. first + count - 1."""
    m = 0xFFFFFFFF
    out, words, group = [], None, None
    for i in range(first, first + count):
        if i // 8 != group:
            group = i // 8
            words = philox((group & m, group >> 32, offset & m, offset >> 32),
                           (seed & m, seed >> 32))
        out.append(words[i % 8 // 2] >> (16 * (i % 2)) & 0xFFFF)
    return torch.tensor(out)


def dropout(x, p, seed, offset, residual=None):
    t = round(p * 65536)
    keep = keep_bits(0, x.numel(), seed, offset).view(x.shape) >= t
    scale = 65536 / (65536 - t) if t < 65536 else 0.0
    out = torch.where(keep, x.double().cpu() * scale, torch.zeros(1, dtype=torch.float64))
    return out if residual is None else out + residual.double().cpu()
