"""Row operators (layer norm, gated feed-forward, dropout) on the GPU against
plain float64 implementations, element by element, under the bounds that
rows_common derives."""
import ctypes

import pytest
import torch

from submanifold_sparse_convolution_coord_b200 import binding
from submanifold_sparse_convolution_coord_b200.binding import (SubMIndex, smc_dropout,
                                                               smc_layer_norm,
                                                               smc_layer_norm_backward)

import rows_common as rc

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _randn(*shape, seed=0, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _index(n):
    i = torch.arange(n, device=DEV)
    c = torch.stack([i // 2 ** 18, i // 4096 % 64, i // 64 % 64, i % 64], 1)
    return SubMIndex(c.to(torch.int32))


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
NORM_SHAPES = [(1, 1), (5, 2), (1, 64), (3, 7), (424, 16), (1000, 64), (129, 128), (77, 130),
               (50, 255), (64, 512), (33, 515), (20, 1000), (300, 1024), (9, 2048), (5, 4099),
               (3, 8192), (2, 16384), (40001, 8), (3001, 96), (700, 12), (513, 24), (260, 48),
               (200, 192), (99, 640), (65, 641), (130, 386), (40, 1282), (7, 2560), (1037, 3)]


def _norm_inputs(n, c, dt, seed=0):
    x = (_randn(n, c, seed=seed) * (0.5 + _randn(c, seed=seed + 1).abs()) +
         3 * _randn(n, 1, seed=seed + 2)).to(dt)
    return (x, 1 + _randn(c, seed=seed + 3, scale=0.3), _randn(c, seed=seed + 4),
            _randn(n, c, seed=seed + 5, dtype=dt))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm(shape, dt):
    x, gamma, beta, _ = _norm_inputs(*shape, rc.DTYPES[dt])
    for g, b in ((gamma, beta), (None, None), (gamma, None), (None, beta)):
        got = smc_layer_norm(x, g, b, 1e-5)
        rc.assert_close(got, rc.norm(x, g, b, 1e-5), rc.norm_bound(x, g, b, 1e-5, x.dtype),
                        f"{shape} {dt} {g is not None} {b is not None}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm_backward(shape, dt):
    x, gamma, _, dy = _norm_inputs(*shape, rc.DTYPES[dt], seed=7)
    for g in (gamma, None):
        got = smc_layer_norm_backward(x, g, dy, 1e-3)
        refs = rc.norm_grads(x, g, dy, 1e-3)
        bounds = rc.norm_grads_bound(x, g, dy, 1e-3, x.dtype)
        for name, a, r, b in zip(("grad_in", "grad_gamma", "grad_beta"), got, refs, bounds):
            if a is None:
                assert g is None and name != "grad_in"
                continue
            rc.assert_close(a, r, b, f"{shape} {dt} {name}")
        again = smc_layer_norm_backward(x, g, dy, 1e-3)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


def test_norm_many_rows():
    """More rows than a grid covers at once, and sums over all of them."""
    x, gamma, beta, dy = _norm_inputs(700001, 16, torch.bfloat16, seed=11)
    rc.assert_close(smc_layer_norm(x, gamma, beta), rc.norm(x, gamma, beta, 1e-5),
                    rc.norm_bound(x, gamma, beta, 1e-5, x.dtype), "forward")
    got = smc_layer_norm_backward(x, gamma, dy)
    for a, r, b in zip(got, rc.norm_grads(x, gamma, dy, 1e-5),
                       rc.norm_grads_bound(x, gamma, dy, 1e-5, x.dtype)):
        rc.assert_close(a, r, b)


@pytest.mark.parametrize("c", [64, 515, 4099])
def test_norm_bad_rows_stay_alone(c):
    """NaN and infinities spoil their own row, constant rows give beta."""
    x, gamma, beta, dy = _norm_inputs(12, c, torch.float32, seed=13)
    clean = smc_layer_norm(x, gamma, beta)
    clean_dx = smc_layer_norm_backward(x, gamma, dy)[0]
    bad = x.clone()
    bad[3, 1] = float("nan")
    bad[5, c - 1] = float("inf")
    bad[7] = 2.5
    got = smc_layer_norm(bad, gamma, beta)
    dx = smc_layer_norm_backward(bad, gamma, dy)[0]
    others = [i for i in range(12) if i not in (3, 5, 7)]
    assert torch.equal(got[others], clean[others]) and torch.equal(dx[others], clean_dx[others])
    assert got[3].isnan().all() and got[5].isnan().all()
    rc.assert_close(got[7:8], rc.norm(bad[7:8], gamma, beta, 1e-5),
                    rc.norm_bound(bad[7:8], gamma, beta, 1e-5, x.dtype))


def test_norm_no_rows_and_in_place():
    x, gamma, beta, dy = _norm_inputs(37, 128, torch.float16, seed=17)
    want = smc_layer_norm(x, gamma, beta)
    y = x.clone()
    assert smc_layer_norm(y, gamma, beta, out=y) is y
    assert torch.equal(y, want)
    assert smc_layer_norm(x[:0], gamma, beta).shape == (0, 128)
    dx, dgamma, dbeta = smc_layer_norm_backward(x[:0], gamma, dy[:0])
    assert dx.shape == (0, 128) and not dgamma.any() and not dbeta.any()


def test_norm_gradient_against_differences():
    """The computed gradient along random directions against central
    differences of the float64 formula (step 1e-5: the difference is off by
    about 1e-10 of the third derivatives plus 1e-11 of rounding)."""
    x, gamma, beta, dy = _norm_inputs(9, 33, torch.float32, seed=19)
    dx, dgamma, dbeta = (v.double() for v in smc_layer_norm_backward(x, gamma, dy, 1e-2))
    w, h = dy.double(), 1e-5

    def loss(a, b, c):
        return float((rc.norm(a, b, c, 1e-2) * w).sum())

    x, gamma, beta = x.double(), gamma.double(), beta.double()
    for seed in range(3):
        d = [_randn(*v.shape, seed=100 + seed).double() for v in (x, gamma, beta)]
        diff = (loss(*(v + h * e for v, e in zip((x, gamma, beta), d))) -
                loss(*(v - h * e for v, e in zip((x, gamma, beta), d)))) / (2 * h)
        terms = [(a * b).sum() for a, b in zip((dx, dgamma, dbeta), d)]
        size = sum(float((a * b).abs().sum()) for a, b in zip((dx, dgamma, dbeta), d))
        assert abs(diff - float(sum(terms))) <= 1e-5 * size


def test_norm_far_rows():
    """More than 2^31 elements: rows at the start, around 2^31 elements and at
    the end equal those of a call on these rows alone."""
    n, c = 33_600_000, 64
    x = torch.empty(n, c, dtype=torch.bfloat16, device=DEV)
    picked = [slice(0, 300), slice((1 << 31) // c - 150, (1 << 31) // c + 150), slice(n - 300, n)]
    x.fill_(1.0)
    for k, rows in enumerate(picked):
        x[rows] = _randn(300, c, seed=60 + k, dtype=torch.bfloat16)
    _, gamma, beta, _ = _norm_inputs(2, c, torch.bfloat16, seed=63)
    y = smc_layer_norm(x, gamma, beta)
    for rows in picked:
        assert torch.equal(y[rows], smc_layer_norm(x[rows].clone(), gamma, beta))
    # y has served; its memory takes the gradient
    dx, dgamma, dbeta = smc_layer_norm_backward(x, gamma, x, grad_in=y)
    for rows in picked:
        part = x[rows].clone()
        assert torch.equal(dx[rows], smc_layer_norm_backward(part, gamma, part)[0])
    # the constant rows have xhat = 0 (their mean is exact) and add n - 900 to dbeta
    parts = [rc.norm_grads(x[rows], gamma, x[rows], 1e-5) for rows in picked]
    want = sum(p[2] for p in parts) + (n - 900)
    size = sum(x[rows].double().abs().sum(0) for rows in picked) + (n - 900)
    rc.assert_close(dbeta, want, n * rc.E32 * size, "dbeta")
    want = sum(p[1] for p in parts)
    bound = sum(rc.norm_grads_bound(x[rows], gamma, x[rows], 1e-5, x.dtype)[1] for rows in picked)
    rc.assert_close(dgamma, want, bound + 1000 * rc.E32 * 900, "dgamma")


def test_norm_refusals():
    x, gamma, beta, dy = _norm_inputs(8, 64, torch.float16, seed=23)
    with pytest.raises(ValueError):
        smc_layer_norm(x.t())  # not contiguous
    with pytest.raises(ValueError):
        smc_layer_norm(x, gamma.half())
    with pytest.raises(ValueError):
        smc_layer_norm(x, gamma[:32].contiguous())
    with pytest.raises(ValueError):
        smc_layer_norm_backward(x, gamma, dy.float())
    with pytest.raises(ValueError):
        smc_layer_norm(x, out=torch.empty(7, 64, dtype=x.dtype, device=DEV))
    with pytest.raises(binding.SmcError):  # overlapping, not the same
        buf = torch.zeros(9 * 64, dtype=torch.float16, device=DEV)
        smc_layer_norm(buf[:512].view(8, 64), out=buf[64:].view(8, 64))
    with pytest.raises(binding.SmcError):
        smc_layer_norm_backward(x, gamma, dy, grad_in=x)
    with pytest.raises(binding.SmcError):  # 2 bytes off a 16-byte boundary
        smc_layer_norm(torch.zeros(65, dtype=torch.float16, device=DEV)[1:].view(1, 64))


# ---------------------------------------------------------------------------
# gated feed-forward
# ---------------------------------------------------------------------------
# (n, cin, hidden)
GATED_SHAPES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (127, 64, 128), (128, 128, 64), (129, 65, 127),
                (300, 100, 387), (424, 128, 512), (257, 512, 256), (1000, 16, 1000),
                (515, 264, 72), (64, 1024, 40), (3000, 8, 8), (2500, 192, 320)]


def _gated_inputs(n, c, h, dt, seed=0, bias=True):
    dtype = rc.DTYPES[dt]
    return (_randn(n, c, seed=seed, dtype=dtype),
            _randn(2, c, h, seed=seed + 1, dtype=dtype, scale=c ** -0.5),
            _randn(2, h, seed=seed + 2, dtype=dtype, scale=0.3) if bias else None,
            _randn(n, h, seed=seed + 3, dtype=dtype))


def _check_gated(idx, x, W, bias, act, dh, what):
    ref = rc.Gated(x, W, bias, act, dh)
    out = idx.gated_forward(x, W, bias, act)
    dx, dW, db = idx.gated_backward(x, W, dh, bias, act)
    torch.cuda.synchronize()
    assert idx.status() == 0
    rc.assert_close(out, ref.out, ref.out_bound, what + " out")
    rc.assert_close(dx, ref.dx, ref.dx_bound, what + " grad_in")
    rc.assert_close(dW, ref.dW, ref.dW_bound, what + " grad_W")
    if bias is None:
        assert db is None
    else:
        rc.assert_close(db, ref.db, ref.db_bound, what + " grad_bias")
    return out, dx, dW, db


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", GATED_SHAPES, ids=str)
def test_gated(shape, dt):
    n, c, h = shape
    with _index(n) as idx:
        for k, act in enumerate(rc.ACTS if n < 1000 else ("silu",)):
            x, W, b, dh = _gated_inputs(n, c, h, dt, seed=10 * k, bias=k % 2 == 0)
            _check_gated(idx, x, W, b, act, dh, f"{shape} {dt} {act}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gated_many_rows(dt):
    """Enough rows that every SM takes several tiles and the sums over rows are
    split many ways; the same call twice gives the same bits."""
    n, c, h = 30001, 128, 200
    with _index(n) as idx:
        x, W, b, dh = _gated_inputs(n, c, h, dt, seed=50)
        first = _check_gated(idx, x, W, b, "gelu", dh, f"many rows {dt}")
        out = idx.gated_forward(x, W, b, "gelu")
        again = (out,) + idx.gated_backward(x, W, dh, b, "gelu")
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gated_fp32_long_sums():
    """fp32 sums are accumulated 64 terms at a time (24 steps of the matrix unit,
    each cutting up to two roundings, and 4 for the parts that are dropped) and
    added up with one rounding per 64 terms and per share of the rows (at most
    148); the bias gradient adds 32 rows by 5 steps, then the 32-row sums."""
    for n, c, h in ((64, 4096, 72), (20001, 100, 136), (300, 64, 3000)):
        with _index(n) as idx:
            x, W, b, dh = _gated_inputs(n, c, h, "f32", seed=110)
            ref = rc.Gated(x, W, b, "silu", dh, terms=lambda m: 52 + m // 64 + 148)
            dx, dW, db = idx.gated_backward(x, W, dh, b)
            rc.assert_close(idx.gated_forward(x, W, b), ref.out, ref.out_bound, f"{n} {c} {h} out")
            rc.assert_close(dx, ref.dx, ref.dx_bound, f"{n} {c} {h} grad_in")
            rc.assert_close(dW, ref.dW, ref.dW_bound, f"{n} {c} {h} grad_W")
            rc.assert_close(db, ref.db, ref.db_bound, f"{n} {c} {h} grad_bias")


_ABORT_SCRIPT = r"""
import sys, torch
sys.path.insert(0, {root!r})
from submanifold_sparse_convolution_coord_b200.binding import SubMIndex
statuses = []
for n, c, h, dt in [(20000, 128, 512, torch.float16), (3000, 64, 64, torch.bfloat16),
                    (3000, 100, 130, torch.float32)]:
    i = torch.arange(n, device="cuda")
    idx = SubMIndex(torch.stack([i * 0, i // 4096, i // 64 % 64, i % 64], 1).to(torch.int32))
    x = torch.randn(n, c, device="cuda").to(dt)
    W = torch.randn(2, c, h, device="cuda").to(dt)
    b, dh = torch.randn(2, h, device="cuda").to(dt), torch.randn(n, h, device="cuda").to(dt)
    for _ in range(2):
        idx.gated_forward(x, W, b)
        idx.gated_backward(x, W, dh, b)
    torch.cuda.synchronize()
    statuses.append(idx.status())
    idx.close()
print("statuses", statuses)
"""


@pytest.mark.parametrize("limit_ns,must_abort", [(200, True), (20000, False)])
def test_gated_bounded_wait_abort_path(limit_ns, must_abort):
    """With the wait limit cut to a debug value, waits give up in mid-pipeline:
    the kernels drain what they issued, free tensor memory, return and report
    through the status word, and the context stays usable."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = _ABORT_SCRIPT.format(root=os.path.dirname(here))
    env = dict(os.environ, SMC_DEBUG_WAIT_LIMIT_NS=str(limit_ns))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    line = [ln for ln in r.stdout.splitlines() if ln.startswith("statuses")][0]
    statuses = eval(line.split(" ", 1)[1])
    assert all(s in (0, -8) for s in statuses), statuses  # ok or a timeout, nothing else
    if must_abort:
        # a wait that the hardware's own suspension covers never looks at the
        # limit, as in short chains of stages; the first case has long ones
        assert statuses[0] == -8, statuses
    with _index(700) as idx:  # the normal limit, in this process
        x, W, b, dh = _gated_inputs(700, 128, 256, "f16", seed=120)
        _check_gated(idx, x, W, b, "silu", dh, "after abort runs")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_gated_large_pre_activations(dt):
    """Gates far out on both sides: the activation's tails."""
    n, c, h = 200, 64, 96
    with _index(n) as idx:
        x, W, b, dh = _gated_inputs(n, c, h, dt, seed=60)
        x = (x * 30).to(x.dtype)
        for act in rc.ACTS:
            _check_gated(idx, x, W, b, act, dh, f"large {dt} {act}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_gated_bad_rows_stay_alone(dt):
    """NaN and infinity in a row reach that row only; in grad_W, every entry
    they touch."""
    n, c, h = 300, 72, 136
    with _index(n) as idx:
        x, W, b, dh = _gated_inputs(n, c, h, dt, seed=70)
        clean = idx.gated_forward(x, W, b)
        clean_dx = idx.gated_backward(x, W, dh, b)[0]
        x2 = x.clone()
        x2[5, 3], x2[200, 71], x2[299, 0] = float("nan"), float("nan"), float("inf")
        got, dx = idx.gated_forward(x2, W, b), idx.gated_backward(x2, W, dh, b)[0]
        others = [i for i in range(n) if i not in (5, 200, 299)]
        assert torch.equal(got[others], clean[others]) and torch.equal(dx[others], clean_dx[others])
        assert got[5].isnan().all() and got[200].isnan().all()
        assert not torch.isfinite(got[299]).all()
        assert idx.status() == 0


def test_gated_gradient_against_differences():
    n, c, h = 13, 21, 34
    with _index(n) as idx:
        x, W, b, dh = _gated_inputs(n, c, h, "f32", seed=80)
        for act in ("none", "silu", "gelu"):
            grads = [v.double() for v in idx.gated_backward(x, W, dh, b, act)]
            at = [v.double() for v in (x, W, b)]

            def loss(a, w, q):
                g, u = a @ w[0] + q[0], a @ w[1] + q[1]
                return float((rc.act(act, g)[0] * u * dh.double()).sum())

            d = [_randn(*v.shape, seed=200).double() for v in at]
            s = 1e-5
            diff = (loss(*(v + s * e for v, e in zip(at, d))) -
                    loss(*(v - s * e for v, e in zip(at, d)))) / (2 * s)
            size = sum(float((a * e).abs().sum()) for a, e in zip(grads, d))
            assert abs(diff - sum(float((a * e).sum()) for a, e in zip(grads, d))) <= 1e-5 * size


def test_gated_far_rows():
    """More than 2^31 hidden values: rows at the start, around 2^31 values and at
    the end, and the weight gradient of all rows (added up in float64 in pieces)."""
    n, c, h = 1_100_000, 16, 2048
    with _index(n) as idx:
        x, W, b, dh = _gated_inputs(n, c, h, "bf16", seed=130)
        out = idx.gated_forward(x, W, b)
        dx, dW, db = idx.gated_backward(x, W, dh, b)
        at = (1 << 31) // h
        for rows in (slice(0, 200), slice(at - 100, at + 100), slice(n - 200, n)):
            ref = rc.Gated(x[rows], W, b, "silu", dh[rows])
            rc.assert_close(out[rows], ref.out, ref.out_bound, "out")
            rc.assert_close(dx[rows], ref.dx, ref.dx_bound, "grad_in")
        want = bound = 0
        for r in range(0, n, 100_000):
            ref = rc.Gated(x[r:r + 100_000], W, b, "silu", dh[r:r + 100_000], terms=lambda m: 0)
            want = want + ref.dW
            bound = bound + ref.dW_bound
            del ref
        # each piece's bound holds a rounding of its own, and no accumulation error:
        # that of n rows, in shares of n / 37, is far below the roundings of dg and du
        assert (dW.double() - want).norm() <= bound.norm()
        assert idx.status() == 0


def test_gated_first_call_captured():
    """The first call of a process may be one that a graph captures."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import sys, torch
sys.path.insert(0, {root!r})
from submanifold_sparse_convolution_coord_b200.binding import (SubMIndex, smc_dropout, smc_layer_norm,
                                                               smc_layer_norm_backward)
i = torch.arange(500, device="cuda")
idx = SubMIndex(torch.stack([i * 0, i * 0, i // 64, i % 64], 1).to(torch.int32))
x = torch.randn(500, 100, device="cuda").half()
W, dh = torch.randn(2, 100, 64, device="cuda").half(), torch.randn(500, 64, device="cuda").half()
gamma = torch.ones(100, device="cuda")
def step():
    y = smc_layer_norm(x, gamma)
    out = smc_dropout(idx.gated_forward(y, W), 0.1, 3)
    dx, dW, _ = idx.gated_backward(y, W, dh)
    return (out, dW) + smc_layer_norm_backward(x, gamma, dx)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = step()
g.replay()
torch.cuda.synchronize()
eager = step()
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
assert idx.status() == 0
print("same")
""".format(root=here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_gated_wanted_gradients_only_and_rows_behind():
    """Gradients that are not asked for are not touched, and nothing behind the
    last row or column is written."""
    n, c, h = 200, 40, 72
    with _index(n) as idx:
        x, W, b, dh = _gated_inputs(n, c, h, "bf16", seed=90)
        full = idx.gated_backward(x, W, dh, b)
        for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)):
            bufs = [torch.full((v.numel() + 64,), 7.0, dtype=v.dtype, device=DEV) for v in full]
            outs = [buf[:v.numel()].view(v.shape) if w else None
                    for buf, v, w in zip(bufs, full, want)]
            binding.smc_gated_backward(idx.handle, x, W, dh, *outs, c, h, b)
            torch.cuda.synchronize()
            for buf, out, v in zip(bufs, outs, full):
                assert (buf[v.numel():] == 7).all()
                assert torch.equal(out, v) if out is not None else (buf == 7).all()
        buf = torch.full((n * h + 64,), 7.0, dtype=x.dtype, device=DEV)
        idx.gated_forward(x, W, b, out=buf[:n * h].view(n, h))
        torch.cuda.synchronize()
        assert (buf[n * h:] == 7).all()


def test_gated_no_rows():
    with SubMIndex(torch.zeros((0, 4), dtype=torch.int32, device=DEV)) as idx:
        x, W, b, dh = _gated_inputs(0, 64, 128, "f16")
        assert idx.gated_forward(x, W, b).shape == (0, 128)
        dx, dW, db = idx.gated_backward(x, W, dh, b)
        assert dx.shape == (0, 64) and not dW.any() and not db.any()


def test_gated_refusals():
    with _index(16) as idx:
        x, W, b, dh = _gated_inputs(16, 64, 128, "f16")
        with pytest.raises(ValueError):
            idx.gated_forward(x[:8], W)  # not this index's rows
        with pytest.raises(ValueError):
            binding.smc_gated_forward(idx.handle, x[:8], W, dh, 64, 128)
        with pytest.raises(ValueError):
            idx.gated_forward(x, W[:, :32].contiguous())
        with pytest.raises(ValueError):
            idx.gated_forward(x, W.transpose(1, 2))
        with pytest.raises(ValueError):
            idx.gated_forward(x, W.float())
        with pytest.raises(ValueError):
            idx.gated_forward(x, W, b[0])
        with pytest.raises(KeyError):
            idx.gated_forward(x, W, activation="tanh")
        with pytest.raises(ValueError):
            idx.gated_backward(x, W, dh[:, :64].contiguous())
        L, bytes_ = binding.lib(), ctypes.c_int64()
        p = [t.data_ptr() for t in (x, W, b, dh)]
        out = torch.empty_like(dh)

        def call(act=2, cin=64, hidden=128, dtype=1, o=out.data_ptr(), w=None, size=0):
            return L.smc_gated_forward(idx.handle, p[0], p[1], p[2], o, cin, hidden, dtype, act, w,
                                       size, None)

        assert call(act=4) == -1 and call(act=-1) == -1 and call(cin=0) == -1
        assert call(hidden=70000) == -1 and call(dtype=3) == -1 and call(o=None) == -1
        assert call(o=p[0]) == -1 and call(o=out.data_ptr() + 2) == -1
        assert L.smc_gated_workspace(idx.handle, 64, 128, 1, 1, ctypes.byref(bytes_)) == 0
        assert bytes_.value > 0
        work = torch.empty(bytes_.value, dtype=torch.uint8, device=DEV)
        dx = torch.empty_like(x)

        def back(i=dx.data_ptr(), w=work.data_ptr(), size=bytes_.value):
            return L.smc_gated_backward(idx.handle, p[0], p[1], p[2], p[3], i, None, None, 64, 128, 1,
                                        2, w, size, None)

        assert back(size=bytes_.value - 1) == -1 and back(w=None) == -1 and back(i=p[0]) == -1
        assert back(w=work.data_ptr() + 8) == -1 and back(i=work.data_ptr()) == -1
        assert back() == 0
        torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 8), (5, 13), (17, 64), (33, 515)], ids=str)
def test_dropout(shape, dt):
    dtype = rc.DTYPES[dt]
    x, res = _randn(*shape, seed=1, dtype=dtype), _randn(*shape, seed=2, dtype=dtype)
    for p, seed, offset in ((0.1, 5, 0), (0.5, (1 << 64) - 3, (1 << 63) + 9), (0.0, 7, 1),
                            (1.0, 7, 1), (1e-6, 9, 2), (0.999, 9, 2)):
        for r in (None, res):
            got = smc_dropout(x, p, seed, offset, residual=r)
            ref = rc.dropout(x, p, seed, offset, r)
            size = ref.abs() if r is None else ref.abs() + r.abs().double().cpu()
            # the scale and the product, or the product and the sum, in fp32
            rc.assert_close(got, ref, rc.rounding(ref, dtype) + 4 * rc.E32 * size,
                            f"{shape} {dt} p={p}")
            if r is None:
                keep = rc.keep_bits(0, x.numel(), seed, offset).view(shape) >= round(p * 65536)
                assert torch.equal(got.cpu() != 0, keep & (x.cpu() != 0))


def test_dropout_far_elements():
    """Counters of elements past 2^31 come from 64-bit indices (an fp16 array
    of 4.3 GB); checked around multiples of 2^31 elements."""
    n = (1 << 31) + 4099
    x = torch.ones(n, dtype=torch.float16, device=DEV)
    got = smc_dropout(x, 0.5, 3, 4, out=x)
    for first in (0, (1 << 31) - 24, n - 4099, n - 24):
        want = rc.keep_bits(first, 24, 3, 4) >= 32768
        assert torch.equal(got[first:first + 24].cpu() == 2, want)
    assert abs(float((got != 0).sum()) / n - 0.5) < 1e-4  # 5 standard deviations are 5.4e-5


def test_dropout_backward_draws_the_same_mask():
    x, g = _randn(100, 77, seed=3), _randn(100, 77, seed=4)
    y, dx = smc_dropout(x, 0.3, 11, 5), smc_dropout(g, 0.3, 11, 5)
    assert torch.equal(y == 0, dx == 0)
    other = smc_dropout(g, 0.3, 11, 6)
    assert not torch.equal(other == 0, dx == 0)
    # the same values in another type: the same mask
    assert torch.equal(smc_dropout(g.half(), 0.3, 11, 5) == 0, (dx == 0) | (g.half() == 0))


def test_dropout_drops_nan_and_infinity():
    x = torch.full((64, 64), float("nan"), device=DEV)
    x[::2] = float("inf")
    got = smc_dropout(x, 0.5, 21, 0)
    keep = (rc.keep_bits(0, x.numel(), 21, 0) >= 32768).view(64, 64).to(DEV)
    assert (got[~keep] == 0).all() and not torch.isfinite(got[keep]).any()


def test_dropout_in_place_empty_and_state():
    x, r = _randn(50, 33, seed=5), _randn(50, 33, seed=6)
    want = smc_dropout(x, 0.2, 31, 40, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(smc_dropout(a, 0.2, 31, 40, residual=r, out=a), want)
    assert torch.equal(smc_dropout(x, 0.2, 31, 40, residual=b, out=b), want)
    assert smc_dropout(x[:0], 0.2, 31).shape == (0, 33)
    state = torch.tensor([31, 38], dtype=torch.int64, device=DEV)
    assert torch.equal(smc_dropout(x, 0.2, 0, 2, residual=r, state=state), want)
    with pytest.raises(binding.SmcError):
        smc_dropout(x, 1.5, 0)
    with pytest.raises(ValueError):
        smc_dropout(x, 0.5, 0, residual=r.half())
    with pytest.raises(ValueError):
        smc_dropout(x, 0.5, 0, state=state[:1])


# ---------------------------------------------------------------------------
# together, on streams, in graphs
# ---------------------------------------------------------------------------
def _block(idx, x, p, seed, stream_offset=0, state=None):
    """A pre-norm feed-forward block as a user writes it, and its backward."""
    gamma, beta, W, b, W2, dy = p
    y = smc_layer_norm(x, gamma, beta)
    h = idx.gated_forward(y, W, b)
    f = idx.forward(h, W2, K=1)
    out = smc_dropout(f, 0.1, seed, stream_offset, residual=x, state=state)
    df = smc_dropout(dy, 0.1, seed, stream_offset, state=state)
    dh = idx.backward_input(df, W2, K=1)
    dW2 = idx.backward_weight(h, df, K=1)
    dyn, dW, db = idx.gated_backward(y, W, dh, b)
    dx, dgamma, dbeta = smc_layer_norm_backward(x, gamma, dyn)
    return out, dx + dy, dgamma, dbeta, dW, db, dW2


def _block_params(n, c, h, dtype):
    return (1 + _randn(c, seed=1, scale=0.2), _randn(c, seed=2, scale=0.2),
            _randn(2, c, h, seed=3, dtype=dtype, scale=c ** -0.5),
            _randn(2, h, seed=4, dtype=dtype, scale=0.1),
            _randn(1, h, c, seed=5, dtype=dtype, scale=h ** -0.5), _randn(n, c, seed=6, dtype=dtype))


def test_block_of_them_together():
    """norm -> gated -> 1x1x1 convolution -> dropout + residual, forward and
    backward in fp32, against float64 autograd of the whole block with the same
    mask.  The bound is that of a chain of fp32 operators: sums of at most 2n =
    800 terms at 2^-24 each, five deep, relative to each result's norm."""
    n, c, h = 400, 48, 136
    x, p = _randn(n, c, seed=0), _block_params(n, c, h, torch.float32)
    with _index(n) as idx:
        got = _block(idx, x, p, 77)
        assert idx.status() == 0
    leaves = [v.double().cpu().requires_grad_() for v in (x,) + p[:5]]
    xd, gamma, beta, W, b, W2 = leaves
    y = rc.norm(xd, gamma, beta, 1e-5)
    hid = torch.nn.functional.silu(y @ W[0] + b[0]) * (y @ W[1] + b[1])
    t = round(0.1 * 65536)
    keep = (rc.keep_bits(0, n * c, 77, 0).view(n, c) >= t).double() * (65536 / (65536 - t))
    out = xd + keep * (hid @ W2[0])
    grads = torch.autograd.grad(out, leaves, p[5].double().cpu())
    want = (out.detach(), grads[0], grads[1], grads[2], grads[3], grads[4], grads[5])
    for a, r in zip(got, want):
        assert float((a.double().cpu() - r).norm() / r.norm()) <= 5 * 800 * rc.E32


def test_block_on_two_streams_and_in_graphs():
    """The block of 16-bit rows: eagerly, on two streams at once, and captured
    twice (two graphs, replayed together) gives the same bits each time."""
    n, c, h = 1500, 64, 192
    dt = torch.bfloat16
    p = _block_params(n, c, h, dt)
    xs = [_randn(n, c, seed=30 + k, dtype=dt) for k in range(2)]
    idx = [_index(n) for _ in range(2)]  # the convolution's backward keeps its workspace per index
    want = [_block(i, x, p, 5) for i, x in zip(idx, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i, x, s in zip(idx, xs, streams):
            with torch.cuda.stream(s):
                got.append(_block(i, x, p, 5))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    state = torch.tensor([5, 0], dtype=torch.int64, device=DEV)
    graphs, outs = [], []
    for i, x in zip(idx, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_block(i, x, p, 0, state=state))
        graphs.append(g)
    for step in range(3):
        state.copy_(torch.tensor([5, step], dtype=torch.int64))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i, x, o in zip(idx, xs, outs):
            assert all(torch.equal(u, v) for u, v in zip(o, _block(i, x, p, 5, step)))
    assert all(i.status() == 0 for i in idx)
    del graphs
    for i in idx:
        i.close()


def test_explicit_stream():
    """A stream argument: work, results and workspaces on that stream, with the
    inputs' memory kept until it has run."""
    s = torch.cuda.Stream()
    x, gamma, beta, dy = _norm_inputs(5000, 256, torch.float16, seed=41)
    want = smc_layer_norm(x, gamma, beta)
    wdx, wdg, wdb = smc_layer_norm_backward(x, gamma, dy)
    drop = smc_dropout(x, 0.4, 1, residual=dy)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        tmp = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        got = smc_layer_norm(tmp, gamma, beta, stream=s)
        del tmp
        trash = torch.full_like(x, 9.0)  # would reuse tmp's memory
        dx, dg, db = smc_layer_norm_backward(x, gamma, dy, stream=s)
        d = smc_dropout(x, 0.4, 1, residual=dy, stream=s)
        s.synchronize()
        assert torch.equal(got, want) and torch.equal(dx, wdx) and torch.equal(dg, wdg)
        assert torch.equal(db, wdb) and torch.equal(d, drop)
        del trash
    with _index(3000) as idx:
        x, W, b, dh = _gated_inputs(3000, 100, 192, "f32", seed=140)
        want = (idx.gated_forward(x, W, b),) + idx.gated_backward(x, W, dh, b)
        got = [torch.empty_like(v) for v in want]
        s.wait_stream(torch.cuda.current_stream())
        binding.smc_gated_forward(idx.handle, x, W, got[0], 100, 192, b, stream=s)
        binding.smc_gated_backward(idx.handle, x, W, dh, *got[1:], 100, 192, b, stream=s)
        s.synchronize()
        assert all(torch.equal(a, v) for a, v in zip(got, want))
