"""Row operators on the GPU where rounding, range or sheer size could spoil them:
sums of one sign over many rows, the tails of the activations, NaN and overflow,
rows of extreme spread, and sums over many rows whose results are exact."""
import pytest
import torch

from submanifold_sparse_convolution_coord_b200 import binding
from submanifold_sparse_convolution_coord_b200.binding import (SubMIndex, smc_layer_norm,
                                                               smc_layer_norm_backward)

import rows_common as rc

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _rand(*shape, seed=0, lo=0.0, hi=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lo + (hi - lo) * torch.rand(*shape, generator=g, device=DEV)


def _randn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _signs(*shape, seed=0, dtype=torch.float32):
    """-1, 0 and 1."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device=DEV, dtype=torch.int8).to(dtype)


def _index(n):
    i = torch.arange(n, device=DEV)
    c = torch.stack([i // 2 ** 18, i // 4096 % 64, i // 64 % 64, i % 64], 1)
    return SubMIndex(c.to(torch.int32))


def _unit_gate(c, h, dtype):
    """W and bias of a bilinear gate with both pre-activations 1: dg = du = dh."""
    return torch.zeros(2, c, h, dtype=dtype, device=DEV), torch.ones(2, h, dtype=dtype, device=DEV)


def _one_sign_allowance(pieces):
    """A piece of a sum is 256 steps of the matrix unit, each cutting at most twice
    2^-23 of a sum that grows evenly (half of its final size on average); the
    pieces are added up with 2^-24 each.  Roundings of results to their type have
    means of their own below 1e-6 (fp16) and 1e-5 (bf16)."""
    return 256 * 2.0 ** -23 + pieces * rc.E32


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gated_weight_gradient_of_one_sign(dt):
    """All terms of the weight gradient positive, and enough tiles (80 for 74
    pairs of SMs) that one accumulation takes all 200,000 rows.  The matrix unit
    cuts its sums, so a loss has one sign and shows in the mean relative error."""
    n, c, h, dtype = 200_000, 1024, 2368, rc.DTYPES[dt]
    x = (_rand(n, c, seed=1, lo=0.5, hi=1.5) * _rand(c, seed=2, lo=1, hi=2)).to(dtype)
    dh = (_rand(n, h, seed=3, lo=0.5, hi=1.5) * _rand(h, seed=4, lo=1, hi=2) / 16).to(dtype)
    W, b = _unit_gate(c, h, dtype)
    dW = torch.empty_like(W)
    with _index(n) as idx:
        binding.smc_gated_backward(idx.handle, x, W, dh, None, dW, None, c, h, b, "none")
        assert idx.status() == 0
    allowed = _one_sign_allowance(n / 4096)
    xd = x.double().t()
    for at in range(0, h, 592):
        ref = xd @ dh[:, at:at + 592].double()
        for half in range(2):
            rel = dW[half, :, at:at + 592].double() / ref - 1
            assert abs(float(rel.mean())) <= allowed + 1e-5, (half, at, float(rel.mean()))
            assert float(rel.abs().max()) <= rc.UNIT[dtype] + 2 * allowed


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gated_input_gradient_of_one_sign(dt):
    """The same for the input gradient's sum over 2 x 65,536 hidden units.  x = 0
    leaves both pre-activations at 1 whatever the weights."""
    n, c, h, dtype = 300, 264, 65536, rc.DTYPES[dt]
    x = torch.zeros(n, c, dtype=dtype, device=DEV)
    W = (_rand(2, c, h, seed=1, lo=0.5, hi=1.5) * _rand(c, 1, seed=2, lo=1, hi=2) / 16).to(dtype)
    dh = (_rand(n, h, seed=3, lo=0.5, hi=1.5) * _rand(n, 1, seed=4, lo=1, hi=2)).to(dtype)
    b = torch.ones(2, h, dtype=dtype, device=DEV)
    dx = torch.empty_like(x)
    with _index(n) as idx:
        binding.smc_gated_backward(idx.handle, x, W, dh, dx, None, None, c, h, b, "none")
        assert idx.status() == 0
    ref = dh.double() @ (W[0].double() + W[1].double()).t()
    rel = dx.double() / ref - 1
    allowed = _one_sign_allowance(2 * h / 4096)
    assert abs(float(rel.mean())) <= allowed + 1e-5
    assert float(rel.abs().max()) <= rc.UNIT[dtype] + 2 * allowed


@pytest.mark.parametrize("n", [300, 60_000])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gated_products_of_one_sign(dt, n):
    """The same for the pre-activations' sums over 65,536 channels, and for dg and
    du, which are computed from them again (up = 1, so out is the gate, du = dh g)."""
    c, h, dtype = 65536 if n == 300 else 8200, 72, rc.DTYPES[dt]
    x = (_rand(n, c, seed=1, lo=0.5, hi=1.5) * _rand(n, 1, seed=2, lo=1, hi=2)).to(dtype)
    W = (_rand(2, c, h, seed=3, lo=0.5, hi=1.5) * _rand(h, seed=4, lo=1, hi=2) / 16).to(dtype)
    W[1] = 0
    b = torch.ones(2, h, dtype=dtype, device=DEV)
    scale = 2.0 ** -7 if n == 300 else 2.0 ** -15  # the bias gradient stays in fp16's range
    dh = torch.full((n, h), scale, dtype=dtype, device=DEV)
    b[0] = 0
    db = torch.empty_like(b)
    with _index(n) as idx:
        out = idx.gated_forward(x, W, b, "none")
        binding.smc_gated_backward(idx.handle, x, W, dh, None, None, db, c, h, b, "none")
        assert idx.status() == 0
    ref = torch.cat([x[r:r + 5000].double() @ W[0].double() for r in range(0, n, 5000)])
    rel = out.double() / ref - 1
    allowed = _one_sign_allowance(c / 4096)
    assert abs(float(rel.mean())) <= allowed + 1e-5
    assert float(rel.abs().max()) <= rc.UNIT[dtype] + 2 * allowed
    # the bias gradient: 32 rows by five steps, then at most 59 sums a warp, and 32 warps
    rel = db[1].double() / (ref * scale).sum(0) - 1
    assert float(rel.abs().max()) <= rc.UNIT[dtype] + 2 * allowed + 100 * rc.E32


def _one_row(gate, dt, act):
    """The gated product of one row whose pre-activations are `gate` and 1, and
    the gradient by the gate for dh = 1: the activation's value and slope."""
    dtype = rc.DTYPES[dt]
    gate = torch.tensor(gate, dtype=torch.float64).to(dtype).to(DEV)
    h = gate.numel()
    x, W = torch.zeros(1, 8, dtype=dtype, device=DEV), torch.zeros(2, 8, h, dtype=dtype, device=DEV)
    b, dh = torch.stack([gate, torch.ones_like(gate)]), torch.ones(1, h, dtype=dtype, device=DEV)
    with _index(1) as idx:
        out = idx.gated_forward(x, W, b, act)
        _, _, db = idx.gated_backward(x, W, dh, b, act)
    return gate.double().cpu(), out[0], db[0]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_silu_far_out(dt):
    """SiLU's slope is s + v s (1 - s) with 1 - s small for large v; both terms
    carry some roundings of 2^-24, and an exponential of v < 0 the error of its
    argument, |v| 2^-23.  Below -87 the kernel's exponential passes the range of
    fp32 and the sigmoid is 0."""
    big = [20, 50, 88, 100, 1e3, 3e4, 6e4]
    if dt != "f16":
        big += [1e5, 1e6, 3e7, 1e9, 1e20, 3e38]
    gate = [s * v for v in big + [0, 0.5, 1, 2, 5, 10, 15] for s in (1, -1)]
    v, out, slope = _one_row(gate, dt, "silu")
    s, t = torch.sigmoid(v), torch.sigmoid(-v)
    rel = (8 + 2 * (-v).clamp(0, 100)) * 2.0 ** -23
    rc.assert_close(out, v * s, rc.rounding(v * s, out.dtype) + rel * (v * s).abs() + 1e-35, "value")
    want = s + v * s * t
    rc.assert_close(slope, want, rc.rounding(want, out.dtype) + rel * (s + v.abs() * s * t) + 1e-35,
                    "slope")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_gelu_tails(dt):
    """GELU's value v cdf(v) and slope cdf(v) + v pdf(v), relative to the terms
    themselves on both sides: 8 roundings of 2^-23 each around the exponential,
    whose argument v^2 / 2 carries two roundings (v^2 2^-23 relative)."""
    gate = [x / 16 for x in range(-12 * 16, 8 * 16 + 1)]
    v, out, slope = _one_row(gate, dt, "gelu")
    cdf = 0.5 * torch.erfc(-v / 2 ** 0.5)
    pdf = torch.exp(-0.5 * v * v) / (2 * torch.pi) ** 0.5
    rel = (8 + v * v) * 2.0 ** -23
    rc.assert_close(out, v * cdf, rc.rounding(v * cdf, out.dtype) + rel * (v * cdf).abs(), "value")
    want = cdf + v * pdf
    rc.assert_close(slope, want, rc.rounding(want, out.dtype) + rel * (cdf + v.abs() * pdf), "slope")


@pytest.mark.parametrize("act", rc.ACTS)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_gated_nan_of_the_weights_shows(dt, act):
    """A NaN in the gate's weights or bias alone reaches every row of its hidden
    unit and, through it, every input gradient; other units stay clean.  Without an
    activation the gate's own gradient, grad_out times up, does not hold the gate."""
    n, c, h, dtype = 300, 72, 136, rc.DTYPES[dt]
    x, dh = _randn(n, c, seed=1, dtype=dtype), _randn(n, h, seed=2, dtype=dtype)
    W, b = _randn(2, c, h, seed=3, dtype=dtype), _randn(2, h, seed=4, dtype=dtype)
    with _index(n) as idx:
        clean, clean_grads = idx.gated_forward(x, W, b, act), idx.gated_backward(x, W, dh, b, act)
        W[0, 5, 17] = float("nan")
        b[0, 100] = float("nan")
        out = idx.gated_forward(x, W, b, act)
        dx, dW, db = idx.gated_backward(x, W, dh, b, act)
    units = [17, 100]
    rest = [u for u in range(h) if u not in units]
    assert out[:, units].isnan().all() and torch.equal(out[:, rest], clean[:, rest])
    assert dx.isnan().all()
    first = 1 if act == "none" else 0
    assert dW[first:, :, units].isnan().all() and db[first:, units].isnan().all()
    assert torch.equal(dW[:, :, rest], clean_grads[1][:, :, rest])
    assert torch.equal(db[:, rest], clean_grads[2][:, rest])
    assert torch.equal(dW[:first], clean_grads[1][:first])


@pytest.mark.parametrize("c", [64, 96, 515, 1024, 1200, 4099])
@pytest.mark.parametrize("spread,size", [(1e-18, 1e4), (1e-16, 1e8), (1e17, 1e-6), (1e15, 1.0)])
def test_norm_backward_of_extreme_spread(c, spread, size):
    """Without eps the result scales with size / spread: what is computed on the
    way stays in range.  Bound: as many roundings as the sums have, relative to
    the row's largest term."""
    x, dy = _randn(20, c, seed=1), _randn(20, c, seed=2) * size
    x = x * spread
    gamma = _randn(c, seed=3)
    dx, dgamma, _ = smc_layer_norm_backward(x, gamma, dy, 0.0)
    ref, rgamma, _ = rc.norm_grads(x, gamma, dy, 0.0)
    bound = 400 * rc.E32 * ref.abs().amax(1, keepdim=True) + 1e-36
    rc.assert_close(dx, ref, bound.expand_as(ref), "grad_in")
    rc.assert_close(dgamma, rgamma, 400 * rc.E32 * rgamma.abs().max().expand_as(rgamma), "grad_gamma")


@pytest.mark.parametrize("c", [49, 64, 98, 515, 784, 1024, 1200, 4099])
def test_norm_of_constant_rows_is_beta(c):
    """Rows whose values are all alike, and whose sum fp32 holds exactly: the mean
    is that value exactly, so the result is beta and xhat is 0."""
    for dt in ("f32", "f16", "bf16"):
        dtype = rc.DTYPES[dt]
        x = torch.tensor([2.5, 100, -7, 1000, -0.375, 3, 48, 2000], device=DEV).to(dtype)
        x = x[:, None].expand(8, c).contiguous()
        gamma, beta, dy = _randn(c, seed=1), _randn(c, seed=2), _randn(8, c, seed=3, dtype=dtype)
        y = smc_layer_norm(x, gamma, beta, 1e-5)
        assert torch.equal(y, beta.to(dtype).expand(8, c))
        dx, dgamma, dbeta = smc_layer_norm_backward(x, gamma, dy, 1e-5)
        assert not dgamma.any()
        g = dy.double() * gamma.double()
        want = (g - g.mean(1, keepdim=True)) * 1e-5 ** -0.5
        size = (g.abs() + g.abs().mean(1, keepdim=True)) * 1e-5 ** -0.5
        rc.assert_close(dx, want, rc.rounding(want, dtype) + 80 * rc.E32 * size)


def test_norm_backward_of_very_many_long_rows():
    """More rows than 65,535 times the 256 of a partial sum, of a length that the
    kernels read again from cache (69 GB of rows and as much of gradients).
    All ones: grad_beta is the number of rows, xhat is 0."""
    n, c = 65_535 * 256 + 300, 2049
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 4 * n * c + 6 * 2 ** 30:
        pytest.skip("needs 143 GB of free memory")
    x = torch.ones(n, c, dtype=torch.bfloat16, device=DEV)
    dx, dgamma, dbeta = smc_layer_norm_backward(x, torch.ones(c, device=DEV), x)
    # sums of 256 ones are exact, and so are those of every 32nd of them; the 32
    # sums of 2^19 or so add up to more than 2^24: half a step each
    assert float((dbeta.double() - n).abs().max()) <= 32 and not dgamma.any()
    assert not dx[:100].any() and not dx[n - 100:].any()
    del x, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_norm_of_every_length(dt):
    """Each number of channels up to the longest rows of registers and some beyond
    has a kernel; every 7th length is checked against float64."""
    dtype = rc.DTYPES[dt]
    n, most = 3, 4200
    x = (_randn(n * most, seed=1) * 2 + 1).to(dtype)
    dy = _randn(n * most, seed=2, dtype=dtype)
    gamma, beta = _randn(most, seed=3), _randn(most, seed=4)
    for c in range(1, most + 1):
        a, d = x[:n * c].view(n, c), dy[:n * c].view(n, c)
        g, b = gamma[:c], beta[:c]
        y = smc_layer_norm(a, g, b, 1e-3)
        grads = smc_layer_norm_backward(a, g, d, 1e-3)
        if c % 7 != 1 and c > 40:
            continue
        rc.assert_close(y, rc.norm(a, g, b, 1e-3), rc.norm_bound(a, g, b, 1e-3, dtype), f"{c}")
        for u, r, e in zip(grads, rc.norm_grads(a, g, d, 1e-3),
                           rc.norm_grads_bound(a, g, d, 1e-3, dtype)):
            rc.assert_close(u, r, e, f"{c} gradients")


def test_norm_backward_beta_without_gamma():
    """A norm with beta alone has a gradient for it."""
    x, dy = _randn(50, 96, seed=1), _randn(50, 96, seed=2)
    plain = smc_layer_norm_backward(x, None, dy)
    assert plain[1] is None and plain[2] is None
    dx, dgamma, dbeta = smc_layer_norm_backward(x, None, dy, param_grads=True)
    want = smc_layer_norm_backward(x, torch.ones(96, device=DEV), dy)
    assert torch.equal(dx, plain[0]) and torch.equal(dx, want[0])
    assert torch.equal(dgamma, want[1]) and torch.equal(dbeta, want[2])
    dx, dgamma, dbeta = smc_layer_norm_backward(x, torch.ones(96, device=DEV), dy, param_grads=False)
    assert torch.equal(dx, want[0]) and dgamma is None and dbeta is None


def _exact(a, b):
    """a^T b of small whole numbers, exact in float64, in pieces of the rows."""
    return sum(a[r:r + 200_000].double().t() @ b[r:r + 200_000].double()
               for r in range(0, a.shape[0], 200_000))


@pytest.mark.parametrize("n,c,h", [(30_001, 128, 200), (1_100_000, 16, 2048), (150_001, 264, 600)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_gated_sums_over_rows_are_exact(dt, n, c, h):
    """Whole numbers whose sums fp32 holds exactly, whatever the order: grad_W and
    grad_bias equal the sums rounded once.  A share of the rows that is lost,
    taken twice or put into the wrong tile changes most entries."""
    dtype = rc.DTYPES[dt]
    x, dh = _signs(n, c, seed=5, dtype=dtype), _signs(n, h, seed=6, dtype=dtype)
    W, b = _unit_gate(c, h, dtype)
    with _index(n) as idx:
        _, dW, db = idx.gated_backward(x, W, dh, b, "none")
        assert idx.status() == 0
    want, sums = _exact(x, dh).to(dtype), dh.double().sum(0).to(dtype)
    for half in range(2):
        assert torch.equal(dW[half], want) and torch.equal(db[half], sums)
    # the rows of a sixty-fourth of the sum would show nearly everywhere
    part = _exact(x[:n // 64], dh[:n // 64])
    assert float(((want.double() - part).to(dtype) != want).float().mean()) > 0.9


@pytest.mark.parametrize("n,c,dt", [(700_001, 16, "bf16"), (700_001, 16, "f32"), (50_001, 515, "f32"),
                                    (60_001, 1200, "f16"), (20_001, 4099, "bf16"),
                                    (33_600_000, 64, "bf16")])
def test_norm_sums_over_rows_are_exact(n, c, dt):
    """grad_beta of whole numbers is exact.  Rows of ones and minus ones around 0
    have xhat = +-r for the same r, so grad_gamma is r times a whole number."""
    dtype = rc.DTYPES[dt]
    dy = _signs(n, c, seed=7, dtype=dtype)
    x = torch.ones(c, dtype=dtype, device=DEV)
    x[1::2] = -1
    x[(c // 2) * 2:] = 0  # an odd channel
    x = x.expand(n, c).contiguous()
    x[n // 3:n // 2] *= -1
    var = (c // 2) * 2 / c
    _, dgamma, dbeta = smc_layer_norm_backward(x, torch.ones(c, device=DEV), dy, 0.5)
    want = torch.zeros(c, dtype=torch.float64, device=DEV)
    products = want.clone()
    for r in range(0, n, 1_000_000):
        d = dy[r:r + 1_000_000].double()
        want += d.sum(0)
        products += (d * x[r:r + 1_000_000].double()).sum(0)
    assert torch.equal(dbeta.double(), want)
    products *= (var + 0.5) ** -0.5
    # r: the variance, the sum with eps and the inverse root, each the same in every
    # row; then a random walk of n steps of r stays below 3 sqrt(n) r, and its n
    # roundings, of random sign, add up to at most 3 sqrt(n) times 2^-24 of that
    bound = 8 * rc.E32 * products.abs() + 9 * n * rc.E32 * (var + 0.5) ** -0.5
    rc.assert_close(dgamma, products, bound, "dgamma")
    assert float((products.abs() > 4 * bound).float().mean()) > 0.9


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_gated_bad_inputs_reach_the_weight_gradient(dt):
    """A NaN in channel k of the input spoils its row's dg and du, so all of
    grad_W and grad_bias; one in grad_out spoils its unit's column only."""
    n, c, h, dtype = 300, 72, 136, rc.DTYPES[dt]
    x, dh = _randn(n, c, seed=1, dtype=dtype), _randn(n, h, seed=2, dtype=dtype)
    W, b = _randn(2, c, h, seed=3, dtype=dtype), _randn(2, h, seed=4, dtype=dtype)
    with _index(n) as idx:
        clean = idx.gated_backward(x, W, dh, b)
        bad = x.clone()
        bad[5, 3] = float("nan")
        _, dW, db = idx.gated_backward(bad, W, dh, b)
        assert dW.isnan().all() and db.isnan().all()
        bad = dh.clone()
        bad[299, 7] = float("nan")
        dx, dW, db = idx.gated_backward(x, W, bad, b)
    rest = [u for u in range(h) if u != 7]
    assert dx[299].isnan().all() and torch.equal(dx[:299], clean[0][:299])
    assert dW[:, :, 7].isnan().all() and torch.equal(dW[:, :, rest], clean[1][:, :, rest])
    assert db[:, 7].isnan().all() and torch.equal(db[:, rest], clean[2][:, rest])


def test_captured_after_other_work():
    """A chain whose kernels are placed early may follow anything in a captured
    graph: a memory copy, a memset, a join of two streams, nothing at all."""
    n, c, h = 500, 100, 64
    x, W = _randn(n, c, seed=1, dtype=torch.float16), _randn(2, c, h, seed=2, dtype=torch.float16)
    dh, gamma = _randn(n, h, seed=3, dtype=torch.float16), torch.ones(c, device=DEV)
    with _index(n) as idx, SubMIndex(torch.zeros(0, 4, dtype=torch.int32, device=DEV)) as none:
        want = idx.gated_forward(x, W)
        grads = idx.gated_backward(x, W, dh)[:2]
        torch.cuda.synchronize()
        buf, zeros = torch.zeros_like(x), torch.ones_like(x)
        side = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            first = smc_layer_norm_backward(x[:0], gamma, x[:0])  # the join alone
            buf.copy_(x)
            a = idx.gated_forward(buf, W)
            zeros.zero_()
            b = idx.gated_backward(buf, W, dh)[:2]
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                d = smc_layer_norm(x, gamma)
            e = smc_layer_norm(x, gamma)
            torch.cuda.current_stream().wait_stream(side)
            f = idx.gated_forward(buf, W)
        for _ in range(3):
            for t in (buf, a, *b, d, e, f, first[1]):
                t.fill_(3)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(a, want) and torch.equal(f, want) and torch.equal(d, e)
            assert all(torch.equal(u, v) for u, v in zip(b, grads)) and not first[1].any()
        assert idx.status() == 0 and none.status() == 0
        del g


def test_gated_fp16_gradient_out_of_range():
    """dg and du are fp16 between the products: a dg beyond 65,504 is infinite
    and shows in its row's and its unit's gradients, and in no others; the same
    gradient scaled down by 2^-8 is right (what loss scaling does)."""
    n, c, h = 200, 64, 96
    x, W = _randn(n, c, seed=1, dtype=torch.float16), _randn(2, c, h, seed=2) / 8
    W, b = W.half(), _randn(2, h, seed=3, dtype=torch.float16)
    dh = _randn(n, h, seed=4, dtype=torch.float16)
    b[:, 11] = 100.0  # u = 100 or so, its gate's slope 1
    dh[20, 11] = 3000.0
    with _index(n) as idx:
        dx, dW, db = idx.gated_backward(x, W, dh, b)
        small = (dh.float() / 256).half()
        got = idx.gated_backward(x, W, small, b)
    rows, units = [r for r in range(n) if r != 20], [u for u in range(h) if u != 11]
    assert not torch.isfinite(dx[20]).any() and torch.isfinite(dx[rows]).all()
    assert not torch.isfinite(dW[:, :, 11]).any() and torch.isfinite(dW[:, :, units]).all()
    assert torch.isinf(db[:, 11]).all() and torch.isfinite(db[:, units]).all()
    ref = rc.Gated(x, W, b, "silu", small)
    for a, r, bound in zip(got, (ref.dx, ref.dW, ref.db), (ref.dx_bound, ref.dW_bound, ref.db_bound)):
        rc.assert_close(a, r, bound)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,h", [(5, 65536, 3), (5, 3, 65536), (300, 4160, 8), (70, 4104, 2056)])
def test_gated_longest_sides(dt, n, c, h):
    """The widest rows and hidden layers there may be, and sums just over a piece,
    against float64 under the bounds of the ordinary shapes."""
    dtype = rc.DTYPES[dt]
    x, dh = _randn(n, c, seed=1, dtype=dtype), _randn(n, h, seed=2, dtype=dtype)
    W = (_randn(2, c, h, seed=3) * c ** -0.5).to(dtype)
    b = _randn(2, h, seed=4, dtype=dtype)
    with _index(n) as idx:
        ref = rc.Gated(x, W, b, "gelu", dh)
        rc.assert_close(idx.gated_forward(x, W, b, "gelu"), ref.out, ref.out_bound, "out")
        dx, dW, db = idx.gated_backward(x, W, dh, b, "gelu")
        rc.assert_close(dx, ref.dx, ref.dx_bound, "grad_in")
        rc.assert_close(dW, ref.dW, ref.dW_bound, "grad_W")
        rc.assert_close(db, ref.db, ref.db_bound, "grad_bias")
        assert idx.status() == 0


def test_one_handle_on_two_streams():
    """Calls on one handle from two streams at once, each with its own workspace."""
    n, c, h = 6000, 136, 392
    with _index(n) as idx:
        sets = [(_randn(n, c, seed=k, dtype=torch.bfloat16), _randn(n, h, seed=9 + k, dtype=torch.bfloat16))
                for k in range(2)]
        W, b = _randn(2, c, h, seed=20, dtype=torch.bfloat16), _randn(2, h, seed=21, dtype=torch.bfloat16)

        def step(x, dh):
            return (idx.gated_forward(x, W, b),) + idx.gated_backward(x, W, dh, b)
        want = [step(*s) for s in sets]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [[], []]
        for _ in range(8):
            for k, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[k].append(step(*sets[k]))
        torch.cuda.synchronize()
        for k in range(2):
            for outs in got[k]:
                assert all(torch.equal(a, w) for a, w in zip(outs, want[k]))
        assert idx.status() == 0
