"""Row operators (layer norm, gated feed-forward, dropout), the part that needs
no GPU: refusals of the C ABI and of the binding, which come before any launch,
and pins of the plain float64 implementations the GPU tests compare with."""
import ctypes

import pytest
import torch

from submanifold_sparse_convolution_coord_b200 import binding

import rows_common as rc

BUF = [0x100000 * (i + 1) for i in range(12)]  # addresses that are never read
INVALID, UNSUPPORTED = -1, -6


@pytest.fixture(scope="module")
def L():
    from submanifold_sparse_convolution_coord_b200.csrc import build
    build.build()
    return binding.lib()


def _norm(L, x=BUF[0], gamma=BUF[1], beta=BUF[2], out=BUF[3], n=4, c=64, dtype=1, eps=1e-5):
    return L.smc_layer_norm(x, gamma, beta, out, n, c, dtype, eps, None)


@pytest.mark.parametrize("bad", [
    {"x": None}, {"out": None}, {"x": BUF[0] + 8}, {"out": BUF[3] + 2}, {"gamma": BUF[1] + 4},
    {"beta": BUF[2] + 4}, {"n": -1}, {"c": 0}, {"dtype": 3}, {"dtype": -1}, {"eps": -1.0},
    {"eps": float("nan")}, {"out": BUF[0] + 16}, {"out": BUF[1]},
], ids=str)
def test_norm_refusals(L, bad):
    assert _norm(L, **bad) == INVALID


def test_norm_sizes(L):
    assert _norm(L, n=1 << 31) == UNSUPPORTED
    assert _norm(L, c=1 << 31) == UNSUPPORTED
    assert _norm(L, n=1 << 30, c=1 << 30) == UNSUPPORTED
    assert _norm(L, x=None, out=None, n=0) == 0  # nothing to do


def _norm_bwd(L, x=BUF[0], gamma=BUF[1], dy=BUF[2], dx=BUF[3], dgamma=BUF[4], dbeta=BUF[5], n=4,
              c=64, dtype=1, eps=1e-5, work=BUF[6], size=1 << 19):
    return L.smc_layer_norm_backward(x, gamma, dy, dx, dgamma, dbeta, n, c, dtype, eps, work, size,
                                     None)


@pytest.mark.parametrize("bad", [
    {"x": None}, {"dy": None}, {"dx": None}, {"dgamma": None}, {"dbeta": None},
    {"dy": BUF[2] + 8}, {"dx": BUF[0]}, {"dx": BUF[2]}, {"dgamma": BUF[5]}, {"dgamma": BUF[1]},
    {"work": None}, {"work": BUF[6] + 4}, {"size": 0}, {"work": BUF[3]}, {"n": -1}, {"c": 0},
    {"dtype": 7}, {"eps": float("nan")},
], ids=str)
def test_norm_backward_refusals(L, bad):
    assert _norm_bwd(L, **bad) == INVALID


def test_workspace_queries(L):
    b = ctypes.c_int64(-1)
    assert L.smc_layer_norm_backward_workspace(10, 64, 0, None) == INVALID
    assert L.smc_layer_norm_backward_workspace(-1, 64, 0, ctypes.byref(b)) == INVALID
    assert b.value == 0
    assert L.smc_gated_workspace(None, 64, 64, 1, 0, ctypes.byref(b)) == INVALID
    assert L.smc_gated_workspace(None, 64, 64, 1, 0, None) == INVALID


def test_gated_needs_a_handle(L):
    assert L.smc_gated_forward(None, BUF[0], BUF[1], None, BUF[2], 64, 64, 1, 2, None, 0, None) == \
        INVALID
    assert L.smc_gated_backward(None, BUF[0], BUF[1], None, BUF[2], BUF[3], BUF[4], None, 64, 64, 1,
                                2, BUF[5], 1 << 20, None) == INVALID


def _drop(L, x=BUF[0], residual=BUF[1], out=BUF[2], count=100, dtype=2, p=0.1, seed=1, offset=0,
          state=None):
    return L.smc_dropout(x, residual, out, count, dtype, p, seed, offset, state, None)


@pytest.mark.parametrize("bad", [
    {"x": None}, {"out": None}, {"x": BUF[0] + 2}, {"residual": BUF[1] + 2}, {"out": BUF[2] + 8},
    {"state": BUF[3] + 8}, {"count": -1}, {"count": 1 << 44}, {"dtype": 3}, {"p": -0.1}, {"p": 1.5},
    {"p": float("nan")}, {"out": BUF[0] + 16}, {"out": BUF[1] + 16}, {"state": BUF[2]},
], ids=str)
def test_dropout_refusals(L, bad):
    assert _drop(L, **bad) == INVALID


def test_dropout_of_nothing(L):
    assert _drop(L, x=None, residual=None, out=None, count=0) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        binding.smc_layer_norm(x)
    with pytest.raises(ValueError):
        binding.smc_layer_norm(x.double())
    with pytest.raises(ValueError):
        binding.smc_layer_norm(x[0])
    with pytest.raises(ValueError):
        binding.smc_layer_norm_backward(x, None, x)
    with pytest.raises(ValueError):
        binding.smc_dropout(x, 0.5, 1)
    with pytest.raises(ValueError):
        binding.smc_dropout(x, 0.5, -1)
    with pytest.raises(ValueError):
        binding.smc_dropout(x, 0.5, 1, 1 << 64)


# ---------------------------------------------------------------------------
# pins of the float64 implementations
# ---------------------------------------------------------------------------
def test_philox_known_answers():
    """The generator's published test vectors (zeros, all ones, digits of pi)."""
    assert philox_hex((0, 0, 0, 0), (0, 0)) == "6627e8d5 e169c58d bc57ac4c 9b00dbd8"
    f = 0xFFFFFFFF
    assert philox_hex((f, f, f, f), (f, f)) == "408f276d 41c83b0e a20bc7c6 6d5451fd"
    assert philox_hex((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344),
                      (0xa4093822, 0x299f31d0)) == "d16cfe09 94fdcceb 5001e420 24126ea1"


def philox_hex(c, k):
    return " ".join("%08x" % w for w in rc.philox(c, k))


def test_norm_matches_torch():
    torch.manual_seed(0)
    x = torch.randn(7, 13, dtype=torch.float64, requires_grad=True)
    g = torch.randn(13, dtype=torch.float64, requires_grad=True)
    b = torch.randn(13, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(7, 13, dtype=torch.float64)
    y = torch.nn.functional.layer_norm(x, (13,), g, b, 1e-3)
    assert torch.allclose(rc.norm(x, g, b, 1e-3), y, atol=1e-12)
    for got, want in zip(rc.norm_grads(x.detach(), g.detach(), dy, 1e-3),
                         torch.autograd.grad(y, [x, g, b], dy)):
        assert torch.allclose(got, want, atol=1e-12)


@pytest.mark.parametrize("name", rc.ACTS)
def test_gated_matches_torch(name):
    torch.manual_seed(1)
    f = torch.nn.functional
    x = torch.randn(6, 5, dtype=torch.float64, requires_grad=True)
    W = torch.randn(2, 5, 9, dtype=torch.float64, requires_grad=True)
    b = torch.randn(2, 9, dtype=torch.float64, requires_grad=True)
    dh = torch.randn(6, 9, dtype=torch.float64)
    fn = {"none": lambda v: v, "relu": f.relu, "silu": f.silu, "gelu": f.gelu}[name]
    y = fn(x @ W[0] + b[0]) * (x @ W[1] + b[1])
    want = torch.autograd.grad(y, [x, W, b], dh)
    r = rc.Gated(x.detach().float().double().to(torch.float32).double().float(), W.detach().float(),
                 b.detach().float(), name, dh.float())
    for got, ref in zip((r.out, r.dx, r.dW, r.db), (y,) + want):
        assert torch.allclose(got, ref, atol=1e-4)  # the inputs were rounded to float32


@pytest.mark.parametrize("name", rc.ACTS)
def test_activation_constants(name):
    """The Lipschitz constants the bounds use hold on a fine grid."""
    v = torch.linspace(-12, 12, 200001, dtype=torch.float64)
    a, s = rc.act(name, v)
    h = v[1] - v[0]
    assert s.abs().max() <= rc.LIP[name]
    if name != "relu":
        assert ((s[1:] - s[:-1]).abs() / h).max() <= rc.LIP2[name] + 1e-9
    assert torch.allclose((a[2:] - a[:-2]) / (2 * h), s[1:-1], atol=1e-4) or name == "relu"
