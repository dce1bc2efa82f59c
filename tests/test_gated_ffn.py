"""Dense gated FFN: the oracle's pins (CPU), refusals (CPU) and the kernels
against the fp64 oracle (GPU).

Tolerances.  A product of K terms in fp32 is off by at most K 2^-23 of the sum of its
terms' magnitudes, whatever the order (each addition rounds or truncates by at most
2^-23).  An operand or result in bf16 is off by half a step, 2^-8.  act and act' use
the approximate exp and division: their sigmoid (or normal distribution) factor is
off by less than 2^-20, so they are off by less than (1 + |z|) 2^-18, and (1 + z^2)
2^-18 for the derivative.  The backward is checked from the z and u that the
forward saved.
"""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_tma_b200 import build as tw_build
from activation_sparse_transformer_tma_b200 import twell
from oracle import layer

BF, F32 = torch.bfloat16, torch.float32
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 8
FAKE = 0x10000
H = 2.0 ** -8
ACTS = ["relu", "silu", "gelu", "gelu_tanh"]


# ----------------------------------------------------------------- CPU: pins --
@pytest.mark.parametrize("act", ACTS)
def test_oracle_equals_autograd_and_differences(act):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((5, 6)), rng.standard_normal((5, 6))
    W = [rng.standard_normal((7, 6)) * 0.5 for _ in range(3)]
    z, u, _, y = layer.gated_ffn(x, *W, act)
    g = layer.gated_ffn_backward(x, dy, *W, act, z, u)
    t = [torch.tensor(v, requires_grad=True) for v in (x, *W)]
    f = {"relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act]
    out = (f(t[0] @ t[1].T) * (t[0] @ t[2].T)) @ t[3]
    np.testing.assert_allclose(y, out.detach().numpy(), rtol=1e-10, atol=1e-12)
    (out * torch.tensor(dy)).sum().backward()
    for key, v in zip(("dx", "dWg", "dWu", "dWd"), t):
        np.testing.assert_allclose(g[key], v.grad.numpy(), rtol=1e-9, atol=1e-11)
    e, p = 1e-6, W[0].copy()
    p[2, 3] += e
    up = np.sum(layer.gated_ffn(x, p, W[1], W[2], act)[3] * dy)
    p[2, 3] -= 2 * e
    down = np.sum(layer.gated_ffn(x, p, W[1], W[2], act)[3] * dy)
    assert abs((up - down) / (2 * e) - g["dWg"][2, 3]) < 1e-6


# ------------------------------------------------------------- CPU: refusals --
@pytest.fixture(scope="module")
def L():
    tw_build.build()
    return twell.lib()


def test_refusals(L):
    ws = L.gated_ffn_workspace_size(100, 128, 256)
    bws = L.gated_ffn_backward_workspace_size(100, 128, 256)
    assert ws > 0 and bws >= 3 * 100 * 256 * 2
    assert L.gated_ffn_workspace_size(-1, 128, 256) == 0

    def f(T=100, d=128, F=256, act=1, z=None, u=None, n=ws, yt=1, **over):
        a = dict(x=FAKE, g=FAKE, w=FAKE, dn=FAKE, y=FAKE, ws=FAKE)
        a.update(over)
        return L.gated_ffn_forward(a["x"], a["g"], a["w"], a["dn"], T, d, F, act, z, u, a["y"], yt,
                                   a["ws"], n, None, None)

    assert f(T=-1) == INVALID and f(act=4) == INVALID and f(act=-1) == INVALID
    assert f(d=100) == UNSUPPORTED and f(F=250) == UNSUPPORTED
    assert f(d=56) == UNSUPPORTED and f(F=56) == UNSUPPORTED
    assert f(z=FAKE) == INVALID                              # z without u
    assert f(yt=9) == INVALID
    for k in ("x", "g", "w", "dn", "y", "ws"):
        assert f(**{k: None}) == INVALID, k
        assert f(**{k: FAKE + 8}) == ALIGN, k
    assert f(n=ws - 1) == WORKSPACE
    assert f(T=0, x=None, y=None, ws=None, n=0) == OK

    def b(T=100, d=128, F=256, act=1, n=bws, xt=1, wt=0, **over):
        names = ("x", "dy", "g", "w", "dn", "z", "u", "dx", "dg", "dw", "dd", "ws")
        a = dict.fromkeys(names, FAKE)
        a.update(over)
        return L.gated_ffn_backward(a["x"], a["dy"], a["g"], a["w"], a["dn"], T, d, F, act, a["z"],
                                    a["u"], a["dx"], xt, a["dg"], a["dw"], a["dd"], wt, a["ws"], n,
                                    None, None)

    assert b(act=7) == INVALID and b(xt=3) == INVALID and b(wt=3) == INVALID
    assert b(F=252) == UNSUPPORTED
    for k in ("x", "dy", "g", "w", "dn", "z", "u", "dx", "dg", "dw", "dd", "ws"):
        assert b(**{k: None}) == INVALID, k
        assert b(**{k: FAKE + 4}) == ALIGN, k
    assert b(n=bws - 1) == WORKSPACE


def test_overlapping_arrays_are_refused(L):
    names = ("x", "dy", "g", "w", "dn", "z", "u", "dx", "dg", "dw", "dd", "ws")
    ws = L.gated_ffn_backward_workspace_size(100, 128, 256)

    def at(**over):
        a = {k: FAKE + 0x100000 * i for i, k in enumerate(names)}
        a.update({k: a[v] + off for k, (v, off) in over.items()})
        return a

    def b(**over):
        a = at(**over)
        return L.gated_ffn_backward(a["x"], a["dy"], a["g"], a["w"], a["dn"], 100, 128, 256, 1,
                                    a["z"], a["u"], a["dx"], 1, a["dg"], a["dw"], a["dd"], 0,
                                    a["ws"], ws, None, None)

    def f(**over):
        a = at(**over)
        return L.gated_ffn_forward(a["x"], a["g"], a["w"], a["dn"], 100, 128, 256, 1, a["z"], a["u"],
                                   a["dx"], 1, a["ws"], ws, None, None)

    for over in (dict(dx=("dy", 0)), dict(dg=("dw", 0)), dict(dd=("dn", 0)), dict(dx=("ws", 1024)),
                 dict(ws=("z", 16)), dict(dw=("dg", 256 * 128 * 4 - 16))):
        assert b(**over) == INVALID, over
    for over in (dict(dx=("x", 0)), dict(z=("u", 0)), dict(ws=("dn", 0)), dict(u=("x", -16))):
        assert f(**over) == INVALID, over


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 64, dtype=BF)
    w = torch.zeros(72, 64, dtype=BF)
    with pytest.raises(ValueError):
        twell.gated_ffn_forward(x, w, w, w, "silu", x, x)    # not on a GPU
    with pytest.raises(ValueError):
        twell._activation("tanh")
    with pytest.raises(ValueError):
        twell._check_ffn(x, w, w, w[:64])
    with pytest.raises(TypeError):
        twell._check_ffn(x.float(), w, w, w)


# ------------------------------------------------------------------ GPU -----
def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, d, F, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)

    return (normal(T, d), normal(T, d), normal(F, d, scale=2 * d ** -0.5),
            normal(F, d, scale=d ** -0.5), normal(F, d, scale=F ** -0.5))


def _half(dtype):
    return H if dtype == BF else 2.0 ** -24


def _product(a, b, da=0.0, db=0.0):
    """Error bound of a @ b in fp32 with operands off by da and db."""
    K = a.shape[1]
    A, B = np.abs(a), np.abs(b)
    out = K * 2.0 ** -23 * (A @ B)
    if np.ndim(da):
        out = out + da @ (B + (db if np.ndim(db) else 0))
    if np.ndim(db):
        out = out + A @ db
    return out


def _near(got, want, tol, dtype):
    err = np.abs(_f64(got) - want) - tol - _half(dtype) * 1.01 * (np.abs(want) + tol)
    assert np.all(err <= 0), float(err.max())


def _close(got, want):
    """The roundings are independent: in the mean the error is far below a bf16 step."""
    e = _f64(got) - want
    assert np.sqrt(np.mean(e ** 2)) <= H * np.sqrt(np.mean(want ** 2)) + 1e-30


def _check_forward(x, Wg, Wu, Wd, act, y, z=None, u=None):
    X, G, W, D = (_f64(t) for t in (x, Wg, Wu, Wd))
    ez, eu, eh, ey = layer.gated_ffn(X, G, W, D, act)
    tz, tu = _product(X, G.T), _product(X, W.T)
    if z is not None:
        _near(z, ez, tz, BF)
        _near(u, eu, tu, BF)
    a, _ = layer.activation(act, ez)
    # |act'| <= 1.13 for all four
    ta = 1.13 * tz + (1 + np.abs(ez)) * 2.0 ** -18
    th = np.abs(a) * tu + (np.abs(eu) + tu) * ta
    th = th + H * (np.abs(eh) + th)
    _near(y, ey, _product(eh, D, th), y.dtype)
    _close(y, ey)


SHAPES = [(1, 64, 64), (2, 2048, 264), (3, 72, 200), (16, 128, 8192), (17, 520, 1024),
          (64, 256, 384), (65, 64, 136), (129, 128, 264), (256, 264, 128), (300, 1000, 520),
          (513, 264, 1032), (1024, 512, 512), (8, 2048, 8192), (100, 1096, 2056), (200, 512, 2048),
          (260, 264, 4104)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d,F", SHAPES)
def test_forward(T, d, F, act):
    x, _, Wg, Wu, Wd = _inputs(T, d, F, T + d + F)
    ws = twell.gated_ffn_workspace(T, d, F)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (BF, F32):
        y = torch.full((T, d), 7.0, dtype=dtype, device="cuda")
        twell.gated_ffn_forward(x, Wg, Wu, Wd, act, y, ws, dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        _check_forward(x, Wg, Wu, Wd, act, y)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d,F", SHAPES)
def test_training_step(T, d, F, act):
    x, dy, Wg, Wu, Wd = _inputs(T, d, F, T * d + F)
    z, u = (torch.full((T, F), 7.0, dtype=BF, device="cuda") for _ in range(2))
    y = torch.empty((T, d), dtype=BF, device="cuda")
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    twell.gated_ffn_forward(x, Wg, Wu, Wd, act, y, ws, z=z, u=u, dev_status=st)
    torch.cuda.synchronize()
    _check_forward(x, Wg, Wu, Wd, act, y, z, u)
    X, DY, G, W, D, Z, Us = (_f64(t) for t in (x, dy, Wg, Wu, Wd, z, u))
    e = layer.gated_ffn_backward(X, DY, G, W, D, act, Z, Us)
    a, da = layer.activation(act, Z)
    t_dh = _product(DY, D.T)
    ta, tda = (1 + np.abs(Z)) * 2.0 ** -18, (1 + Z * Z) * 2.0 ** -18
    t_h = np.abs(Us) * ta
    t_du = np.abs(a) * t_dh + (np.abs(e["dh"]) + t_dh) * ta
    t_dz = np.abs(Us) * (np.abs(da) * t_dh + (np.abs(e["dh"]) + t_dh) * tda)
    t_h, t_du, t_dz = (t + H * (np.abs(v) + t)
                       for t, v in ((t_h, e["h"]), (t_du, e["du"]), (t_dz, e["dz"])))
    for xt, wt in ((BF, F32), (F32, BF)):
        dx = torch.full((T, d), 7.0, dtype=xt, device="cuda")
        dW = [torch.full((F, d), 7.0, dtype=wt, device="cuda") for _ in range(3)]
        twell.gated_ffn_backward(x, dy, Wg, Wu, Wd, act, z, u, dx, *dW, ws, dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        _near(dx, e["dx"], _product(e["du"], W, t_du) + _product(e["dz"], G, t_dz), xt)
        _near(dW[0], e["dWg"], _product(e["dz"].T, X, t_dz.T), wt)
        _near(dW[1], e["dWu"], _product(e["du"].T, X, t_du.T), wt)
        _near(dW[2], e["dWd"], _product(e["h"].T, DY, t_h.T), wt)
        for got, key in zip((dx, *dW), ("dx", "dWg", "dWu", "dWd")):
            _close(got, e[key])


@pytest.mark.gpu
def test_repeats_captures_and_rows_behind():
    T, d, F = 333, 512, 1024
    x, dy, Wg, Wu, Wd = _inputs(T, d, F, 5)
    z, u = (torch.full((T + 4, F), 7.0, dtype=BF, device="cuda") for _ in range(2))
    y, dx = (torch.full((T + 4, d), 7.0, dtype=BF, device="cuda") for _ in range(2))
    dW = [torch.empty((F, d), device="cuda") for _ in range(3)]
    ws = twell.gated_ffn_workspace(T, d, F, training=True)

    def step():
        twell.gated_ffn_forward(x, Wg, Wu, Wd, "silu", y[:T], ws, z=z[:T], u=u[:T])
        twell.gated_ffn_backward(x, dy, Wg, Wu, Wd, "silu", z[:T], u[:T], dx[:T], *dW, ws)

    step()
    torch.cuda.synchronize()
    for t in (z, u, y, dx):
        assert (t[T:] == 7).all()
    keep = [t.clone() for t in (z, u, y, dx, *dW)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (z, u, y, dx, *dW):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, k in zip((z, u, y, dx, *dW), keep):
        assert torch.equal(t[:T] if t.shape[0] == T + 4 else t, k[:T] if k.shape[0] == T + 4 else k)


@pytest.mark.gpu
def test_large_values_and_empty_batches():
    T, d, F = 40, 64, 64
    x, dy, Wg, Wu, Wd = _inputs(T, d, F, 6)
    x[0] = 1e4                                              # gates of +-1e4: act saturates
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    for act in ACTS:
        z, u = (torch.empty((T, F), dtype=BF, device="cuda") for _ in range(2))
        y, dx = (torch.empty((T, d), device="cuda") for _ in range(2))
        dW = [torch.empty((F, d), device="cuda") for _ in range(3)]
        twell.gated_ffn_forward(x, Wg, Wu, Wd, act, y, ws, z=z, u=u)
        twell.gated_ffn_backward(x, dy, Wg, Wu, Wd, act, z, u, dx, *dW, ws)
        torch.cuda.synchronize()
        _check_forward(x, Wg, Wu, Wd, act, y, z, u)
        assert all(torch.isfinite(t).all() for t in (dx, *dW))
    e = torch.empty((0, d), dtype=BF, device="cuda")
    ez = torch.empty((0, F), dtype=BF, device="cuda")
    dW = [torch.full((F, d), 7.0, device="cuda") for _ in range(3)]
    twell.gated_ffn_forward(e, Wg, Wu, Wd, "gelu", e, ez, z=ez, u=ez)
    twell.gated_ffn_backward(e, e, Wg, Wu, Wd, "gelu", ez, ez, e, *dW, ez)
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in dW)
