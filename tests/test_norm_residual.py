"""Norms around a block: the oracle's pins (CPU), refusals (CPU) and the kernels
against the fp64 oracle (GPU).

Tolerances, in units of u = 2^-24.  A sum over d columns is 8 fused multiply-adds
a thread, 5 levels over a warp and up to 32 warps added in order: 45u of the sum
of magnitudes.  An inverse norm halves that (its sum has one sign) and adds 4
roundings: 27u.  The mean of a product adds 5u to 45u.  Elementwise results add
their own few roundings, and a bf16 result half a step, 2^-8.
"""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_tma_b200 import build as tw_build
from activation_sparse_transformer_tma_b200 import twell
from oracle import layer

U = 2.0 ** -24
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 8
FAKE = 0x10000
BF, F32 = torch.bfloat16, torch.float32


# ----------------------------------------------------------------- CPU: pins --
def _case(rng, T, d, group, post=True, gate=True, pre=True):
    rows = -(-T // group) if gate else 0
    return dict(y=rng.standard_normal((T, d)), r=2 * rng.standard_normal((T, d)),
                w_post=1 + 0.2 * rng.standard_normal(d) if post else None,
                gate=rng.standard_normal((rows, d)) if gate else None,
                w_pre=1 + 0.2 * rng.standard_normal(d) if pre else None)


@pytest.mark.parametrize("post,gate,pre", [(1, 1, 1), (0, 1, 1), (1, 0, 1), (1, 1, 0), (0, 0, 0)])
def test_oracle_backward_equals_differences_and_autograd(post, gate, pre):
    rng = np.random.default_rng(3)
    T, d, group, a, s, eps = 5, 12, 2, 0.9, 0.5, 1e-3
    c = _case(rng, T, d, group, post, gate, pre)
    dr_out, dn = rng.standard_normal((T, d)), rng.standard_normal((T, d)) if pre else None

    def loss(**over):
        v = dict(c, **over)
        r1, n, _, _ = layer.norm_forward(v["y"], v["r"], v["w_post"], v["gate"], v["w_pre"],
                                         gate_group=group, a=a, s=s, eps=eps)
        return np.sum(r1 * dr_out) + (np.sum(n * dn) if pre else 0.0)

    r1, _, p, q = layer.norm_forward(c["y"], c["r"], c["w_post"], c["gate"], c["w_pre"],
                                     gate_group=group, a=a, s=s, eps=eps)
    g = layer.norm_backward(dn, dr_out, c["y"], r1, c["w_post"], c["gate"], c["w_pre"], p, q,
                            gate_group=group, a=a, s=s)
    names = {"y": "dy", "r": "dr", "w_post": "dw_post", "gate": "dgate", "w_pre": "dw_pre"}
    for key, out in names.items():
        if c[key] is None:
            continue
        for i in rng.choice(c[key].size, 6, replace=False):
            h, x = 1e-6, c[key].copy()
            x.flat[i] += h
            up = loss(**{key: x})
            x.flat[i] -= 2 * h
            assert abs((up - loss(**{key: x})) / (2 * h) - g[out].flat[i]) < 1e-6
    # the whole of it against automatic differentiation
    t = {k: torch.tensor(v, requires_grad=True) for k, v in c.items() if v is not None}
    o = t["y"]
    if post:
        o = o / torch.sqrt(o.square().mean(1, keepdim=True) + eps) * t["w_post"]
    if gate:
        o = t["gate"][torch.arange(T) // group] * o
    r2 = a * t["r"] + s * o
    total = (r2 * torch.tensor(dr_out)).sum()
    if pre:
        n2 = r2 / torch.sqrt(r2.square().mean(1, keepdim=True) + eps) * t["w_pre"]
        total = total + (n2 * torch.tensor(dn)).sum()
    total.backward()
    for key in t:
        np.testing.assert_allclose(g[names[key]], t[key].grad.numpy(), rtol=1e-9, atol=1e-12)


def test_oracle_forward_by_hand():
    # mean(y^2) = 25/2; r' = 1*r + 2*(3,4)/3.5355.. ; w_pre doubles
    r1, n, p, q = layer.norm_forward(np.array([[3.0, 4.0]]), np.array([[1.0, 1.0]]), np.ones(2),
                                     np.array([[2.0, 0.0]]), np.array([2.0, 2.0]), gate_group=1,
                                     eps=0.0)
    assert p[0] == pytest.approx(1 / np.sqrt(12.5))
    assert r1[0].tolist() == pytest.approx([1 + 6 / np.sqrt(12.5), 1.0])
    assert n[0].tolist() == pytest.approx((2 * r1[0] / np.sqrt(np.mean(r1[0] ** 2))).tolist())


# ------------------------------------------------------------- CPU: refusals --
@pytest.fixture(scope="module")
def L():
    tw_build.build()
    return twell.lib()


def _block(T=10, d=64, group=0, w_post=FAKE, gate=None, w_pre=FAKE, eps=1e-6, dtypes=(1, 0, 1, 1),
           a=1.0):
    return twell.TwNormBlockC(T, d, group, *dtypes, a, 1.0, eps, w_post, gate, w_pre)


def test_forward_refusals(L):
    def f(b, y=FAKE, r=FAKE, ro=FAKE, n=FAKE, p=None, q=None):
        return L.norm_residual_forward(ctypes.byref(b), y, r, ro, n, p, q, None)

    assert L.norm_residual_forward(None, FAKE, FAKE, FAKE, FAKE, None, None, None) == INVALID
    for bad in (dict(T=-1), dict(d=0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(a=float("inf")), dict(dtypes=(1, 0, 5, 1)), dict(gate=FAKE, group=0)):
        assert f(_block(**bad)) == INVALID, bad
    assert f(_block(d=60)) == UNSUPPORTED
    assert f(_block(d=8200)) == UNSUPPORTED
    assert f(_block(w_pre=FAKE + 4)) == ALIGN
    assert f(_block(), r=FAKE + 8) == ALIGN
    assert f(_block(), r=None) == INVALID
    assert f(_block(), ro=None) == INVALID                   # a block without its residual sum
    assert f(_block(), n=None) == INVALID                    # w_pre without n
    assert f(_block(w_pre=None)) == INVALID                  # n without w_pre
    assert f(_block(w_pre=None), n=None, q=FAKE) == INVALID
    assert f(_block(w_post=None), p=FAKE) == INVALID
    assert f(_block(), y=None, ro=None) == INVALID           # no block, but a w_post
    assert f(_block(w_post=None, w_pre=None), y=None, ro=None, n=None) == INVALID
    assert f(_block(T=0), y=None, r=None, ro=None, n=None) == OK   # an empty batch


def test_backward_refusals(L):
    size = L.norm_residual_backward_workspace_size(10, 64, 0)
    assert size > 0 and L.norm_residual_backward_workspace_size(-1, 64, 0) == 0
    names = ["dn", "dr_out", "y", "r_out", "rstd_post", "rstd_pre", "dy", "dr", "dw_post", "dgate",
             "dw_pre", "ws"]

    def f(b, n=size, **over):
        a = dict.fromkeys(names, FAKE)
        a["dgate"] = None
        a.update(over)
        return L.norm_residual_backward(ctypes.byref(b), *[a[k] for k in names], n, None)

    assert f(_block(), n=size - 1) == WORKSPACE
    for bad in (dict(dr=None), dict(dn=None), dict(dw_pre=None), dict(dw_post=None), dict(dy=None),
                dict(r_out=None), dict(rstd_pre=None), dict(rstd_post=None), dict(ws=None),
                dict(dgate=FAKE)):
        assert f(_block(), **bad) == INVALID, bad
    assert f(_block(w_pre=None), dn=None, dw_pre=None, rstd_pre=None, dr_out=None) == INVALID
    assert f(_block(gate=FAKE, group=5)) == INVALID          # a gate without its gradient
    assert f(_block(), dy=FAKE + 8) == ALIGN


def test_overlapping_arrays_are_refused(L):
    # 10 x 64: 1280 bytes of bf16 (y, n), 2560 of fp32 (r)
    y, r, ro, n, w = (FAKE + 0x10000 * k for k in range(5))
    b = _block(w_post=w, w_pre=w + 0x1000)

    def f(y=y, r=r, ro=ro, n=n):
        return L.norm_residual_forward(ctypes.byref(b), y, r, ro, n, None, None, None)

    assert f(ro=r + 1280) == INVALID and f(n=r) == INVALID and f(ro=y) == INVALID
    assert f(n=w) == INVALID and f(ro=n) == INVALID and f(n=y + 16) == INVALID
    size = L.norm_residual_backward_workspace_size(10, 64, 0)
    names = ["dn", "dr_out", "y", "r_out", "rstd_post", "rstd_pre", "dy", "dr", "dw_post", "dgate",
             "dw_pre", "ws"]

    def g(**over):
        a = {k: FAKE + 0x10000 * i for i, k in enumerate(names)}
        a["dgate"] = None
        a.update({k: a[v] for k, v in over.items()})
        return L.norm_residual_backward(ctypes.byref(b), *[a[k] for k in names], size, None)

    for k, v in (("dr", "r_out"), ("dw_post", "dw_pre"), ("ws", "y"), ("dy", "dr"), ("dr", "dn"),
                 ("dw_pre", "rstd_pre")):
        assert g(**{k: v}) == INVALID, (k, v)


def test_binding_refuses_host_tensors_and_mixed_weights():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        twell.norm_residual_forward(x, x, None, None, x[0], x, x)
    with pytest.raises(TypeError):
        twell._norm_block(4, 8, F32, F32, F32, (torch.zeros(8), None, torch.zeros(8, dtype=BF)),
                          (None, None, None), 0, 1.0, 1.0, 0.0)
    with pytest.raises(ValueError):
        twell._norm_block(4, 8, F32, F32, F32, (None, torch.zeros(3, 8), None), (None, None, None),
                          2, 1.0, 1.0, 0.0)
    with pytest.raises(TypeError):
        twell._norm_block(4, 8, torch.float16, F32, F32, (None, None, None), (None, None, None), 0,
                          1.0, 1.0, 0.0)


# ------------------------------------------------------------------ GPU -----
def _dev(c, y, r, w):
    want = dict(y=y, r=r, w_post=w, gate=w, w_pre=w)
    return {k: None if v is None else torch.tensor(v, device="cuda").to(want[k])
            for k, v in c.items()}


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else U


def _check_forward(t, r_out, n_out, p, q, group, a, s, eps):
    e = {k: _f64(v) for k, v in t.items()}
    want_r, want_n, want_p, want_q = layer.norm_forward(
        e["y"], e["r"], e["w_post"], e["gate"], e["w_pre"], gate_group=group, a=a, s=s, eps=eps)
    block = np.abs(want_r - a * e["r"])
    r_tol = U * (2 * np.abs(a * e["r"]) + 35 * block)        # fp32, before its own rounding
    assert np.all(np.abs(_f64(r_out) - want_r) <= r_tol + _half(r_out.dtype) * np.abs(want_r) * 1.01)
    if want_p is not None:
        assert np.all(np.abs(_f64(p) - want_p) <= 28 * U * want_p)
    if want_n is not None:
        rel = 28 * U + np.sqrt(np.sum(r_tol ** 2, axis=1) /
                               np.maximum(np.sum(want_r ** 2, axis=1), 1e-300))
        n_tol = (np.abs(want_n) * (rel[:, None] + 3 * U) +
                 r_tol * np.abs(want_q[:, None] * e["w_pre"]))
        assert np.all(np.abs(_f64(n_out) - want_n) <= n_tol + _half(n_out.dtype) * np.abs(want_n) * 1.01)
        assert np.all(np.abs(_f64(q) - want_q) <= rel * want_q)


GATES = ["none", "one", 1, 7, 40]
SHAPES = [(1, 8), (1, 2048), (3, 136), (37, 256), (300, 264), (65, 1000), (333, 2048), (5, 4104),
          (40, 8192)]


def _group(gate, T):
    return {"none": 0, "one": T + 5}.get(gate, gate)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(T, d, gate):
    rng = np.random.default_rng(T * 10000 + d)
    group = _group(gate, T)
    for i, (yt, rt, nt, wt, post, pre) in enumerate([(BF, F32, BF, BF, True, True),
                                                     (F32, BF, F32, F32, True, True),
                                                     (BF, BF, BF, F32, False, True),
                                                     (F32, F32, F32, BF, True, False)]):
        t = _dev(_case(rng, T, d, group, post, group > 0, pre), yt, rt, wt)
        r_out = torch.full((T, d), 7.0, dtype=rt, device="cuda")
        n_out = torch.empty((T, d), dtype=nt, device="cuda") if pre else None
        p = torch.empty(T, device="cuda") if post else None
        q = torch.empty(T, device="cuda") if pre else None
        twell.norm_residual_forward(t["y"], t["r"], t["w_post"], t["gate"], t["w_pre"], r_out,
                                    n_out, gate_group=group, res_scale=0.75, block_scale=0.5,
                                    eps=1e-5, rstd_post=p, rstd_pre=q)
        torch.cuda.synchronize()
        _check_forward(t, r_out, n_out, p, q, group, 0.75, 0.5, float(np.float32(1e-5)))


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(1, 64), (70, 512), (9, 5000)])
def test_first_norm_of_a_network_and_its_gradient(T, d):
    rng = np.random.default_rng(T)
    c = _case(rng, T, d, 0, False, False, True)
    t = _dev(c, F32, F32, F32)
    n = torch.empty((T, d), dtype=BF, device="cuda")
    q = torch.empty(T, device="cuda")
    twell.norm_residual_forward(None, t["r"], None, None, t["w_pre"], None, n, rstd_pre=q)
    want = layer.norm_forward(None, _f64(t["r"]), None, None, _f64(t["w_pre"]))
    assert np.all(np.abs(_f64(n) - want[1]) <= (31 * U + 2.0 ** -8) * np.abs(want[1]) * 1.01)
    dn = torch.tensor(rng.standard_normal((T, d)), device="cuda").to(BF)
    dr, dw = torch.empty((T, d), device="cuda"), torch.empty(d, device="cuda")
    twell.norm_residual_backward(dn, None, None, t["r"], None, None, t["w_pre"], None, q, None, dr,
                                 None, None, dw, twell.norm_residual_backward_workspace(T, d))
    torch.cuda.synchronize()
    _check_backward(dict(dn=dn, dr_out=None, y=None, r_out=t["r"], w_post=None, gate=None,
                         w_pre=t["w_pre"], p=None, q=q), dict(dr=dr, dw_pre=dw), 0, 1.0, 1.0)


def _check_backward(t, got, group, a, s):
    e = {k: _f64(v) for k, v in t.items()}
    w = layer.norm_backward(e["dn"], e["dr_out"], e["y"], e["r_out"], e["w_post"], e["gate"],
                            e["w_pre"], e["p"], e["q"], gate_group=group, a=a, s=s)
    G = w["G"]
    T, d = G.shape
    g_tol = 2 * U * np.abs(G)
    terms = np.zeros_like(G)                                 # magnitudes that G is summed from
    if e["dr_out"] is not None:
        g_tol = g_tol + U * np.abs(e["dr_out"])
        terms = terms + np.abs(e["dr_out"])
    if e["dn"] is not None:
        q = e["q"][:, None]
        rh, ee = e["r_out"] * q, e["dn"] * e["w_pre"]
        inner = np.mean(ee * rh, axis=1, keepdims=True)
        e1 = 50 * U * np.mean(np.abs(ee * rh), axis=1, keepdims=True)
        g_tol = g_tol + q * (4 * U * np.abs(ee) + np.abs(rh) * (e1 + 4 * U * np.abs(inner)))
        terms = terms + q * (np.abs(ee) + np.abs(rh * inner))
        # a sum over T tokens, in any order: T roundings at most, and 3 of the terms
        tol = (T + 24) * U * np.sum(np.abs(e["dn"] * rh), axis=0)
        assert np.all(np.abs(_f64(got["dw_pre"]) - w["dw_pre"]) <= tol)
    # without a block there is no residual scale, and dr is G itself
    scale = 1.0 if e["y"] is None else abs(a)
    dr = got["dr"]
    assert np.all(np.abs(_f64(dr) - w["dr"]) <=
                  scale * g_tol + (U + _half(dr.dtype) * 1.01) * np.abs(w["dr"]))
    if e["y"] is None:
        return
    row = np.arange(T) // group if e["gate"] is not None else None
    gt = 1.0 if row is None else e["gate"][row]
    k = s * gt * G
    k_tol = np.abs(s * gt) * g_tol + 3 * U * np.abs(k)
    yh = e["y"] if e["p"] is None else e["y"] * e["p"][:, None]
    o = yh if e["w_post"] is None else yh * e["w_post"]
    if e["w_post"] is None:
        dy_tol = k_tol
    else:
        f, f_tol = k * e["w_post"], np.abs(e["w_post"]) * k_tol + U * np.abs(k * e["w_post"])
        inner = np.mean(f * yh, axis=1, keepdims=True)
        # the mean of f yh is summed from the terms of G one by one, each product rounded as in a
        # sum of their magnitudes
        e2 = np.mean(f_tol * np.abs(yh) + 50 * U * np.abs(s * gt * e["w_post"] * terms * yh),
                     axis=1, keepdims=True)
        dy_tol = e["p"][:, None] * (f_tol + 4 * U * np.abs(f) +
                                    np.abs(yh) * (e2 + 4 * U * np.abs(inner)))
        tol = np.sum(k_tol * np.abs(yh) + (T + 24) * U * np.abs(k * yh), axis=0)
        assert np.all(np.abs(_f64(got["dw_post"]) - w["dw_post"]) <= tol)
    dy = got["dy"]
    assert np.all(np.abs(_f64(dy) - w["dy"]) <= dy_tol + _half(dy.dtype) * 1.01 * np.abs(w["dy"]))
    if row is not None:
        tol = np.zeros_like(e["gate"])
        np.add.at(tol, row, g_tol * np.abs(s * o) + (T + 24) * U * np.abs(s * G * o))
        assert np.all(np.abs(_f64(got["dgate"]) - w["dgate"]) <= tol)


def _backward(rng, T, d, group, yt, rt, nt, wt, post, pre, with_dr, a=0.75, s=0.5):
    t = _dev(_case(rng, T, d, group, post, group > 0, pre), yt, rt, wt)

    def normal(dtype):
        return torch.tensor(rng.standard_normal((T, d)), device="cuda").to(dtype)

    def inverse(x):
        return 1 / torch.sqrt(x.float().square().mean(1) + 1e-5)

    t["r_out"] = t.pop("r")
    t.update(dn=normal(nt) if pre else None, dr_out=normal(rt) if with_dr else None,
             p=inverse(t["y"]) if post else None, q=inverse(t["r_out"]) if pre else None)

    def empty(on, shape, dtype=F32):
        return torch.full(shape, 7.0, dtype=dtype, device="cuda") if on else None

    got = dict(dy=empty(True, (T, d), yt), dr=empty(True, (T, d), rt), dw_post=empty(post, (d,)),
               dgate=empty(group > 0, (-(-T // group) if group else 0, d)), dw_pre=empty(pre, (d,)))
    ws = twell.norm_residual_backward_workspace(T, d, group)

    def run(**kw):
        twell.norm_residual_backward(t["dn"], t["dr_out"], t["y"], t["r_out"], t["w_post"],
                                     t["gate"], t["w_pre"], t["p"], t["q"], got["dy"], got["dr"],
                                     got["dw_post"], got["dgate"], got["dw_pre"], ws,
                                     gate_group=group, res_scale=a, block_scale=s, **kw)

    return t, got, run


@pytest.mark.gpu
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,d", SHAPES + [(5000, 64)])
def test_backward(T, d, gate):
    rng = np.random.default_rng(T * 10000 + d)
    group = _group(gate, T)
    for yt, rt, nt, wt, post, pre, with_dr in [(BF, F32, BF, BF, True, True, True),
                                               (F32, BF, F32, F32, True, True, False),
                                               (BF, BF, BF, F32, False, True, True),
                                               (F32, F32, F32, BF, True, False, True)]:
        t, got, run = _backward(rng, T, d, group, yt, rt, nt, wt, post, pre, with_dr)
        run()
        torch.cuda.synchronize()
        _check_backward(t, got, group, 0.75, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(2000, 64), (1500, 1000), (900, 2048), (60, 4104)])
@pytest.mark.parametrize("group", [2, 12, 31, 50, 100, 333])
def test_backward_of_groups_of_every_length(T, d, group):
    """Groups to a team each, to a CTA each, and cut into several items."""
    rng = np.random.default_rng(T + group)
    t, got, run = _backward(rng, T, d, group, BF, F32, BF, BF, True, True, True)
    run()
    torch.cuda.synchronize()
    _check_backward(t, got, group, 0.75, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(5001, 64), (3001, 520), (1501, 1000), (901, 2048), (301, 4096), (301, 8192)])
@pytest.mark.parametrize("group", [1, 2])
def test_backward_of_many_short_groups(T, d, group):
    """Several groups a team, each of one row, or of two and the last of one."""
    rng = np.random.default_rng(T + group)
    for yt, rt, nt, wt, post, pre, with_dr in [(BF, F32, BF, BF, True, True, True),
                                               (F32, F32, F32, F32, True, True, True),
                                               (BF, BF, BF, F32, False, True, True)]:
        t, got, run = _backward(rng, T, d, group, yt, rt, nt, wt, post, pre, with_dr)
        run()
        torch.cuda.synchronize()
        _check_backward(t, got, group, 0.75, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,group", [(50, 8192, 7), (90, 8192, 40), (300, 8192, 300), (90, 4096, 40),
                                       (90, 4096, 3), (200, 2048, 33), (90, 512, 40)])
def test_all_fp32_with_gate_rows(T, d, group):
    """The most shared memory that a width asks for."""
    rng = np.random.default_rng(T + d + group)
    t, got, run = _backward(rng, T, d, group, F32, F32, F32, F32, True, True, True)
    run()
    torch.cuda.synchronize()
    _check_backward(t, got, group, 0.75, 0.5)
    for k in ("r", "r_out"):
        t[k] = t["r_out"].clone()
    n = torch.empty_like(t["r"])
    twell.norm_residual_forward(t["y"], t["r"], t["w_post"], t["gate"], t["w_pre"], t["r_out"], n,
                                gate_group=group, res_scale=0.75, block_scale=0.5, eps=1e-5,
                                rstd_post=t["p"], rstd_pre=t["q"])
    torch.cuda.synchronize()
    f = {k: t[k] for k in ("y", "r", "w_post", "gate", "w_pre")}
    _check_forward(f, t["r_out"], n, t["p"], t["q"], group, 0.75, 0.5, float(np.float32(1e-5)))


@pytest.mark.gpu
def test_remaining_dtype_combinations():
    rng = np.random.default_rng(8)
    for yt in (BF, F32):
        for rt in (BF, F32):
            for nt in (BF, F32):
                t, got, run = _backward(rng, 50, 520, 20, yt, rt, nt, F32, True, True, True)
                run()
                torch.cuda.synchronize()
                _check_backward(t, got, 20, 0.75, 0.5)


@pytest.mark.gpu
def test_outputs_may_be_their_inputs_and_repeats_are_bitwise_equal():
    rng = np.random.default_rng(1)
    t, got, run = _backward(rng, 700, 1000, 100, BF, F32, BF, BF, True, True, True)
    run()
    torch.cuda.synchronize()
    keep = {k: v.clone() for k, v in got.items()}
    run()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], keep[k]) for k in got)
    got["dr"], got["dy"] = t["dr_out"], t["y"]              # in place
    run()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], keep[k]) for k in got)
    # forward: r_out over r, n_out over y
    t = _dev(_case(rng, 200, 1000, 0, True, False, True), BF, F32, BF)
    ro, no = torch.empty_like(t["r"]), torch.empty_like(t["y"])
    twell.norm_residual_forward(t["y"], t["r"], t["w_post"], None, t["w_pre"], ro, no)
    twell.norm_residual_forward(t["y"], t["r"], t["w_post"], None, t["w_pre"], t["r"], t["y"])
    torch.cuda.synchronize()
    assert torch.equal(ro, t["r"]) and torch.equal(no, t["y"])


@pytest.mark.gpu
def test_rows_behind_the_last_token_stay_and_empty_batches():
    rng = np.random.default_rng(2)
    t = _dev(_case(rng, 5, 72, 0, True, False, True), BF, F32, BF)
    ro, no = torch.full((9, 72), 7.0, device="cuda"), torch.full((9, 72), 7.0, device="cuda")
    twell.norm_residual_forward(t["y"], t["r"], t["w_post"], None, t["w_pre"], ro[:5], no[:5])
    torch.cuda.synchronize()
    assert (ro[5:] == 7).all() and (no[5:] == 7).all()
    e = torch.empty((0, 72), device="cuda")
    twell.norm_residual_forward(e, e, t["w_post"].float(), None, t["w_pre"].float(), e, e)
    dw = torch.full((2, 72), 7.0, device="cuda")
    twell.norm_residual_backward(e, None, e, e, t["w_post"], None, t["w_pre"], e[:, 0], e[:, 0], e,
                                 e, dw[0], None, dw[1], torch.empty(0, device="cuda"))
    torch.cuda.synchronize()
    assert (dw == 0).all()


@pytest.mark.gpu
def test_captured_backwards_replay_beside_an_eager_one():
    rng = np.random.default_rng(4)
    t, got, run = _backward(rng, 333, 512, 50, BF, F32, BF, BF, True, True, True)
    run()
    torch.cuda.synchronize()
    keep = {k: v.clone() for k, v in got.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for v in got.values():
        v.zero_()
    graph.replay()
    t2, got2, run2 = _backward(rng, 333, 512, 50, BF, F32, BF, BF, True, True, True)
    run2()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], keep[k]) for k in got)
    _check_backward(t2, got2, 50, 0.75, 0.5)
