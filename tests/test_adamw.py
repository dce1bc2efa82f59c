"""AdamW step: the oracle's pins (CPU), the entry point's refusals (CPU), and
the kernels against the fp64 oracle (GPU).

Tolerances, in units of u = 2^-24 (half an fp32 step, relative): beta and
1 - beta are rounded once (u each), and m is one product and one fused
multiply-add on top, so m is off by at most 4u of |beta1 m| + |(1-beta1) g|.
v is a sum of non-negative terms: 4u.  The denominator adds half of that and
three roundings (square root, bias factor, sum): 6u.  The update is that, the
division, the step size and its product: 4 + 6 + 3 = 13u of its terms; the
parameter adds 1u for its decay factor and 1u for the final sum.
"""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_tma_b200 import build as tw_build
from activation_sparse_transformer_tma_b200 import twell
from oracle import layer

U = 2.0 ** -24
OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3
FAKE = 0x10000


# ----------------------------------------------------------------- CPU: pins --
def test_oracle_equals_torch_adamw():
    rng = np.random.default_rng(0)
    p, steps = rng.standard_normal(50), [rng.standard_normal(50) for _ in range(4)]
    q = torch.from_numpy(p.copy()).requires_grad_()
    opt = torch.optim.AdamW([q], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m = v = np.zeros(50)
    for t, g in enumerate(steps, 1):
        q.grad = torch.from_numpy(g)
        opt.step()
        p, m, v, _ = layer.adamw(p, g, m, v, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=t,
                                 weight_decay=0.1)
    np.testing.assert_allclose(p, q.detach().numpy(), rtol=1e-12)


def test_oracle_code_laws_by_hand():
    # one block, largest |m| = 2: code 127, and a quarter of it at 127/2 = 63.5 -> 64 (ties to even)
    pos, scale = layer.adamw_positions(np.array([2.0, 0.5, 0.0]), 127)
    assert pos.tolist() == [127.0, 63.5, 0.0] and scale.tolist() == [2.0 / 16129]
    assert layer.adamw_m_value([127, -127, 0], scale).tolist() == pytest.approx([2.0, -2.0, 0.0])
    pos, scale = layer.adamw_positions(np.sqrt([4.0, 0.25]), 255)
    assert pos.tolist() == [255.0, 127.5]
    assert layer.adamw_v_value([255, 0], scale).tolist() == pytest.approx([4.0, 0.0])


# ------------------------------------------------------------- CPU: refusals --
@pytest.fixture(scope="module")
def L():
    tw_build.build()
    return twell.lib()


def _desc(base=FAKE, n=300, bits=32, **over):
    t = twell.TwAdamwTensorC(n, base, None, base + 0x1000, base + 0x2000, base + 0x3000, None, None,
                             None, None, twell.TW_F32, twell.TW_F32, twell.TW_F32, bits, 0.0)
    if bits == 8:
        t.m_scale, t.v_scale = base + 0x4000, base + 0x5000
    for k, x in over.items():
        setattr(t, k, x)
    return t


def _call(L, *descs, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, count=None, step_dev=None):
    arr = (twell.TwAdamwTensorC * max(len(descs), 1))(*descs)
    a = twell.TwAdamwArgsC(lr, b1, b2, eps, step, None, step_dev, None)
    return L.adamw_step(arr, len(descs) if count is None else count, ctypes.byref(a), None)


def test_refusals(L):
    assert _call(L) == OK                                     # nothing to do
    assert _call(L, _desc(n=0, p=None, g=None)) == OK
    assert L.adamw_step(None, 1, None, None) == INVALID
    assert _call(L, _desc(), count=-1) == INVALID
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(eps=0.0),
                dict(eps=1e-60), dict(eps=1e-39), dict(step=0)):
        assert _call(L, _desc(), **bad) == INVALID
    assert _call(L, _desc(), step_dev=FAKE + 2) == ALIGN
    assert _call(L, _desc(n=-1)) == INVALID
    assert _call(L, _desc(n=1 << 41)) == UNSUPPORTED
    assert _call(L, _desc(bits=16)) == UNSUPPORTED
    assert _call(L, _desc(m=None)) == INVALID
    assert _call(L, _desc(p_dtype=7)) == INVALID
    assert _call(L, _desc(weight_decay=-0.1)) == INVALID
    assert _call(L, _desc(master=FAKE + 0x6000)) == INVALID   # a master copy of an fp32 parameter
    assert _call(L, _desc(m_scale=FAKE + 0x4000)) == INVALID  # scales belong to 8-bit moments
    assert _call(L, _desc(bits=8, v_scale=None)) == INVALID
    assert _call(L, _desc(bits=8, m_values=FAKE + 0x6000)) == INVALID  # both or neither
    assert _call(L, _desc(g=FAKE + 0x1004)) == ALIGN


def test_overlapping_arrays_are_refused(L):
    assert _call(L, _desc(), _desc()) == INVALID                      # the same parameter twice
    assert _call(L, _desc(), _desc(FAKE + 0x10000, m=FAKE + 0x2000 + 1184)) == INVALID
    assert _call(L, _desc(), _desc(FAKE + 0x10000, g=FAKE)) == INVALID  # reads what another writes
    assert _call(L, _desc(g=FAKE)) == INVALID                         # its own parameter
    # 300 fp32 elements end at 1200: the next 16-byte address is free
    assert _call(L, _desc(m=FAKE + 1200, n=300), count=0) == OK


def test_packing_refuses_wrong_tensors():
    f = torch.zeros(8)
    ok = dict(p=f, g=f.clone(), m=f.clone(), v=f.clone())
    with pytest.raises(ValueError):
        twell.AdamWTensors([ok])                              # not on a GPU
    with pytest.raises(TypeError):
        twell.AdamWTensors([dict(ok, grad=f)])
    with pytest.raises(ValueError):
        twell.AdamWTensors([dict(ok, m=None)])
    with pytest.raises(TypeError):
        twell.AdamWTensors([dict(ok, m=f.to(torch.int8))])    # p is packed first: still no GPU
    assert twell.adamw_step(twell.AdamWTensors([]), lr=1e-3) is None
    assert [twell.adamw_blocks(n) for n in (0, 1, 256, 257)] == [0, 1, 1, 2]


# ------------------------------------------------------------------ GPU -----
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _make(n, seed, bits=32, p=torch.float32, g=torch.float32, master=False, zero=False):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(scale):
        return torch.randn(n, generator=gen, device="cuda") * scale

    w = normal(0.05)
    t = dict(p=w.to(p), g=normal(0.02).to(g), master=w.clone() if master else None,
             weight_decay=0.1)
    if bits == 32:
        t.update(m=normal(0.01), v=normal(0.02).square())
        if zero:
            t["m"].zero_(), t["v"].zero_()
        return t
    nb = twell.adamw_blocks(n)
    t.update(m=torch.zeros(n, dtype=torch.int8, device="cuda"),
             v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
             m_scale=torch.zeros(nb, device="cuda"), v_scale=torch.zeros(nb, device="cuda"),
             m_values=torch.empty(n, device="cuda"), v_values=torch.empty(n, device="cuda"))
    if not zero:
        t["m"].copy_(torch.randint(-127, 128, (n,), generator=gen, device="cuda"))
        t["v"].copy_(torch.randint(1, 256, (n,), generator=gen, device="cuda"))
        t["m_scale"].fill_(0.02 / 127 ** 2)
        t["v_scale"].fill_(0.02 / 255 ** 2)
    return t


def _before(t):
    src = t["p"] if t["master"] is None else t["master"]
    if t["m"].dtype == torch.int8:
        m = layer.adamw_m_value(t["m"].cpu().numpy(), t["m_scale"].cpu().numpy())
        v = layer.adamw_v_value(t["v"].cpu().numpy(), t["v_scale"].cpu().numpy())
    else:
        m, v = _f64(t["m"]), _f64(t["v"])
    return _f64(src), _f64(t["g"]), m, v


def _check(t, before, step, weight_decay=0.1, grad_scale=1.0, **hyper):
    p0, g, m0, v0 = before
    h = dict(HYPER, **hyper)
    p, m, v, terms = layer.adamw(p0, g, m0, v0, step=step, weight_decay=weight_decay,
                                 grad_scale=grad_scale, **h)
    # the states' own decoding costs 3 roundings of an 8-bit m and 7 of v (8-bit only), a gradient
    # scale one more: 16u and 6u cover both forms
    tol = U * (2 * np.abs(p0) + np.abs(p) + 24 * terms)
    if t["master"] is not None:
        assert np.all(np.abs(_f64(t["master"]) - p) <= tol)
        assert torch.equal(t["p"], t["master"].to(torch.bfloat16))
    else:
        half = 2.0 ** -8 if t["p"].dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(_f64(t["p"]) - p) <= tol + half * np.abs(p))
    m_tol = 8 * U * (np.abs(h["beta1"] * m0) + np.abs((1 - h["beta1"]) * grad_scale * g))
    v_tol = 14 * U * v
    if t["m"].dtype != torch.int8:
        assert np.all(np.abs(_f64(t["m"]) - m) <= m_tol)
        assert np.all(np.abs(_f64(t["v"]) - v) <= v_tol)
        return
    mc, vc = t["m"].cpu().numpy().astype(np.int64), t["v"].cpu().numpy().astype(np.int64)
    ms, vs = _f64(t["m_scale"]), _f64(t["v_scale"])
    # the code is within half a step of the exact position; the position moves with the
    # moment's error, and by 4u relative for its reciprocal, product and square root
    top_slack = 1 + 32 * U
    for code, scale, x, tol_x, most in ((np.abs(mc), ms, np.abs(m), m_tol, 127),
                                        (vc, vs, np.sqrt(v), 8 * U * np.sqrt(v), 255)):
        pos_hi, want = layer.adamw_positions(x + tol_x, most)
        pos_lo, _ = layer.adamw_positions(np.maximum(x - tol_x, 0), most)
        assert np.all(code <= pos_hi * top_slack + 0.5 + 1e-4)
        floor = np.minimum(pos_lo / top_slack - 0.5 - 1e-4, most)
        assert np.all(code >= floor)
        assert np.all(np.abs(scale - want) <= 64 * U * want)
    assert np.all((vc > 0) == (v > 0))
    sure = np.abs(m) > m_tol
    assert np.all((np.sign(mc) == np.sign(m))[sure & (mc != 0)])
    # the values that come back are those of the codes
    np.testing.assert_allclose(_f64(t["m_values"]), layer.adamw_m_value(mc, ms), rtol=4 * U)
    np.testing.assert_allclose(_f64(t["v_values"]), layer.adamw_v_value(vc, vs), rtol=8 * U)


SIZES = [1, 3, 4, 255, 256, 257, 8191, 8193, 100003]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g,master", [(torch.float32, torch.float32, False),
                                        (torch.bfloat16, torch.float32, True),
                                        (torch.bfloat16, torch.bfloat16, True),
                                        (torch.bfloat16, torch.bfloat16, False)])
def test_step_over_many_sizes(bits, p, g, master):
    ts = [_make(n, i, bits, p, g, master, zero=i % 3 == 2) for i, n in enumerate(SIZES)]
    before = [_before(t) for t in ts]
    twell.adamw_step(twell.AdamWTensors(ts), step=7, **HYPER)
    torch.cuda.synchronize()
    for t, b in zip(ts, before):
        _check(t, b, 7)


@pytest.mark.gpu
def test_300_tensors_and_mixed_states_take_several_launches():
    ts = [_make(1 + 37 * i % 700, i, bits=8 if i % 2 else 32, zero=True) for i in range(300)]
    before = [_before(t) for t in ts]
    twell.adamw_step(twell.AdamWTensors(ts), step=1, **HYPER)
    torch.cuda.synchronize()
    for t, b in zip(ts, before):
        _check(t, b, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_bytes_behind_a_tensor_stay(bits):
    """Odd-sized tensors inside larger buffers: what lies behind is not written."""
    n, room = 261, 512
    full = _make(room, 5, bits)
    keep = {k: x.clone() for k, x in full.items() if torch.is_tensor(x)}
    t = {k: (x if not torch.is_tensor(x) or k.endswith("_scale") else x[:n]) for k, x in full.items()}
    before = _before(t)
    twell.adamw_step(twell.AdamWTensors([t]), step=3, **HYPER)
    torch.cuda.synchronize()
    _check(t, before, 3)
    for k, x in keep.items():
        if not k.endswith(("_scale", "_values")):
            assert torch.equal(full[k][n:], x[n:]), k


@pytest.mark.gpu
def test_captured_step_reads_its_scalars_at_each_replay():
    ts = [_make(n, 40 + i, 32, torch.bfloat16, torch.float32, True) for i, n in enumerate((1000, 9000))]
    step = torch.ones(1, dtype=torch.int32, device="cuda")
    lr, gs = torch.tensor([1e-3], device="cuda"), torch.tensor([1.0], device="cuda")
    plan = twell.AdamWTensors(ts)
    kw = dict(HYPER, lr=0.0, step_dev=step, lr_dev=lr, grad_scale=gs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twell.adamw_step(plan, **kw)
    for s, (r, scale) in enumerate(((1e-3, 1.0), (5e-4, 0.25), (2e-3, 2.0)), 1):
        step.fill_(s), lr.fill_(r), gs.fill_(scale)
        before = [_before(t) for t in ts]
        graph.replay()
        torch.cuda.synchronize()
        for t, b in zip(ts, before):
            _check(t, b, s, lr=float(np.float32(r)), grad_scale=scale)


@pytest.mark.gpu
def test_non_finite_gradients_show_in_their_block_alone():
    t = _make(1024, 9, 8)
    t["g"][300] = float("inf")
    t["g"][700] = float("nan")
    twell.adamw_step(twell.AdamWTensors([t]), step=2, **HYPER)
    torch.cuda.synchronize()
    bad = torch.isnan(t["m_values"]).view(4, 256)
    assert bad[1].all() and bad[2].all() and not bad[0].any() and not bad[3].any()
    assert torch.equal(torch.isnan(t["v_values"]).view(4, 256), bad)
    assert torch.isnan(t["p"]).sum() == 2      # inf/inf and NaN: the others moved as usual


@pytest.mark.gpu
def test_two_streams_at_once_and_a_later_state():
    a, b = _make(50000, 1, 32), _make(50000, 2, 32)
    before = _before(a), _before(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    twell.adamw_step(twell.AdamWTensors([a]), step=5, stream=s1, **HYPER)
    twell.adamw_step(twell.AdamWTensors([b]), step=5, stream=s2, **HYPER)
    torch.cuda.synchronize()
    _check(a, before[0], 5)
    _check(b, before[1], 5)
