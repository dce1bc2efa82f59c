"""AdamW step: arrays side by side and the device scalars' places, 8-bit moments in a captured
step, and without the values written."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_tma_b200 import build as tw_build
from activation_sparse_transformer_tma_b200 import twell
from test_adamw import FAKE, HYPER, INVALID, _before, _check, _desc, _make


@pytest.fixture(scope="module")
def L():
    tw_build.build()
    return twell.lib()


def _call(L, lr_dev=None, step_dev=None, grad_scale=None, **over):
    a = twell.TwAdamwArgsC(1e-3, 0.9, 0.99, 1e-8, 1, lr_dev, step_dev, grad_scale)
    return L.adamw_step((twell.TwAdamwTensorC * 1)(_desc(**over)), 1, ctypes.byref(a), None)


@pytest.mark.parametrize("word", ["lr_dev", "step_dev", "grad_scale"])
def test_device_scalars_inside_written_arrays_are_refused(L, word):
    """Some warps would read the word before it is overwritten and others after."""
    t = _desc()
    for at in (t.p, t.p + 4, t.m + 4 * 299, t.v + 16):
        assert _call(L, **{word: at}) == INVALID, hex(at - FAKE)
    s = _desc(bits=8)
    for at in (s.m_scale + 4, s.v_scale, s.v + 296):
        assert _call(L, bits=8, **{word: at}) == INVALID, hex(at - FAKE)


def test_arrays_16_bytes_too_near_are_refused(L):
    # 300 fp32 elements end at 1200, 300 codes at 300
    assert _call(L, g=FAKE + 1200 - 16) == INVALID
    assert _call(L, m=FAKE + 1200 - 16) == INVALID
    assert _call(L, bits=8, v=FAKE + 0x2000 + 300 - 12) == INVALID


@pytest.mark.gpu
def test_arrays_side_by_side_and_scalars_just_behind_them():
    n = 300                                                 # 1200 bytes: a multiple of 16
    t = _make(n, 3)
    room = torch.full((4 * n + 8,), 7.0, device="cuda")
    for i, k in enumerate(("p", "m", "g", "v")):
        room[i * n:(i + 1) * n] = t[k]
        t[k] = room[i * n:(i + 1) * n]
    scalars = room[4 * n:4 * n + 2]
    scalars.copy_(torch.tensor([2e-3, 0.5]))
    before = _before(t)
    twell.adamw_step(twell.AdamWTensors([t]), step=3, lr_dev=scalars[:1], grad_scale=scalars[1:],
                     **dict(HYPER, lr=0.0))
    torch.cuda.synchronize()
    _check(t, before, 3, lr=float(np.float32(2e-3)), grad_scale=0.5)
    assert torch.equal(scalars, torch.tensor([2e-3, 0.5], device="cuda"))
    assert (room[4 * n + 2:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("p,g,master", [(torch.float32, torch.float32, False),
                                        (torch.bfloat16, torch.bfloat16, True)])
def test_captured_8_bit_steps_with_device_scalars_and_without_values(p, g, master):
    """The values are an aid: without them every other array gets the same bits."""
    sizes = (1, 257, 1000, 9000)
    with_v = [_make(n, 60 + i, 8, p, g, master, zero=i % 2 == 1) for i, n in enumerate(sizes)]
    plain = [{k: x.clone() if torch.is_tensor(x) else x for k, x in t.items()
              if not k.endswith("_values")} for t in with_v]
    step = torch.ones(1, dtype=torch.int32, device="cuda")
    lr, gs = torch.tensor([1e-3], device="cuda"), torch.tensor([1.0], device="cuda")
    kw = dict(HYPER, lr=0.0, step_dev=step, lr_dev=lr, grad_scale=gs)
    plans = twell.AdamWTensors(with_v), twell.AdamWTensors(plain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for plan in plans:
            twell.adamw_step(plan, **kw)
    for s, (r, scale) in enumerate(((1e-3, 1.0), (5e-4, 0.25), (2e-3, 2.0)), 1):
        step.fill_(s), lr.fill_(r), gs.fill_(scale)
        before = [_before(t) for t in with_v]
        graph.replay()
        torch.cuda.synchronize()
        for t, b, q in zip(with_v, before, plain):
            _check(t, b, s, lr=float(np.float32(r)), grad_scale=scale)
            for k, x in q.items():
                if torch.is_tensor(x):
                    assert torch.equal(x, t[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_give_the_bits_of_host_scalars(bits):
    """A step count past 2^16 and a learning rate that fp32 holds exactly."""
    a = [_make(n, 80 + n, bits) for n in (5, 3000)]
    b = [{k: x.clone() if torch.is_tensor(x) else x for k, x in t.items()} for t in a]
    for s in (1, 2, 1000, 100001):
        twell.adamw_step(twell.AdamWTensors(a), step=s, **dict(HYPER, lr=2.0 ** -9))
        twell.adamw_step(twell.AdamWTensors(b), step_dev=torch.full((1,), s, dtype=torch.int32,
                                                                    device="cuda"),
                         lr_dev=torch.full((1,), 2.0 ** -9, device="cuda"), **dict(HYPER, lr=0.0))
        torch.cuda.synchronize()
        for t, q in zip(a, b):
            for k, x in t.items():
                if torch.is_tensor(x):
                    assert torch.equal(x, q[k]), (s, k)
