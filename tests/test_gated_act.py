"""Activations of the dense gated FFN and their derivatives, value by value, read out of the
kernels through identity weights, against fp64.

Tolerances.  u and dh are 1, products with one term are exact, so h, du and dz are act(z) and
act'(z), evaluated in fp32 and rounded once (half a bf16 step, 2^-8).  In fp32 the relative
error of act for |z| <= 9 is that of its sigmoid or normal distribution.  SiLU: 12 steps of
2^-23 for exp(9), 2 for the division.  GELU (tanh): exp's argument goes to 66, is off by 4
roundings (66 * 4 * 2^-24 = 2^-16) and exp itself by 79 steps (2^-16.7).  GELU:
exp(-z^2 / 2) has an argument to 41, off by 2 roundings (2^-17.6), and 49 steps of its own
(2^-17.4); the factor beside it is off by 2^-20.  All are below 2^-14.
Derivatives for z <= -3 are a multiple of the same factor or of exp(-z^2 / 2) (off by
2^-16.5), and their second term takes off at most an eighth: below 2^-13.  Above -3 they are
off by (1 + z^2) 2^-18.
"""
import numpy as np
import pytest
import torch

from scipy.special import expit, ndtr

from activation_sparse_transformer_tma_b200 import twell

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H = 2.0 ** -8
ACTS = ["relu", "silu", "gelu", "gelu_tanh"]


def _f64(t):
    return t.detach().double().cpu().numpy()


def _exact(act, z):
    """act and act' in fp64 without a difference of nearly equal numbers: 1 + tanh(k), for
    instance, has no digit left at z = -9, where it is 2e-29."""
    if act == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if act == "gelu":
        return z * ndtr(z), ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    k2, dk2 = z, 1.0
    if act == "gelu_tanh":                                  # 0.5 (1 + tanh(k)) = expit(2k)
        c = np.sqrt(8 / np.pi)
        k2, dk2 = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
    return z * expit(k2), expit(k2) + z * expit(k2) * expit(-k2) * dk2


def _grid(T, F, lo, hi):
    """bf16 values from lo to hi, the F columns' steps subdivided by the T rows."""
    z = lo + (hi - lo) * (np.arange(F)[None, :] + np.arange(T)[:, None] / T) / F
    return torch.tensor(z, device="cuda").to(BF)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [1, 48, 200])
def test_activations_value_by_value(T, act):
    """T up to 112 by the kernels for few tokens, above by those for many."""
    d = F = 512
    ws = twell.gated_ffn_workspace(T, d, F)
    eye = torch.eye(F, d, device="cuda").to(BF)
    for lo, hi in ((-9.0, -3.0), (-3.0, 9.0)):
        # z[t, j] = c[t] w[j] exactly: both factors have 8 bits
        c = torch.linspace(1.0, 1.25, T, device="cuda").to(BF)
        w = torch.linspace(lo, hi / 1.25 if hi > 0 else hi, F, device="cuda").to(BF)
        w = torch.clamp(w.float(), min=-9.0 / 1.25).to(BF)
        x = torch.zeros(T, d, device="cuda", dtype=BF)
        x[:, 0], x[:, 1] = c, 1.0
        Wg, Wu = (torch.zeros(F, d, device="cuda", dtype=BF) for _ in range(2))
        Wg[:, 0], Wu[:, 1] = w, 1.0
        y = torch.empty(T, d, device="cuda")
        twell.gated_ffn_forward(x, Wg, Wu, eye, act, y, ws)
        z = _f64(c)[:, None] * _f64(w)[None, :]
        want = _exact(act, z)[0]
        err = np.abs(_f64(y) - want) - (H + 2.0 ** -14) * np.abs(want)
        assert err.max() <= 0, z[np.unravel_index(err.argmax(), err.shape)]


@pytest.mark.parametrize("act", ACTS)
def test_derivatives_value_by_value(act):
    T, d, F = 200, 512, 512
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    eye = torch.eye(F, d, device="cuda").to(BF)
    x = torch.eye(T, d, device="cuda").to(BF)              # dW[j, t] is the factor of token t
    one = torch.ones(T, d, device="cuda").to(BF)
    for lo, hi in ((-9.0, -3.0), (-3.0, 9.0)):
        z = _grid(T, F, lo, hi)
        u = torch.ones(T, F, device="cuda").to(BF)
        dx = torch.empty(T, d, device="cuda")
        dWg, dWu, dWd = (torch.empty(F, d, device="cuda") for _ in range(3))
        twell.gated_ffn_backward(x, one, eye, eye, eye, act, z, u, dx, dWg, dWu, dWd, ws)
        a, da = _exact(act, _f64(z))
        got_du, got_dz = _f64(dWu)[:, :T].T, _f64(dWg)[:, :T].T
        assert (np.abs(got_du - a) - (H + 2.0 ** -14) * np.abs(a)).max() <= 0
        if hi <= -3.0:
            tol = (H + 2.0 ** -13) * np.abs(da)
        else:
            tol = H * np.abs(da) + (1 + _f64(z) ** 2) * 2.0 ** -18
        assert (np.abs(got_dz - da) - tol).max() <= 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [40, 200])
def test_gates_far_out_saturate(act, T):
    """z^2 passes fp32's range: act is z or 0 and act' 1 or 0, not a product of 0 and infinity."""
    d = F = 256
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    far = torch.tensor([1e3, 1e10, 1e19, 1e20, 3e38, -1e3, -1e10, -1e19, -1e20, -3e38],
                       device="cuda").repeat(F // 10 + 1)[:F].to(BF)
    eye = torch.eye(F, d, device="cuda").to(BF)
    x = torch.zeros(T, d, device="cuda", dtype=BF)
    x[:, 0], x[:, 1] = 1.0, 1.0
    Wg, Wu = (torch.zeros(F, d, device="cuda", dtype=BF) for _ in range(2))
    Wg[:, 0], Wu[:, 1] = far, 1.0
    y = torch.empty(T, d, device="cuda")
    twell.gated_ffn_forward(x, Wg, Wu, eye, act, y, ws)
    a, da = _exact(act, _f64(far))
    assert np.array_equal(_f64(y), np.broadcast_to(a, (T, d)))
    z, u = far.repeat(T, 1), torch.ones(T, F, device="cuda").to(BF)
    one = torch.ones(T, d, device="cuda").to(BF)
    x = torch.eye(T, d, device="cuda").to(BF)
    dx = torch.empty(T, d, device="cuda")
    dWg, dWu, dWd = (torch.empty(F, d, device="cuda") for _ in range(3))
    twell.gated_ffn_backward(x, one, eye, eye, eye, act, z, u, dx, dWg, dWu, dWd, ws)
    assert np.array_equal(_f64(dWg)[:, :T].T, np.broadcast_to(da, (T, F)))
    assert np.array_equal(_f64(dWu)[:, :T].T, np.broadcast_to(a, (T, F)))
