"""Dense gated FFN over many tiles: several tiles a pair of CTAs, whole and half-width tiles
in one launch, dx and the weight gradients in one launch and apart, against a plain fp64
computation on the GPU.

Tolerances.  With about normal inputs, errors of elements are sums of many independent
roundings, each of at most half a bf16 step, 2^-8 of the value and far less in the mean
(2^-8 / sqrt(3) where the value's mantissa is uniform).  y rounds h and itself; the
gradients, computed from the kept z and u, round one operand of each product and the result.
That is at most sqrt(2) 2^-8 / sqrt(3) = 0.82 2^-8 of a matrix's root mean square, fp32 sums
adding less than 2^-14.  Over 32 x 32 elements the mean square of independent errors strays
by a few in a hundred, and that of the values by as much: 2 * 2^-8 is twice what a patch can
be off, and one element that is wrong by its own size puts 1/32 = 8 * 2^-8 into its patch.
"""
import numpy as np
import pytest
import torch

from activation_sparse_transformer_tma_b200 import twell

BF, F32 = torch.bfloat16, torch.float32
H = 2.0 ** -8


def _inputs(T, d, F, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)

    return (normal(T, d), normal(T, d), normal(F, d, scale=2 * d ** -0.5),
            normal(F, d, scale=d ** -0.5), normal(F, d, scale=F ** -0.5))


def _silu(z):
    p = torch.sigmoid(z)
    return z * p, p * (1 + z * (1 - p))


def _patches(e):
    """Root mean square of each 32 x 32 patch (those at the ends over what exists of them)."""
    T, d = e.shape
    full = torch.zeros(-(-T // 32) * 32, -(-d // 32) * 32, dtype=e.dtype, device=e.device)
    full[:T, :d] = e.square()
    ones = torch.zeros_like(full)
    ones[:T, :d] = 1

    def total(v):
        return v.view(v.shape[0] // 32, 32, -1, 32).sum((1, 3))

    return (total(full) / total(ones)).sqrt(), total(ones)


def _near(name, got, want):
    err, n = _patches(got.double() - want)
    # a patch of few elements strays further: 4 standard deviations of a mean of n squares
    limit = 2 * H * want.square().mean().sqrt() * (1 + 4 * (2 / n).sqrt())
    worst = (err / limit).max()
    assert worst <= 1, (name, float(worst))


def _backward(a, act, z, u, dx, dW, ws, st):
    x, dy, Wg, Wu, Wd = a
    twell.gated_ffn_backward(x, dy, Wg, Wu, Wd, act, z, u, dx, *dW, ws, dev_status=st)


def _gradients(a, z, u):
    x, dy, Wg, Wu, Wd = (t.double() for t in a)
    z, u = z.double(), u.double()
    act, der = _silu(z)
    dh = dy @ Wd.T
    du, dz = dh * act, dh * u * der
    return du @ Wu + dz @ Wg, [dz.T @ x, du.T @ x, (act * u).T @ dy]


# dx of few tiles and undivided, then weight gradients by the same pairs of CTAs
@pytest.mark.gpu
@pytest.mark.parametrize("T,d,F", [(64, 4096, 384), (64, 8192, 512), (260, 4104, 1032),
                                   (400, 4608, 264), (1024, 1536, 4096)])
def test_dx_and_weight_gradients_of_different_types_in_one_launch(T, d, F):
    a = _inputs(T, d, F, T + d + F)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    z, u = (torch.randn(T, F, generator=g, device="cuda").to(BF) for _ in range(2))
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(xt, wt):
        dx = torch.full((T, d), 7.0, dtype=xt, device="cuda")
        dW = [torch.full((F, d), 7.0, dtype=wt, device="cuda") for _ in range(3)]
        _backward(a, "silu", z, u, dx, dW, ws, st)
        return dx, dW

    dx32, dW32 = step(F32, F32)
    dx16, dW16 = step(BF, BF)
    want_dx, want_dW = _gradients(a, z, u)
    for dx, dW in ((dx32, dW32), (dx16, dW16)):
        _near("dx", dx, want_dx)
        for k in range(3):
            _near(k, dW[k], want_dW[k])
    for _ in range(10):
        for xt, wt in ((F32, BF), (BF, F32)):
            dx, dW = step(xt, wt)
            assert torch.equal(dx, dx32 if xt == F32 else dx16)
            for got, want in zip(dW, dW32 if wt == F32 else dW16):
                assert torch.equal(got, want)
    assert int(st) == 0
