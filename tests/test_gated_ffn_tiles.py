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


# On 148 SMs (74 pairs), in tiles of gate-up, y, dh and dx:
#   (2100, 2568, 2608)  189, 99, 99, 99: several a pair in all four products, nine tile rows, whole
#                       and halved tiles of y and dx, dx and the weight gradients apart
#   (2100, 1280, 640)   45, 45, 27, 45: whole tiles alone, one a pair, dx apart
#   (5000, 136, 1032)   180, 40 halves, 100, 40 halves: several a pair, twenty tile rows
#   (3000, 264, 2104)   204, 48, 108, 48: halves, and weight gradients by pairs that had a tile of dx
#   (260, 4104, 1032)   18, 68, 10, 68: wide rows, weight gradients whole and halved
STEPS = [(2100, 2568, 2608), (2100, 1280, 640), (5000, 136, 1032), (3000, 264, 2104),
         (260, 4104, 1032)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,F", STEPS)
def test_steps_of_many_tiles(T, d, F):
    a = _inputs(T, d, F, T + d * F)
    x, dy, Wg, Wu, Wd = a
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    X, _, G, U, D = (t.double() for t in a)
    z64, u64 = X @ G.T, X @ U.T
    y64 = (_silu(z64)[0] * u64) @ D
    want = None
    for dtype in (BF, F32):
        z, u = (torch.full((T + 1, F), 7.0, dtype=BF, device="cuda") for _ in range(2))
        y, y0 = (torch.full((T + 1, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        twell.gated_ffn_forward(x, Wg, Wu, Wd, "silu", y0[:T], ws, dev_status=st)
        ws.fill_(255)                                       # what a workspace held does not matter
        twell.gated_ffn_forward(x, Wg, Wu, Wd, "silu", y[:T], ws, z=z[:T], u=u[:T], dev_status=st)
        assert torch.equal(y, y0)
        for name, got, exact in (("z", z, z64), ("u", u, u64), ("y", y, y64)):
            assert (got[T:] == 7).all()
            _near(name, got[:T], exact)
        if want is None:
            want = _gradients(a, z[:T], u[:T])
        for dw_dtype in (BF, F32):
            dx = torch.full((T + 1, d), 7.0, dtype=dtype, device="cuda")
            dW = [torch.full((F + 1, d), 7.0, dtype=dw_dtype, device="cuda") for _ in range(3)]
            ws.fill_(255)
            _backward(a, "silu", z[:T], u[:T], dx[:T], [w[:F] for w in dW], ws, st)
            assert (dx[T:] == 7).all() and all((w[F:] == 7).all() for w in dW)
            _near("dx", dx[:T], want[0])
            for k in range(3):
                _near(("dWg", "dWu", "dWd")[k], dW[k][:F], want[1][k])
    assert int(st) == 0


# one token's NaN or infinity: few tokens, tiles, divided reductions, several tiles a pair
@pytest.mark.gpu
@pytest.mark.parametrize("T,d,F", [(40, 264, 520), (300, 264, 1032), (130, 512, 4096),
                                   (2100, 520, 1032)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_token_that_is_not_finite_stays_alone(T, d, F, value):
    a = _inputs(T, d, F, 3 * T)
    x, dy, Wg, Wu, Wd = a
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    bad, rest = T - 3, torch.arange(T, device="cuda") != T - 3

    def step(x, dy, z=None, u=None):
        y, dx = (torch.empty((T, d), device="cuda") for _ in range(2))
        dW = [torch.empty((F, d), device="cuda") for _ in range(3)]
        if z is None:
            z, u = (torch.empty((T, F), dtype=BF, device="cuda") for _ in range(2))
            twell.gated_ffn_forward(x, Wg, Wu, Wd, "silu", y, ws, z=z, u=u)
        _backward((x, dy, Wg, Wu, Wd), "silu", z, u, dx, dW, ws, None)
        return y, z, u, dx, dW

    y, z, u, dx, dW = step(x, dy)
    xn = x.clone()
    xn[bad, 5] = value
    yn, zn, un, dxn, _ = step(xn, dy)
    for got, want in ((yn, y), (zn, z), (un, u), (dxn, dx)):
        assert torch.equal(got[rest], want[rest])
    assert not torch.isfinite(yn[bad]).any()
    dyn = dy.clone()
    dyn[bad, 7] = value
    _, _, _, dxn, dWn = step(x, dyn, z, u)
    assert torch.equal(dxn[rest], dx[rest]) and not torch.isfinite(dxn[bad]).any()
    col = torch.arange(d, device="cuda") != 7
    assert torch.equal(dWn[2][:, col], dW[2][:, col])       # dWd: that column of dy alone
    assert not torch.isfinite(dWn[2][:, 7]).any()
