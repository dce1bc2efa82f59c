"""Norms around a block at the ends of their range: empty batches, sizes that are refused."""
import pytest
import torch

from activation_sparse_transformer_tma_b200 import build as tw_build
from activation_sparse_transformer_tma_b200 import twell


@pytest.fixture(scope="module")
def L():
    tw_build.build()
    return twell.lib()


@pytest.mark.parametrize("group", [0, 1, 7, 2 ** 31 - 1])
def test_workspace_of_an_empty_batch_and_of_refused_sizes_is_empty(L, group):
    size = L.norm_residual_backward_workspace_size
    assert size(0, 64, group) == 0
    for T, d in ((-1, 64), (10, 0), (10, -8), (10, 60), (10, 8200), (10, 2 ** 31 - 8)):
        assert size(T, d, group) == 0, (T, d)
    assert size(10, 64, -1) == 0
    for T, d in ((1, 8), (10, 64), (2 ** 31 - 1, 8192)):
        # a partial row of each of the two vectors' gradients at least
        assert size(T, d, group) >= 2 * 4 * d, (T, d)


@pytest.mark.parametrize("group", [4, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63 - 1])
def test_a_group_past_32_bits_is_one_group(group):
    """Cut to 32 bits it would be another group: 2^32 + 1 a gate row per token, read past the one."""
    f = torch.float32
    b = twell._norm_block(4, 8, f, f, f, (None, torch.zeros(1, 8), None), (None, None, None), group,
                          1.0, 1.0, 0.0)
    assert b.gate_group >= 4
    assert (twell.norm_residual_backward_workspace_size(10, 64, group + 6) ==
            twell.norm_residual_backward_workspace_size(10, 64, 10))


def test_sizes_past_32_bits_are_refused():
    f = torch.float32
    big = 2 ** 32 + 1
    with pytest.raises(ValueError):
        twell._norm_block(big, 8, f, f, f, (None, None, None), (None, None, None), 0, 1.0, 1.0, 0.0)
    for sizes in ((big, 64, 64), (1, big, 64), (1, 64, big)):
        with pytest.raises(ValueError):
            twell.gated_ffn_workspace_size(*sizes)
        with pytest.raises(ValueError):
            twell.gated_ffn_backward_workspace_size(*sizes)
    with pytest.raises(ValueError):
        twell.norm_residual_backward_workspace_size(big, 64)
    some = twell.AdamWTensors([])
    some.count = 1
    with pytest.raises(ValueError):
        twell.adamw_step(some, lr=1e-3, step=2 ** 32 + 5)


@pytest.mark.gpu
def test_one_gate_row_for_a_group_past_32_bits():
    T, d = 5, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    y, r = (torch.randn(T, d, generator=g, device="cuda") for _ in range(2))
    gate = torch.randn(1, d, generator=g, device="cuda")
    outs = []
    for group in (T, 2 ** 32 + 1):
        out = torch.empty_like(r)
        twell.norm_residual_forward(y, r, None, gate, None, out, None, gate_group=group)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(*outs)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 1, 5])
def test_backward_of_an_empty_batch_with_the_workspace_it_asks_for(group):
    d = 72
    e = torch.empty((0, d), device="cuda")
    q = torch.empty(0, device="cuda")
    w = torch.ones(d, device="cuda")
    dw = torch.full((2, d), 7.0, device="cuda")
    ws = twell.norm_residual_backward_workspace(0, d, group)
    gate = e if group else None
    twell.norm_residual_backward(e, e, e, e, w, gate, w, q, q, e, e, dw[0],
                                 e.clone() if group else None, dw[1], ws, gate_group=group)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def _case(T, d, group, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    f = torch.float32
    c = dict(y=normal(T, d), r=normal(T, d, dtype=f), dn=normal(T, d), dr=normal(T, d, dtype=f),
             gate=normal(-(-T // group), d), w_post=normal(d), w_pre=normal(d))
    return c


def _both(c, group, over_dn=False):
    """All outputs of a forward and of the backward behind it."""
    T, d = c["r"].shape
    o = dict(r_out=torch.empty_like(c["r"]), n_out=torch.empty_like(c["y"]),
             p=torch.empty(T, device="cuda"), q=torch.empty(T, device="cuda"))
    twell.norm_residual_forward(c["y"], c["r"], c["w_post"], c["gate"], c["w_pre"], o["r_out"],
                                o["n_out"], gate_group=group, rstd_post=o["p"], rstd_pre=o["q"])
    dn = c["dn"].clone()
    o.update(dy=dn if over_dn else torch.empty_like(c["y"]), dr=torch.empty_like(c["r"]),
             dw_post=torch.empty(d, device="cuda"), dw_pre=torch.empty(d, device="cuda"),
             dgate=torch.empty(c["gate"].shape, device="cuda"))
    ws = twell.norm_residual_backward_workspace(T, d, group)
    ws.fill_(255)                                           # what a workspace held does not matter
    twell.norm_residual_backward(dn, c["dr"], c["y"], o["r_out"], c["w_post"], c["gate"],
                                 c["w_pre"], o["p"], o["q"], o["dy"], o["dr"], o["dw_post"],
                                 o["dgate"], o["dw_pre"], ws, gate_group=group)
    return o


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,group", [(9, 72, 1), (300, 264, 7), (1000, 2048, 300), (40, 8192, 40)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_token_that_is_not_finite_stays_alone(T, d, group, value):
    c = _case(T, d, group)
    want = _both(c, group)
    bad = T // 2
    rest = torch.arange(T, device="cuda") != bad
    groups = torch.arange(c["gate"].shape[0], device="cuda") != bad // group
    columns = torch.arange(d, device="cuda") != 5
    per_row = ("r_out", "n_out", "p", "q", "dy", "dr")
    for key in ("y", "r", "dn", "dr"):
        e = dict(c, **{key: c[key].clone()})
        e[key][bad, 5] = value
        got = _both(e, group)
        for k in per_row:
            assert torch.equal(got[k][rest], want[k][rest]), (key, k)
        assert torch.equal(got["dgate"][groups], want["dgate"][groups]), key
        assert not torch.isfinite(got["dr" if key != "y" else "dy"][bad]).all(), key
    # dn reaches the other columns of dw_pre through nothing
    e = dict(c, dn=c["dn"].clone())
    e["dn"][bad, 5] = value
    got = _both(e, group)
    assert torch.equal(got["dw_pre"][columns], want["dw_pre"][columns])
    assert not torch.isfinite(got["dw_pre"][5])


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,group", [(9, 72, 1), (700, 1000, 100), (40, 8192, 40)])
def test_dy_over_dn(T, d, group):
    c = _case(T, d, group, 1)
    apart, over = _both(c, group), _both(c, group, over_dn=True)
    for k in apart:
        assert torch.equal(apart[k], over[k]), k
