"""The operators around the FFN where offsets pass 32 bits: more than 2^32 elements in an array,
checked at both ends against calls on (or an fp64 computation of) the ends alone."""
import pytest
import torch

from activation_sparse_transformer_tma_b200 import twell

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _normal(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(generator=g).mul_(scale)


@pytest.fixture(autouse=True)
def _memory():
    free, _ = torch.cuda.mem_get_info()
    if free < 80 << 30:
        pytest.skip("80 GB of device memory are needed")
    yield
    torch.cuda.empty_cache()


def test_norms_of_more_than_2_32_elements():
    T, d, group = 2 ** 29 + 5, 8, 2 ** 20
    y, r, dn, dr_out = (_normal(i, T, d) for i in range(4))
    gate = _normal(4, -(-T // group), d)
    w_post, w_pre = _normal(5, d), _normal(6, d)
    p, q = (torch.empty(T, device="cuda") for _ in range(2))

    def forward(y, r, gate, p, q):
        r_out, n_out = torch.empty_like(r), torch.empty_like(r)
        twell.norm_residual_forward(y, r, w_post, gate, w_pre, r_out, n_out, gate_group=group,
                                    rstd_post=p, rstd_pre=q)
        return r_out, n_out

    r_out, n_out = forward(y, r, gate, p, q)
    last = (T // group) * group                             # the last gate row's tokens
    for at, rows in ((0, slice(0, group)), (T // group, slice(last, T))):
        n = rows.stop - rows.start
        pe, qe = (torch.empty(n, device="cuda") for _ in range(2))
        want = forward(y[rows], r[rows], gate[at:at + 1], pe, qe)
        assert torch.equal(r_out[rows], want[0]) and torch.equal(n_out[rows], want[1])
        assert torch.equal(p[rows], pe) and torch.equal(q[rows], qe)
    del n_out, r

    def backward(dn, dr_out, y, r_out, gate, p, q):
        n = y.shape[0]
        dy, dr = torch.empty_like(y), torch.empty_like(y)
        dw, dgate = torch.empty(2, d, device="cuda"), torch.empty(gate.shape, device="cuda")
        ws = twell.norm_residual_backward_workspace(n, d, group)
        twell.norm_residual_backward(dn, dr_out, y, r_out, w_post, gate, w_pre, p, q, dy, dr, dw[0],
                                     dgate, dw[1], ws, gate_group=group)
        return dy, dr, dgate

    dy, dr, dgate = backward(dn, dr_out, y, r_out, gate, p, q)
    for at, rows in ((0, slice(0, group)), (T // group, slice(last, T))):
        want = backward(dn[rows], dr_out[rows], y[rows], r_out[rows], gate[at:at + 1], p[rows],
                        q[rows])
        assert torch.equal(dy[rows], want[0]) and torch.equal(dr[rows], want[1])
        # the same terms in another order: n roundings of 2^-24 of their magnitudes at most
        n = rows.stop - rows.start
        k = (dr[rows].float() * y[rows].float() * p[rows][:, None] * w_post.float()).abs().sum(0)
        assert ((dgate[at] - want[2][0]).abs() <= 2 * n * 2.0 ** -24 * k + 1e-6).all()


def test_ffn_of_more_than_2_32_activations():
    T, d, F = 65800, 64, 65544                              # z, u, h: 4.31e9 elements each
    x, dy = _normal(0, T, d), _normal(1, T, d)
    Wg, Wu = (_normal(i, F, d, scale=d ** -0.5) for i in (2, 3))
    Wd = _normal(4, F, d, scale=F ** -0.5)
    z, u = (torch.empty((T, F), dtype=BF, device="cuda") for _ in range(2))
    y, dx = (torch.empty((T, d), device="cuda") for _ in range(2))
    dW = [torch.empty((F, d), device="cuda") for _ in range(3)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = twell.gated_ffn_workspace(T, d, F, training=True)
    twell.gated_ffn_forward(x, Wg, Wu, Wd, "silu", y, ws, z=z, u=u, dev_status=st)
    twell.gated_ffn_backward(x, dy, Wg, Wu, Wd, "silu", z, u, dx, *dW, ws, dev_status=st)
    assert int(st) == 0

    def near(got, want):
        # one operand rounded to bf16, independent over the terms: 2^-8 / sqrt(3) in the mean
        err = (got.double() - want).square().mean().sqrt()
        assert err <= 2.0 ** -8 * want.square().mean().sqrt()

    def act(z):
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))

    X, D, G, U, DN = (t.double() for t in (x, dy, Wg, Wu, Wd))
    for rows in (slice(0, 64), slice(T - 64, T)):           # tokens at both ends
        z64, u64 = X[rows] @ G.T, X[rows] @ U.T
        near(z[rows], z64)
        near(u[rows], u64)
        near(y[rows], (act(z64)[0] * u64) @ DN)
        a, da = act(z[rows].double())
        dh = D[rows] @ DN.T
        near(dx[rows], (dh * a) @ U + (dh * u[rows].double() * da) @ G)
    for units in (slice(0, 64), slice(F - 64, F)):          # units at both ends, over all tokens
        zu, uu = z[:, units].double(), u[:, units].double()
        a, da = act(zu)
        dh = D @ DN[units].T
        near(dW[0][units], (dh * uu * da).T @ X)
        near(dW[1][units], (dh * a).T @ X)
        near(dW[2][units], (a * uu).T @ D)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_more_than_2_32_elements(bits):
    n = 2 ** 32 + 300
    t = dict(p=_normal(0, n, scale=0.02), g=_normal(1, n, scale=1e-3), weight_decay=0.1)
    if bits == 32:
        t.update(m=_normal(2, n, scale=1e-4, dtype=torch.float32),
                 v=torch.full((n,), 1e-6, device="cuda"))
    else:
        nb = twell.adamw_blocks(n)
        t.update(m=torch.zeros(n, dtype=torch.int8, device="cuda"),
                 v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                 m_scale=torch.zeros(nb, device="cuda"), v_scale=torch.zeros(nb, device="cuda"))
    ends = []
    for first, last in ((0, 1024), (2 ** 32 - 512, n)):     # whole blocks of 256, and the tail
        ends.append((first, {
            k: x[first // 256:-(-last // 256)].clone() if k.endswith("_scale")
            else x[first:last].clone() if torch.is_tensor(x) else x for k, x in t.items()}))
    for step in (1, 2):
        twell.adamw_step(twell.AdamWTensors([t]), lr=1e-3, step=step)
        twell.adamw_step(twell.AdamWTensors([e for _, e in ends]), lr=1e-3, step=step)
    torch.cuda.synchronize()
    for first, e in ends:
        for k, x in e.items():
            if torch.is_tensor(x):
                at = first // 256 if k.endswith("_scale") else first
                assert torch.equal(t[k][at:at + x.numel()], x), (first, k)
