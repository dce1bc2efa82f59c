"""The operators as a layer uses them together: norms, FFN (dense gated, and the
sparse path), residual, their gradients and the AdamW step, against one fp64
computation of the whole; and two captured steps that share a workspace."""
import numpy as np
import pytest
import torch

from activation_sparse_transformer_tma_b200 import twell
from oracle import layer

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def _f64(t):
    return t.detach().double().cpu().numpy()


class Layer:
    """r1 = r + gate * norm(ffn(norm(r; w_in)); w_post), then the next block's norm."""

    def __init__(self, T, d, F, act, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * scale

        self.T, self.d, self.F, self.act = T, d, F, act
        self.master = {"Wg": normal(F, d, scale=d ** -0.5), "Wu": normal(F, d, scale=d ** -0.5),
                       "Wd": normal(F, d, scale=F ** -0.5)}
        self.vec = {"w_in": 1 + normal(d, scale=0.1), "w_post": 1 + normal(d, scale=0.1),
                    "gate": normal(d, scale=0.5), "w_next": 1 + normal(d, scale=0.1)}
        self.w = {k: v.to(BF) for k, v in self.master.items()}
        self.r, self.dn = normal(T, d), normal(T, d).to(BF)
        self.dr = normal(T, d)

        def empty(*shape, dtype=F32):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.x, self.y, self.n = (empty(T, d, dtype=BF) for _ in range(3))
        self.r1, self.dr0, self.dr_in = (empty(T, d) for _ in range(3))
        self.z, self.u = (empty(T, F, dtype=BF) for _ in range(2))
        self.dy, self.dx = (empty(T, d, dtype=BF) for _ in range(2))
        self.rs = [empty(T) for _ in range(3)]
        self.grad = {k: torch.zeros_like(v) for k, v in {**self.master, **self.vec}.items()}
        self.ws = twell.gated_ffn_workspace(T, d, F, training=True)
        self.nws = twell.norm_residual_backward_workspace(T, d, T)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tensors = [dict(p=self.w[k], master=self.master[k], g=self.grad[k],
                        m=torch.zeros(F * d, dtype=torch.int8, device="cuda"),
                        v=torch.zeros(F * d, dtype=torch.uint8, device="cuda"),
                        m_scale=torch.zeros(twell.adamw_blocks(F * d), device="cuda"),
                        v_scale=torch.zeros(twell.adamw_blocks(F * d), device="cuda"),
                        weight_decay=0.1) for k in self.w]
        tensors += [dict(p=v, g=self.grad[k], m=torch.zeros_like(v), v=torch.zeros_like(v))
                    for k, v in self.vec.items()]
        self.plan = twell.AdamWTensors(tensors)
        self.step = torch.ones(1, dtype=torch.int32, device="cuda")

    def forward_backward(self):
        t, v, g = twell, self.vec, self.grad
        t.norm_residual_forward(None, self.r, None, None, v["w_in"], None, self.x, eps=EPS,
                                rstd_pre=self.rs[0])
        t.gated_ffn_forward(self.x, self.w["Wg"], self.w["Wu"], self.w["Wd"], self.act, self.y,
                            self.ws, z=self.z, u=self.u, dev_status=self.status)
        t.norm_residual_forward(self.y, self.r, v["w_post"], v["gate"], v["w_next"], self.r1, self.n,
                                gate_group=self.T, eps=EPS, rstd_post=self.rs[1],
                                rstd_pre=self.rs[2])
        t.norm_residual_backward(self.dn, self.dr, self.y, self.r1, v["w_post"], v["gate"],
                                 v["w_next"], self.rs[1], self.rs[2], self.dy, self.dr0,
                                 g["w_post"], g["gate"], g["w_next"], self.nws, gate_group=self.T)
        t.gated_ffn_backward(self.x, self.dy, self.w["Wg"], self.w["Wu"], self.w["Wd"], self.act,
                             self.z, self.u, self.dx, g["Wg"], g["Wu"], g["Wd"], self.ws,
                             dev_status=self.status)
        t.norm_residual_backward(self.dx, self.dr0, None, self.r, None, None, v["w_in"], None,
                                 self.rs[0], None, self.dr_in, None, None, g["w_in"], self.nws)

    def update(self, **kw):
        twell.adamw_step(self.plan, lr=1e-3, **kw)


def _whole(L):
    """The same in one fp64 graph: r1, n, and all gradients."""
    t = {k: torch.tensor(_f64(v), requires_grad=True) for k, v in {**L.w, **L.vec, "r": L.r}.items()}
    f = {"relu": torch.relu, "silu": torch.nn.functional.silu}[L.act]

    def norm(v):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)

    x = norm(t["r"]) * t["w_in"]
    y = (f(x @ t["Wg"].T) * (x @ t["Wu"].T)) @ t["Wd"]
    r1 = t["r"] + t["gate"] * (norm(y) * t["w_post"])
    n = norm(r1) * t["w_next"]
    ((n * torch.tensor(_f64(L.dn))).sum() + (r1 * torch.tensor(_f64(L.dr))).sum()).backward()
    return r1.detach().numpy(), n.detach().numpy(), {k: v.grad.numpy() for k, v in t.items()}


def _rel(got, want):
    return np.linalg.norm(_f64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("T,d,F,act", [(37, 128, 264, "silu"), (300, 256, 520, "silu"),
                                       (130, 64, 128, "relu")])
def test_a_layer_trains_one_step(T, d, F, act):
    L = Layer(T, d, F, act, T)
    r1, n, grads = _whole(L)
    L.forward_backward()
    torch.cuda.synchronize()
    assert int(L.status) == 0
    # x, z, u, h, y, dy, du, dz, dx and the gradients' operands are bf16: at most a dozen
    # independent roundings of 2^-8 half-steps on a path, each 2^-9 in the mean
    tol = 12 * 2.0 ** -8
    assert _rel(L.r1, r1) < tol and _rel(L.n, n) < tol
    assert _rel(L.dr_in, grads["r"]) < tol
    for k in L.grad:
        assert _rel(L.grad[k], grads[k]) < (2 * tol if act == "relu" else tol), k
    before = {k: _f64(v) for k, v in {**L.master, **L.vec}.items()}
    L.update(step=1)
    torch.cuda.synchronize()
    for k, p in {**L.master, **L.vec}.items():
        want, _, _, _ = layer.adamw(before[k], _f64(L.grad[k]), 0.0, 0.0, lr=1e-3, beta1=0.9,
                                    beta2=0.999, eps=1e-8, step=1,
                                    weight_decay=0.1 if k in L.w else 0.0)
        # the first step moves by lr; 2^-20 covers the update's roundings
        assert np.all(np.abs(_f64(p) - want) <= 2.0 ** -24 * 3 * np.abs(want) + 1e-3 * 2.0 ** -20)
        if k in L.w:
            assert torch.equal(L.w[k], p.to(BF))


def test_norms_around_the_sparse_ffn():
    """The sparse path takes the norm's output as it is, and its y and dx feed the norms."""
    T, d, F, C_h = 200, 256, 512, 64
    L = Layer(T, d, F, "relu", 3)
    st = L.status
    twell.norm_residual_forward(None, L.r, None, None, L.vec["w_in"], None, L.x, eps=EPS,
                                rstd_pre=L.rs[0])
    g = twell.Twell(T, F, 128)
    hy = twell.Hybrid(T, F, C_h, backup_cap=T)
    y = torch.empty((T, d), device="cuda")
    twell.twell_gate_gemm(L.x, L.w["Wg"], g, dev_status=st)
    twell.twell_to_hybrid(g, hy, dev_status=st)
    twell.hybrid_ffn_forward(L.x, hy, L.w["Wu"], L.w["Wd"], y, dev_status=st)
    twell.norm_residual_forward(y, L.r, L.vec["w_post"], L.vec["gate"], L.vec["w_next"], L.r1, L.n,
                                gate_group=T, eps=EPS, rstd_post=L.rs[1], rstd_pre=L.rs[2])
    dy = torch.empty((T, d), device="cuda")
    twell.norm_residual_backward(L.dn, L.dr, y, L.r1, L.vec["w_post"], L.vec["gate"],
                                 L.vec["w_next"], L.rs[1], L.rs[2], dy, L.dr0, L.grad["w_post"],
                                 L.grad["gate"], L.grad["w_next"], L.nws, gate_group=T)
    ws = torch.empty(twell.hybrid_ffn_backward_workspace_size(T, d, F, C_h, T), dtype=torch.uint8,
                     device="cuda")
    dx = torch.empty((T, d), device="cuda")
    twell.hybrid_ffn_backward(L.x, dy.to(BF), hy, L.w["Wg"], L.w["Wu"], L.w["Wd"], 0.0, dx,
                              L.grad["Wg"], L.grad["Wu"], L.grad["Wd"], ws, dev_status=st)
    twell.norm_residual_backward(dx, L.dr0, None, L.r, None, None, L.vec["w_in"], None, L.rs[0],
                                 None, L.dr_in, None, None, L.grad["w_in"], L.nws)
    torch.cuda.synchronize()
    assert int(st) == 0
    r1, n, grads = _whole(L)
    # as above; a gate that rounding takes across zero changes whole terms, so twice as wide
    tol = 24 * 2.0 ** -8
    assert _rel(L.r1, r1) < tol and _rel(L.n, n) < tol and _rel(L.dr_in, grads["r"]) < tol
    for k in L.grad:
        assert _rel(L.grad[k], grads[k]) < tol, k


def test_captured_steps_replay_with_new_inputs():
    """A whole step captured once: replays with other inputs equal eager steps bit for bit, and
    an eager step of another layer between them changes nothing."""
    A, B, other = (Layer(150, 128, 256, "silu", 7) for _ in range(3))
    graph = torch.cuda.CUDAGraph()
    A.forward_backward()                    # loads modules before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        A.forward_backward()
        A.update(step_dev=A.step)
    for s in range(1, 4):
        g = torch.Generator(device="cuda")
        g.manual_seed(100 + s)
        r = torch.randn(150, 128, generator=g, device="cuda")
        A.r.copy_(r), B.r.copy_(r)
        A.step.fill_(s)
        graph.replay()
        other.forward_backward()
        B.forward_backward()
        B.update(step_dev=B.step.fill_(s))
        torch.cuda.synchronize()
        for k in A.grad:
            assert torch.equal(A.grad[k], B.grad[k]), k
        for k in A.master:
            assert torch.equal(A.master[k], B.master[k]) and torch.equal(A.w[k], B.w[k])
        for k in A.vec:
            assert torch.equal(A.vec[k], B.vec[k])


@pytest.mark.parametrize("T", [1, 20, 112, 113, 300])
def test_calls_queued_back_to_back_equal_separate_ones(T):
    """Optimiser steps, forwards and backwards on shared workspaces, nothing waiting between them:
    each call sees the weights that the step before it wrote, bit for bit as with a wait after
    every call."""
    def run(wait):
        L = Layer(T, 256, 512, "silu", 11)
        out = []
        for s in range(1, 5):
            L.forward_backward()
            out += [t.clone() for t in (L.y, L.n, L.dr_in, *L.grad.values())]
            L.update(step=s)
            if wait:
                torch.cuda.synchronize()
            twell.gated_ffn_forward(L.x, L.w["Wg"], L.w["Wu"], L.w["Wd"], L.act, L.y, L.ws)
            out.append(L.y.clone())
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert int(L.status) == 0
        return out + [v.clone() for v in L.w.values()]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 100])
def test_few_tokens_captured_with_an_optimiser_step_between(T):
    """The few-token kernels read a weight before the kernel in front of them has ended: not
    before the optimiser step that wrote it."""
    A, B = (Layer(T, 256, 1024, "gelu_tanh" if T == 3 else "relu", 5) for _ in range(2))

    def steps(L):
        for _ in range(3):
            L.forward_backward()
            L.update(step_dev=L.step)
            twell.gated_ffn_forward(L.x, L.w["Wg"], L.w["Wu"], L.w["Wd"], L.act, L.y, L.ws)

    steps(B)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps(A)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(A.y, B.y)
    for k in A.w:
        assert torch.equal(A.w[k], B.w[k])


def test_two_streams_with_workspaces_of_their_own():
    A, B, C, D = (Layer(T, 128, 256, "silu", T) for T in (40, 200, 40, 200))
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for L, s in zip((A, B), streams):
            with torch.cuda.stream(s):
                L.forward_backward()
    torch.cuda.synchronize()
    C.forward_backward(), D.forward_backward()
    torch.cuda.synchronize()
    for L, M in ((A, C), (B, D)):
        assert torch.equal(L.n, M.n) and all(torch.equal(L.grad[k], M.grad[k]) for k in L.grad)
