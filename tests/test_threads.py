"""Calls from other host threads: one whose first CUDA call is the library's, and two at once."""
import threading

import pytest
import torch

from activation_sparse_transformer_tma_b200 import twell

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _in_thread(*calls):
    """Runs each call in a thread of its own, all at once; raises what they raised."""
    errors = []

    def run(f):
        try:
            f()
        except Exception as e:                              # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


class Step:
    """Forward and backward of the dense gated FFN and of the norms, and an AdamW step."""

    def __init__(self, T, seed, d=256, F=512):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.x, self.dn = normal(T, d), normal(T, d)
        self.r = normal(T, d).float()
        self.W = [normal(F, d, scale=d ** -0.5) for _ in range(3)]
        self.w = normal(d)
        self.y, self.n, self.dy, self.dx = (empty(T, d, dtype=BF) for _ in range(4))
        self.z, self.u = (empty(T, F, dtype=BF) for _ in range(2))
        self.r1, self.dr = empty(T, d), empty(T, d)
        self.p, self.q = empty(T), empty(T)
        self.dw, self.dW = empty(2, d), [empty(F, d) for _ in range(3)]
        self.ws = twell.gated_ffn_workspace(T, d, F, training=True)
        self.nws = twell.norm_residual_backward_workspace(T, d)
        self.plan = twell.AdamWTensors([dict(p=p, g=g, m=torch.zeros_like(g), v=torch.zeros_like(g))
                                        for p, g in zip(self.W, self.dW)])

    def run(self, stream=None, steps=1):
        for s in range(1, steps + 1):
            twell.gated_ffn_forward(self.x, *self.W, "silu", self.y, self.ws, z=self.z, u=self.u,
                                    stream=stream)
            twell.norm_residual_forward(self.y, self.r, self.w, None, self.w, self.r1, self.n,
                                        rstd_post=self.p, rstd_pre=self.q, stream=stream)
            twell.norm_residual_backward(self.dn, self.r, self.y, self.r1, self.w, None, self.w,
                                         self.p, self.q, self.dy, self.dr, self.dw[0], None,
                                         self.dw[1], self.nws, stream=stream)
            twell.gated_ffn_backward(self.x, self.dy, *self.W, "silu", self.z, self.u, self.dx,
                                     *self.dW, self.ws, stream=stream)
            twell.adamw_step(self.plan, lr=1e-3, step=s, stream=stream)

    def results(self):
        return [self.y, self.n, self.r1, self.dy, self.dr, self.dw, self.dx, *self.dW, *self.W]


@pytest.mark.parametrize("T", [20, 300])
def test_first_cuda_call_of_a_thread(T):
    """No runtime call has bound the device's context in the new thread yet."""
    a, b = Step(T, 1), Step(T, 1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    _in_thread(lambda: a.run(s))
    b.run()
    torch.cuda.synchronize()
    for got, want in zip(a.results(), b.results()):
        assert torch.equal(got, want)


def test_first_cuda_call_of_a_thread_is_the_backward_or_the_gate():
    a, s = Step(300, 2), torch.cuda.Stream()
    g = twell.Twell(300, 512, 32)
    a.run()
    torch.cuda.synchronize()
    _in_thread(lambda: twell.gated_ffn_backward(a.x, a.dy, *a.W, "silu", a.z, a.u, a.dx, *a.dW, a.ws,
                                                stream=s))
    _in_thread(lambda: twell.twell_gate_gemm(a.x, a.W[0], g, stream=s))
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [20, 300])
def test_two_threads_at_once(T):
    """Each on a stream, workspaces and tensors of its own: the bits of one after the other."""
    a, b, c, d = (Step(T, seed) for seed in (1, 2, 1, 2))
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    _in_thread(lambda: a.run(streams[0], 50), lambda: b.run(streams[1], 50))
    c.run(steps=50)
    d.run(steps=50)
    torch.cuda.synchronize()
    for one, other in ((a, c), (b, d)):
        for got, want in zip(one.results(), other.results()):
            assert torch.equal(got, want)
