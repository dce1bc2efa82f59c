"""Dense gated FFN: the kernels' waits are bounded.  With the operands' loads withheld (a test aid)
every wait for them runs out after its short limit, the status word says so, nothing is written,
and the next call is as right as ever."""
import time

import pytest
import torch

from activation_sparse_transformer_tma_b200 import twell

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LIMIT_NS = 20_000_000


class Case:
    def __init__(self, T, d, F):
        g = torch.Generator(device="cuda")
        g.manual_seed(T)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)

        self.T, self.d, self.F = T, d, F
        self.x, self.dy = normal(T, d), normal(T, d)
        self.W = [normal(F, d, scale=d ** -0.5) for _ in range(3)]
        self.ws = twell.gated_ffn_workspace(T, d, F, training=True)

    def outputs(self):
        def full(*shape):
            return torch.full(shape, 7.0, dtype=BF, device="cuda")

        T, d, F = self.T, self.d, self.F
        return full(T, d), full(T, F), full(T, F), full(T, d), [full(F, d) for _ in range(3)]

    def forward(self, y, z, u, st):
        twell.gated_ffn_forward(self.x, *self.W, "gelu", y, self.ws, z=z, u=u, dev_status=st)

    def backward(self, z, u, dx, dW, st):
        twell.gated_ffn_backward(self.x, self.dy, *self.W, "gelu", z, u, dx, *dW, self.ws,
                                 dev_status=st)


def _withheld(call):
    """Runs the call with its loads withheld; its status bits."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    twell.lib().tw_test_withhold_next_gated_ffn_loads(LIMIT_NS)
    t0 = time.perf_counter()
    call(st)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 2.0
    return twell.status_bits(st)


# few tokens (with and without a divided reduction); tiles with divided reductions; dx and the
# weight gradients in one launch and apart; several tiles a pair
@pytest.mark.parametrize("T,d,F", [(20, 256, 512), (100, 1096, 264), (300, 256, 520),
                                   (1024, 1536, 1032), (2100, 1280, 640)])
def test_waits_run_out_and_the_next_call_is_right(T, d, F):
    c = Case(T, d, F)
    y, z, u, dx, dW = c.outputs()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.forward(y, z, u, st)
    c.backward(z, u, dx, dW, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    y1, z1, u1, dx1, dW1 = c.outputs()
    assert "TW_ERR_TIMEOUT" in _withheld(lambda s: c.forward(y1, z1, u1, s))
    assert all((t == 7).all() for t in (y1, z1, u1))
    assert "TW_ERR_TIMEOUT" in _withheld(lambda s: c.backward(z, u, dx1, dW1, s))
    assert all((t == 7).all() for t in (dx1, *dW1))
    c.forward(y1, z1, u1, st)
    c.backward(z1, u1, dx1, dW1, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for got, want in zip((y1, z1, u1, dx1, *dW1), (y, z, u, dx, *dW)):
        assert torch.equal(got, want)
