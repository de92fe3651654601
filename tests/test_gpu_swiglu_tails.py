"""The gated activation where exp(-gate) is very large or very small, against 64 bits.

With U = 2^-24: the sigmoid's exponent is reduced to within 2^-25 (0.35 U of the power), the power is
off by 2 U, the sum and the reciprocal by U each, in all below 5 U, and by half of binary32's least
magnitude, 2^-150, where it falls below the normal numbers; the two products after it by U each.
"""
import pytest
import torch

from tests.expert_common import assert_within, half_step, torch_dtype
from tests.layer_common import U
from tests.test_gpu_few import WEIGHTS
from tests.test_gpu_few_exact import Exact

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
LEAST = 2.0 ** -149


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


def _gates(dtype):
    g = torch.linspace(-112, 40, 64 * 256, dtype=torch.float64, device=DEV).to(torch_dtype(dtype))
    ends = torch.tensor([-1e30, -3e38, 3e38, 1e30, 0.0, -0.0, 1e-38, -1e-38], device=DEV).to(g.dtype)
    g[:8] = ends
    return g.view(64, 256)


@pytest.mark.parametrize("up", [1.0, 2.0 ** 40, -2.0 ** 80])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu(td, dtype, up):
    g = _gates(dtype)
    u = torch.full_like(g, up)
    y = torch.empty_like(g)
    td.moonep_swiglu(g, u, y)
    want = g.double() * torch.sigmoid(g.double()) * up
    least = torch.finfo(y.dtype).tiny * torch.finfo(y.dtype).eps
    bound = want.abs() * (7 * U + half_step(y.dtype) * 1.01) + abs(up) * (g.double().abs() + 1) * LEAST + least
    # -3e38 and -1e30 have a sigmoid of zero
    bound[0, :2] = least
    big = want.abs() > torch.finfo(y.dtype).max
    assert torch.equal(torch.isinf(y), big)
    assert_within(y[~big], want[~big], bound[~big], "out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_backward(td, dtype):
    """1 - s is off by 6 U, the bracket 1 + g (1 - s) by 8 U (1 + |g|), s and the products by 8 U more."""
    g = _gates(dtype)
    g[0, :4] = 1.0
    go, u = torch.full_like(g, 2.0 ** 40), torch.full_like(g, 3.0)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    td.moonep_swiglu_backward(go, g, u, dg, du)
    s, x = torch.sigmoid(g.double()), g.double()
    rest = torch.sigmoid(-x)  # 1 - s
    wg, wu = 3 * 2.0 ** 40 * s * (1 + x * rest), 2.0 ** 40 * x * s
    least = torch.finfo(g.dtype).tiny * torch.finfo(g.dtype).eps
    tiny = 3 * 2.0 ** 40 * (1 + x.abs()) * LEAST + least
    assert_within(dg, wg, 3 * 2.0 ** 40 * s * (1 + x.abs()) * (16 * U) + wg.abs() * half_step(g.dtype) * 1.01 + tiny,
                  "grad_gate")
    assert_within(du, wu, wu.abs() * (7 * U + half_step(g.dtype) * 1.01) + tiny, "grad_up")


@pytest.mark.parametrize("gate", [-86.0, -90.0, -100.0])
@pytest.mark.parametrize("kind", WEIGHTS)
def test_layer_for_a_few_tokens(td, kind, gate):
    """The same activation in the layer for a few tokens: one value of the gate for all columns, and
    weights of the tokens that bring the result back among the normal numbers."""
    for T in (3, 30):
        layer = Exact(td, kind, T, 1, 96, 96, seed=80 + T, size=60)
        layer.x[..., 0] = gate
        x = torch.tensor(gate, dtype=torch.float64)
        want = layer.want / 64 * float(x * torch.sigmoid(x))
        got = layer.run().double()
        # A column of the activation is off by 7 U. Three of them, of 2^25 last bits together, make a
        # result of bf16 rows, in 8 additions that are off by 2 U of 2^24 each.
        mag = want.abs() if kind.startswith("f32") else 3 * 2.0 ** 24 * 2.0 ** 60 * abs(float(x * torch.sigmoid(x)))
        least = 2.0 ** 24 * 2.0 ** 60 * 2 * abs(gate) * LEAST
        bound = mag * (11 * U) + least + want.abs() * half_step(layer.dtype) * 1.01
        assert_within(got, want, bound, f"{T} tokens")
