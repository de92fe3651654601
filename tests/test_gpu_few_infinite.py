"""Infinite weights of the layer for a few tokens, where the sum's value follows from the signs."""
import pytest
import torch

from tests.gpu_common import say
from tests.test_gpu_few_exact import Exact

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_infinite_weights(td, kind):
    """A column of the activation that is a number other than zero times an infinite weight is an
    infinity of the product's sign, whatever number it is; zero times it is NaN, and so are two
    infinities of both signs. An infinite activation stays one."""
    inf = float("inf")
    for i, (T, E, H, F, size) in enumerate([(3, 1, 128, 96, 0), (9, 1, 128, 96, 0), (40, 1, 128, 96, 0),
                                            (5, 1, 6400, 96, 0), (7, 1, 128, 96, -106)]):
        layer = Exact(td, kind, T, E, H, F, seed=50 + i, size=size)
        down, step = layer.mats[2], 3 if kind == "bf16" else 1
        few_bits = 2 if kind == "bf16" else 0  # a column whose values are 8 bits
        down[0, 5, 0] = inf                    # 24 bits
        down[0, 6, step + few_bits] = -inf
        down[0, 7, 0], down[0, 7, step + few_bits] = inf, -inf
        down[0, 8, 0], down[0, 8, step + few_bits] = inf, inf
        down[0, 9] = 0
        down[0, 9, F - 1] = inf
        layer.x[0, 0, 1:1 + 3 * layer.J] = 0   # token 0: all columns are zero
        say(f"infinite weights {(T, E, H, F)} {kind}")
        got, sign = layer.run(), layer.w.reshape(T)
        last = 64 * layer.x[0, :, 1 + 3 * (F // 3 - 1) + 1].float() * sign if kind == "bf16" else None
        if kind == "f32":
            last = 64 * layer.x[0, :, F].float() * sign
        for n, want in ((5, sign * inf), (6, sign * -inf), (7, sign * float("nan")), (8, sign * inf), (9, last * inf)):
            want = want.clone()
            want[0] = float("nan")
            assert torch.equal(torch.nan_to_num(got[:, n].float(), nan=7.0), torch.nan_to_num(want, nan=7.0)), n
        assert bool(torch.isfinite(got[:, 10:].float()).all())
        # an infinite weight of a token makes its activation infinite: times an infinite and
        # finite entries of one sign it stays infinite
        layer = Exact(td, kind, T, E, H, F, seed=50 + i)
        for m in layer.mats:
            m.fill_(1)
        layer.mats[2][0, 4, 3] = inf
        layer.x.fill_(1)
        layer.w[0, 0, 0] = inf
        got = layer.run()
        assert bool((got[0] == inf).all())
        assert bool((got[1:, 4].float() == layer.w.reshape(T)[1:] * inf).all())
        assert bool(torch.isfinite(got[1:, 5:].float()).all())


@pytest.mark.parametrize("kind", ["bf16_mx", "f32_mx"])
def test_values_past_the_range(td, kind):
    """A code whose value passes binary32's range (2 times 2^127 here) counts as an infinity, in
    the first products and in the last one, whatever numbers it meets."""
    inf = float("inf")
    for T in (3, 9, 40):
        layer = Exact(td, kind, T, 1, 128, 96, seed=60 + T)
        for m in layer.mats[0::2]:
            m.fill_(0x22)                      # ones
        layer.x.fill_(1)
        layer.mats[4][0, 4, 1] = 0x24          # 2, 1
        layer.mats[5][0, 4, 0] = 254
        got, sign = layer.run().float(), layer.w.reshape(T)
        assert bool((got[:, 4] == sign * inf).all()) and bool(torch.isfinite(got[:, 5:]).all())
        layer.mats[2][0, 7, 1] = 0x24          # U: column 7 of the activation
        layer.mats[3][0, 7, 0] = 254
        got = layer.run().float()
        assert bool((got == sign[:, None] * inf).all())
