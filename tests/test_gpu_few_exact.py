"""The layer for a few tokens where every result is exact: one value of a row is selected by
weights of 0, 1 and -1, so that all 24 bits of what the kernels hold between and before their
products show in the output, and no tolerance is needed.

silu(64) is 64 in binary32 (1 + e^-64 rounds to 1). Values of 24 bits times 64 and a power of two
are exact, and sums of such that stay below 2^24 of their last bits are exact in any order.
"""
import pytest
import torch

from tests.expert_common import torch_dtype
from tests.gpu_common import say
from tests.layer_common import mx_pack
from tests.test_gpu_few import WEIGHTS, Layer

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


# T, E, H, F: each number of columns that the kernels tell apart, wide rows, whole groups of 512
SHAPES = [(1, 8, 64, 96), (4, 2, 64, 96), (7, 1, 96, 96), (20, 1, 64, 96), (40, 2, 64, 192), (64, 1, 512, 512),
          (5, 2, 6400, 96), (3, 3, 512, 1024), (24, 4, 1056, 64), (16, 300, 32, 64), (40, 2, 4608, 96), (20, 1, 4128, 64)]


class Exact:
    """A call whose weights select. bf16 rows: token t's x holds 64 and triples (b0, b1 2^8, b2 2^16)
    of random bytes; column 3 j of the activation is 64 (b0 + b1 2^8 + b2 2^16), the next two
    64 b2 2^16 and 64 b1 2^8, and row n of D takes the first less the two others: 64 b0. binary32
    rows: x holds 64 and values of 24 bits, each of which goes to a column of its own and, by a
    row of D, to the output."""

    def __init__(self, td, kind, T, E, H, F, seed, size=0):
        self.td, self.mx = td, kind.endswith("mx")
        self.dtype = torch_dtype(kind.split("_")[0])
        self.dims = td.Dims(1, E, 1, T, 0, td.BF16 if self.dtype == torch.bfloat16 else td.F32, H)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.ids = torch.randint(0, E, (1, T, 1), generator=g, device=DEV).to(torch.int32)
        sign = 1 - 2 * torch.randint(0, 2, (1, T, 1), generator=g, device=DEV)
        self.w = (sign * 2.0 ** size).float()
        x = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        x[:, 0] = 64
        gate, up, down = (torch.zeros(s, dtype=torch.float64, device=DEV) for s in ((E, F, H), (E, F, H), (E, H, F)))
        gate[:, :, 0] = 1
        n, e = torch.arange(H, device=DEV), torch.arange(E, device=DEV)
        if self.dtype == torch.bfloat16:
            J = self.J = min((H - 1) // 3, F // 3)
            b = torch.randint(1, 256, (T, J, 3), generator=g, device=DEV).double()
            x[:, 1:1 + 3 * J] = (b * torch.tensor([1.0, 2.0 ** 8, 2.0 ** 16], device=DEV)).flatten(1)
            j = torch.arange(J, device=DEV)
            for i in range(3):
                up[:, 3 * j, 1 + 3 * j + i] = 1
            up[:, 3 * j + 1, 1 + 3 * j + 2] = 1
            up[:, 3 * j + 2, 1 + 3 * j + 1] = 1
            pick = (n[None] + e[:, None]) % J  # [E, H]
            for i, s in enumerate((1, -1, -1)):
                down.scatter_(2, (3 * pick + i)[..., None], float(s))
            source = b[:, :, 0]
        else:
            J = self.J = min(H - 1, F)
            b = torch.randint(2 ** 22, 2 ** 23, (T, J), generator=g, device=DEV).double() * 2 + 1
            x[:, 1:1 + J] = b
            j = torch.arange(J, device=DEV)
            up[:, j, 1 + j] = 1
            pick = (n[None] + e[:, None]) % J
            down.scatter_(2, pick[..., None], 1.0)
            source = b
        mine = self.ids.reshape(T).long()
        self.pick = pick
        self.want = 64 * source.gather(1, pick[mine]) * self.w.reshape(T, 1).double()
        self.x = x.to(self.dtype).reshape(1, T, H)
        assert torch.equal(self.x[0].double(), x)
        self.mats = []
        for m in (gate, up, down):
            if self.mx:
                code = torch.where(m < 0, 10, torch.where(m > 0, 2, 0))  # -1, 1, 0
                self.mats += mx_pack(code, torch.full(m.shape[:-1] + (m.shape[-1] // 32,), 127, device=DEV))
            else:
                self.mats.append(m.to(self.dtype).contiguous())
        self.out = torch.full_like(self.x, 3.0)
        self.work = td.new_layer_workspace(self.dims, F, DEV).fill_(0xff)

    def run(self):
        call = self.td.moonep_expert_layer_mx if self.mx else self.td.moonep_expert_layer
        call(self.dims, self.ids, self.w, self.x, *self.mats, self.out, self.work)
        return self.out[0]


@pytest.mark.parametrize("kind", WEIGHTS)
def test_all_bits_reach_the_output(td, kind):
    """Between the products the activation keeps binary32's 24 bits, and so do binary32 rows that
    meet weights of fewer bits."""
    for i, shape in enumerate(SHAPES):
        say(f"exact layer {shape} {kind}")
        layer = Exact(td, kind, *shape, seed=i)
        got = layer.run().double()
        assert torch.equal(got, layer.want), f"{shape}: {int((got != layer.want).sum())} of {got.numel()} differ"


@pytest.mark.parametrize("kind", WEIGHTS)
def test_all_bits_of_small_magnitudes(td, kind):
    """All 24 bits from magnitudes of 2^-100 on: the activation's are 64 2^size and more, binary32
    rows' too."""
    for i, shape in enumerate([(3, 2, 64, 96), (20, 1, 64, 96)]):
        layer = Exact(td, kind, *shape, seed=70 + i, size=-106)
        assert float(layer.want.abs().min()) >= 2.0 ** -100
        assert torch.equal(layer.run().double(), layer.want), "activation"
        if kind.startswith("f32"):
            layer = Exact(td, kind, *shape, seed=70 + i)
            layer.x[..., 1:] *= 2.0 ** -122
            layer.want *= 2.0 ** -122
            assert float(layer.x[0, :, 1].abs().min()) >= 2.0 ** -100
            assert torch.equal(layer.run().double(), layer.want), "rows"


@pytest.mark.parametrize("kind", WEIGHTS)
def test_wide_rows_of_many_tokens(td, kind):
    """Rows just past 4096 columns, where a workgroup takes 32 of them, with up to 16, 32 and 64
    tokens, against the plain form."""
    for i, shape in enumerate([(1, 40, 5, 2, 4608, 96), (1, 64, 3, 2, 4160, 512), (1, 33, 12, 5, 4096, 64),
                               (1, 17, 6, 2, 4128, 160), (1, 7, 9, 3, 4608, 64)]):
        say(f"wide layer {shape} {kind}")
        Layer(td, kind, *shape, 90 + i).check(str(shape))
