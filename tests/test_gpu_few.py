"""The whole layer for a few tokens on the GPU, against its plain form in 64 bits, whose bound
on binary32's sums and roundings stands with it (tests/layer_common.py)."""
import pytest
import torch

from tests.expert_common import assert_within, half_step, torch_dtype
from tests.gpu_common import say
from tests.layer_common import mx_values, plain_layer, scale_cols

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
WEIGHTS = ["bf16", "f32", "bf16_mx", "f32_mx"]


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch_dtype(dtype))


class Layer:
    """Inputs of one call, its buffers and its plain form."""

    def __init__(self, td, kind, R, S, E, K, H, F, seed):
        dtype, self.mx = kind.split("_")[0], kind.endswith("mx")
        self.td, self.H, self.F = td, H, F
        self.dims = td.Dims(R, E, K, S, 0, td.BF16 if dtype == "bf16" else td.F32, H)
        dt = torch_dtype(dtype)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.ids = torch.rand((R, S, E), generator=g, device=DEV).topk(K, -1).indices.to(torch.int32)
        self.w = torch.rand((R, S, K), generator=g, device=DEV) + 0.1
        self.x = _rand((R, S, H), dtype, seed + 1)
        self.mats, self.scales = [], []
        for i, (n, k) in enumerate(((F, H), (F, H), (H, F))):
            m = _rand((E, n, k), "f32" if self.mx else dtype, seed + 2 + i, k ** -0.5)
            if self.mx:
                q = torch.empty((E, n, k // 2), dtype=torch.uint8, device=DEV)
                s = torch.empty((E, n, scale_cols(k)), dtype=torch.uint8, device=DEV)
                td.moonep_quantize_rows_mx(m, q, s)
                s[..., k // 32:] = 255  # bytes behind the blocks are not used
                m = q
                self.scales.append(s)
            self.mats.append(m)
        self.out = torch.full((R, S, H), 9.0, dtype=dt, device=DEV)
        self.work = td.new_layer_workspace(self.dims, F, DEV).fill_(0xff)

    def run(self, out=None, work=None, stream=None):
        out, work = self.out if out is None else out, self.work if work is None else work
        if self.mx:
            both = [t for pair in zip(self.mats, self.scales) for t in pair]
            self.td.moonep_expert_layer_mx(self.dims, self.ids, self.w, self.x, *both, out, work, stream=stream)
        else:
            self.td.moonep_expert_layer(self.dims, self.ids, self.w, self.x, *self.mats, out, work, stream=stream)
        return out

    def values(self):
        if not self.mx:
            return [m.double() for m in self.mats]
        return [mx_values(q, s, 2 * q.shape[-1]) for q, s in zip(self.mats, self.scales)]

    def plain(self):
        K, H = self.dims.K, self.H
        pieces = 2.0 ** -16 if self.x.dtype == torch.bfloat16 else 0.0
        want, bound = plain_layer(self.ids.reshape(-1, K), self.w.reshape(-1, K), self.x.reshape(-1, H),
                                  *self.values(), self.dims.E, pieces)
        return want, bound + want.abs() * half_step(self.out.dtype) * 1.01

    def check(self, what):
        self.run()
        torch.cuda.synchronize()
        want, bound = self.plain()
        assert_within(self.out.reshape(-1, self.H), want, bound, what)


# R, S, E, K, H, F in units of 32 columns and odd multiples of the smallest unit
SHAPES = [
    (1, 1, 1, 1, 32, 32),
    (1, 1, 8, 2, 96, 64),
    (1, 1, 40, 16, 1056, 160),
    (2, 3, 8, 3, 288, 96),
    (1, 16, 4, 4, 160, 224),     # every token on every expert
    (4, 4, 64, 8, 512, 256),
    (1, 17, 6, 2, 128, 96),
    (1, 33, 12, 5, 96, 416),
    (1, 64, 3, 2, 224, 64),      # more tokens of an expert than one tile takes
    (1, 64, 100, 16, 64, 128),
    (1, 64, 1, 1, 64, 32),
    (1, 5, 1024, 4, 64, 32),
    (1, 64, 64, 64, 32, 32),
    (1, 2, 3, 2, 4128, 1056),
    # wide rows of out, rows of whole 512 values, more than 1024 workgroups of the first kernel
    (1, 24, 8, 2, 6400, 64),
    (1, 3, 40, 4, 6656, 512),
    (1, 40, 9, 3, 512, 1024),
    (1, 64, 128, 16, 96, 320),
]
ODD = {"bf16": [(1, 3, 5, 2, 8, 8), (2, 9, 6, 4, 264, 24), (1, 40, 9, 3, 1032, 200), (1, 5, 4, 2, 6152, 40)],
       "f32": [(1, 3, 5, 2, 4, 4), (2, 9, 6, 4, 132, 20), (1, 40, 9, 3, 516, 100), (1, 5, 4, 2, 6148, 36)]}


@pytest.mark.parametrize("kind", WEIGHTS)
def test_layer(td, kind):
    for i, (R, S, E, K, H, F) in enumerate(SHAPES + ODD.get(kind, [])):
        say(f"layer {(R, S, E, K, H, F)} {kind}")
        layer = Layer(td, kind, R, S, E, K, H, F, 30 * i)
        layer.check(str((R, S, E, K, H, F)))
        first = layer.out.clone()
        layer.out.fill_(1.0)
        layer.work.random_()
        assert torch.equal(layer.run(), first), "the workspace's old contents reach the output"


@pytest.mark.parametrize("kind", WEIGHTS)
def test_ids_outside_and_repeated(td, kind):
    """Entries without an expert contribute nothing, whatever their weight; a repeated expert
    counts as often; a token without any is zeros."""
    for S, E in ((6, 40), (40, 5)):  # slots by entries, and by experts
        layer = Layer(td, kind, 1, S, E, 4, 96, 64, 7)
        layer.ids[0, 0] = torch.tensor([-1, E, 2, -2 ** 31], dtype=torch.int32)
        layer.w[0, 0] = torch.tensor([float("nan"), float("inf"), 0.5, float("nan")])
        layer.ids[0, 1] = torch.tensor([3, 3, 1, 3], dtype=torch.int32)
        layer.ids[0, 2] = torch.tensor([2 ** 31 - 1, -1, -1, E], dtype=torch.int32)
        layer.ids[0, 3] = 2
        layer.ids[0, 4] = torch.tensor([0, -1, 0, 1], dtype=torch.int32)
        layer.w[0, 5] = torch.tensor([0.0, -1.0, 2.0, 0.0])
        layer.check("ids")
        assert bool((layer.out[0, 2] == 0).all())


@pytest.mark.parametrize("kind", WEIGHTS)
def test_no_valid_ids_at_all(td, kind):
    layer = Layer(td, kind, 1, 20, 6, 2, 64, 32, 1)
    layer.ids.fill_(-1)
    assert bool((layer.run() == 0).all())


@pytest.mark.parametrize("kind", WEIGHTS)
def test_infinities_reach_their_tokens_only(td, kind):
    """NaN and infinities in a token, and in an expert's matrices, reach the tokens that have
    that expert and no other."""
    layer = Layer(td, kind, 1, 24, 6, 2, 160, 64, 11)
    want, bound = layer.plain()
    layer.x[0, 3, 100] = float("nan")
    layer.x[0, 4, 7] = float("inf")
    for m, e in zip(range(3), (1, 2, 4)):
        if layer.mx:
            layer.scales[m][e, 5, 1] = 255
        else:
            layer.mats[m][e, 5, 33] = float("inf") if m != 1 else float("nan")
    layer.run()
    hit = ((layer.ids[0] == 1) | (layer.ids[0] == 2) | (layer.ids[0] == 4)).any(-1)
    hit[3] = hit[4] = True
    free = ~hit
    assert int(free.sum()) >= 2 and int(hit.sum()) >= 6
    assert_within(layer.out[0][free], want[free], bound[free], "untouched tokens")
    bad = ~torch.isfinite(layer.out[0].float()).all(-1)
    assert torch.equal(bad, hit)


@pytest.mark.parametrize("kind", ["bf16", "f32_mx"])
def test_views_streams_and_two_at_once(td, kind):
    """Gate and up as halves of one tensor; two calls at once on two streams with a workspace
    each; matrices at other distances are refused."""
    layer = Layer(td, kind, 1, 9, 10, 3, 128, 96, 5)
    want = layer.run().clone()
    F = 96
    layer.mats[:2] = [t for t in (torch.cat(layer.mats[:2], 1),) for t in (t[:, :F], t[:, F:])]
    if layer.mx:
        layer.scales[:2] = [t for t in (torch.cat(layer.scales[:2], 1),) for t in (t[:, :F], t[:, F:])]
    assert torch.equal(layer.run(), want)
    other = Layer(td, kind, 1, 33, 10, 3, 128, 96, 6)
    alone = other.run().clone()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    layer.out.zero_()
    other.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        layer.run(stream=a)
        other.run(stream=b)
    torch.cuda.synchronize()
    assert torch.equal(layer.out, want) and torch.equal(other.out, alone)
    layer.mats[1] = layer.mats[1].contiguous()
    with pytest.raises(ValueError):
        layer.run()
    with pytest.raises(ValueError):
        other.run(work=other.work[:-1])
    with pytest.raises(ValueError):
        other.run(out=other.out[:, :1])


@pytest.mark.parametrize("kind", WEIGHTS)
def test_replayed_graph(td, kind):
    """Captured once, replayed on other tokens and routes with eager calls that share the
    workspace between the replays."""
    layer = Layer(td, kind, 2, 10, 12, 3, 192, 128, 8)
    layer.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    for seed in (1, 2, 3):
        new = Layer(td, kind, 2, 10, 12, 3, 192, 128, 100 + seed)
        layer.ids.copy_(new.ids)
        layer.w.copy_(new.w)
        layer.x.copy_(new.x)
        layer.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = layer.out.clone()
        eager = torch.empty_like(layer.out)
        layer.run(out=eager)
        torch.cuda.synchronize()
        assert torch.equal(got, eager), f"replay {seed}"


def test_offsets_past_32_bits(td):
    """Experts whose matrices begin past 2^32 bytes."""
    E, H, F = 40, 8192, 8192
    layer = Layer(td, "bf16", 1, 2, 2, 2, H, F, 3)
    want = layer.run().clone()
    mats = []
    for m in layer.mats:
        big = torch.zeros((E,) + tuple(m.shape[1:]), dtype=m.dtype, device=DEV)
        big[-2:] = m
        mats.append(big)
    layer.mats = mats
    layer.dims = td.Dims(1, E, 2, 2, 0, td.BF16, H)
    layer.ids += E - 2
    assert torch.equal(layer.run(), want)
