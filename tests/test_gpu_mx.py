"""The experts' products of 4-bit rows and matrices on the GPU, against their plain form in 64
bits: a sum of n products in binary32 is within n * 2^-23 * sum |products| of the exact one
whatever its order, and its store is off by half a step of the output's type."""
import pytest
import torch

from tests.expert_common import ADD, assert_within, half_step, make_table, segments
from tests.gpu_common import say
from tests.layer_common import mx_values, scale_cols
from tests.test_gpu_experts import KINDS, _dims, _rand, _table

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


def _mx(td, shape, seed, scale=1.0, wide=True):
    """(codes, scales) of random rows [*lead, n]; blocks of sizes some powers of two apart."""
    v = _rand(shape, "f32", seed, scale)
    if wide:
        g = torch.Generator(device=DEV).manual_seed(seed + 1)
        e = torch.randint(-3, 4, shape[:-1] + (shape[-1] // 32,), generator=g, device=DEV)
        v = v * torch.exp2(e.float()).repeat_interleave(32, -1)
    q = torch.empty(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, device=DEV)
    s = torch.empty(shape[:-1] + (scale_cols(shape[-1]),), dtype=torch.uint8, device=DEV)
    if v.numel():
        td.moonep_quantize_rows_mx(v, q, s)
    s[..., shape[-1] // 32:] = 255  # bytes behind the blocks are not used
    return q, s


def _plain(table, G, B, x, w, dup_w):
    R, SK, n_out = x.shape[0], x.shape[1], w.shape[1]
    y = torch.zeros((R, SK, n_out), dtype=torch.float64, device=DEV)
    mag, written = torch.zeros_like(y), torch.zeros((R, SK), dtype=torch.bool, device=DEV)
    for r, j, lo, hi in segments(table, G, B, SK):
        if lo < 0 or hi <= lo:
            continue
        m = (w[r * G + j] if j < G else dup_w[r, j - G]).t().contiguous()
        y[r, lo:hi], mag[r, lo:hi], written[r, lo:hi] = x[r, lo:hi] @ m, x[r, lo:hi].abs() @ m.abs(), True
    return y, mag, written


# R, E, K, S, B, n_in, n_out: one block, one step and a part of it, tails of rows and columns
SHAPES = [
    (1, 1, 1, 1, 0, 32, 16),
    (1, 2, 1, 3, 1, 64, 8),
    (2, 4, 2, 5, 2, 96, 40),
    (8, 64, 8, 1, 8, 256, 128),
    (3, 21, 5, 33, 2, 288, 136),
    (2, 6, 2, 150, 3, 160, 520),
    (4, 16, 2, 64, 4, 512, 256),
    (1, 3, 3, 400, 1, 1056, 264),
    (2, 2, 2, 600, 1, 64, 1032),
    (1, 4, 1, 7, 0, 2048, 24),
    (3, 9, 1, 20, 3, 4128, 48),
]
# enough rows and columns for each of the larger tiles, with ragged segments and tails
LARGE = [
    (8, 32, 2, 600, 2, 544, 1160),
    (8, 64, 4, 200, 3, 800, 776),
    (8, 64, 4, 400, 2, 288, 104),
    (16, 64, 2, 20, 1, 1056, 136),
    (2, 4, 2, 1100, 1, 1312, 520),
    (8, 64, 4, 200, 3, 800, 520),
    # rows of whole 512 values, whose scales are loaded two steps at a time
    (8, 32, 2, 600, 2, 512, 1160),
    (8, 64, 4, 200, 3, 1536, 776),
    (8, 64, 4, 200, 3, 1536, 520),
    (8, 64, 4, 60, 2, 1024, 776),
    (16, 64, 2, 20, 1, 1024, 136),
    (2, 4, 2, 1100, 1, 2560, 520),
    (1, 3, 2, 30, 0, 4096, 48),
]


def _check(td, shape, kind, dtype, seed):
    R, E, K, S, B, n_in, n_out = shape
    G, SK = E // R, S * K
    dims = _dims(td, R, E, K, S, B, dtype)
    table = _table(kind, R, E, K, S, B, seed)
    x, xs = _mx(td, (R, SK, n_in), seed)
    w, ws = _mx(td, (E, n_out, n_in), seed + 2)
    dw, dws = _mx(td, (R, B, n_out, n_in), seed + 4)
    values = [mx_values(q, s, n_in) for q, s in ((x, xs), (w, ws), (dw, dws))]
    want, mag, written = _plain(table, G, B, *values)
    # what no segment names may hold anything: it is not read into a result
    x[~written], xs[~written] = 0x77, 255
    for r in range(R):
        for b in range(min(B, table.shape[1] - 1 - G)):
            if table[r, G + b] < 0 or table[r, G + b + 1] <= table[r, G + b]:
                dws[r, b] = 255
    y = torch.full((R, SK, n_out), 3.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device=DEV)
    seg = torch.from_numpy(table).to(DEV)
    say(f"mx matmul {shape} {kind} {dtype}")
    td.moonep_expert_matmul_mx(dims, seg, x, xs, w, ws, dw, dws, y)
    torch.cuda.synchronize()
    bound = mag * (n_in * ADD) + want.abs() * half_step(y.dtype) * 1.01
    assert_within(y[written], want[written], bound[written], "y")
    assert bool((y[~written] == 3.0).all()), "a row of no segment was written"
    again = torch.full_like(y, 3.0)
    td.moonep_expert_matmul_mx(dims, seg, x, xs, w, ws, dw, dws, again)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_matmul(td, kind, dtype):
    for i, shape in enumerate(SHAPES):
        _check(td, shape, kind, dtype, 100 + i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_large(td, shape, dtype):
    for i, kind in enumerate(("full", "over", "behind")):
        _check(td, shape, kind, dtype, 300 + i)


def test_exact_sums(td):
    """Small whole numbers: every sum is exact, whatever its order."""
    R, E, K, S, B, n_in, n_out = 2, 4, 2, 90, 1, 1024, 264
    dims = _dims(td, R, E, K, S, B, "f32")
    g = torch.Generator(device=DEV).manual_seed(5)
    pick = torch.tensor([0, 2, 4, 6, 10, 12], dtype=torch.uint8, device=DEV)  # 0, 1, 2, 4, -1, -2

    def codes(*lead):
        a, b = (pick[torch.randint(0, 6, lead + (n_in // 2,), generator=g, device=DEV)] for _ in range(2))
        s = torch.randint(127, 130, lead + (scale_cols(n_in),), generator=g, device=DEV).to(torch.uint8)
        return a | b << 4, s

    (x, xs), (w, ws), (dw, dws) = codes(R, S * K), codes(E, n_out), codes(R, B, n_out)
    table = make_table([[40, 80, 60], [100, 0, 80]], R, 2, 2, S * K)
    want = _plain(table, 2, B, *(mx_values(q, s, n_in) for q, s in ((x, xs), (w, ws), (dw, dws))))[0]
    y = torch.zeros((R, S * K, n_out), device=DEV)
    td.moonep_expert_matmul_mx(dims, torch.from_numpy(table).to(DEV), x, xs, w, ws, dw, dws, y)
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("rows", [5, 300], ids=["few", "many"])
def test_nan_scales_and_all_scales(td, rows):
    """A scale of 255 makes its own row, or its own column, NaN and nothing else; scales from
    end to end of their range multiply out."""
    R, E, K, S, B, n_in, n_out = 1, 2, 1, rows, 0, 320, 72
    dims = _dims(td, R, E, K, S, B, "f32")
    x, xs = _mx(td, (R, S, n_in), 1)
    w, ws = _mx(td, (E, n_out, n_in), 2)
    table = make_table([[rows - 2, 2]], R, 2, 1, S)
    seg = torch.from_numpy(table).to(DEV)
    xs[0, 3, 9], ws[0, 70, 0] = 255, 255
    y = torch.zeros((R, S, n_out), device=DEV)
    td.moonep_expert_matmul_mx(dims, seg, x, xs, w, ws, None, None, y)
    bad = torch.isnan(y[0])
    want = torch.zeros_like(bad)
    want[3] = True
    want[:rows - 2, 70] = True
    assert torch.equal(bad, want)
    for sx, sw in ((0, 254), (254, 0), (1, 200), (127, 127), (254, 127)):
        xs[..., :10], ws[..., :10] = sx, sw
        want, mag, _ = _plain(table, 2, 0, mx_values(x, xs, n_in), mx_values(w, ws, n_in), None)
        td.moonep_expert_matmul_mx(dims, seg, x, xs, w, ws, None, None, y)
        # past binary32's range sums may be infinite, or NaN where infinities meet
        keep = mag < 2.0 ** 127
        bound = mag * (n_in * ADD) + want.abs() * half_step(y.dtype) * 1.01
        assert_within(y[keep], want[keep], bound[keep], f"scales {sx}, {sw}")


def test_views_of_larger_blocks(td):
    """Matrices that are parts of larger blocks, and others that are refused."""
    R, E, K, S, B, n_in, n_out = 2, 4, 1, 30, 2, 128, 64
    dims = _dims(td, R, E, K, S, B, "bf16")
    x, xs = _mx(td, (R, S, n_in), 1)
    w, ws = _mx(td, (E, 3, n_out, n_in), 2)
    dw, dws = _mx(td, (R, B, 3, n_out, n_in), 3)
    table = _table("full", R, E, K, S, B, 4)
    seg = torch.from_numpy(table).to(DEV)
    y, z = (torch.zeros((R, S, n_out), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    td.moonep_expert_matmul_mx(dims, seg, x, xs, w[:, 1], ws[:, 1], dw[:, :, 1], dws[:, :, 1], y)
    td.moonep_expert_matmul_mx(dims, seg, x, xs, w[:, 1].contiguous(), ws[:, 1].contiguous(),
                               dw[:, :, 1].contiguous(), dws[:, :, 1].contiguous(), z)
    assert torch.equal(y, z)
    with pytest.raises(ValueError):
        td.moonep_expert_matmul_mx(dims, seg, x, xs, w[:, 1], ws[:, 1], dw[:, :, 1].contiguous(), dws[:, :, 1], y)
    with pytest.raises(ValueError):
        td.moonep_expert_matmul_mx(dims, seg, x, xs[..., :2], w[:, 1], ws[:, 1], dw[:, :, 1], dws[:, :, 1], y)
    with pytest.raises(TypeError):
        td.moonep_expert_matmul_mx(dims, seg, x.view(torch.int8), xs, w[:, 1], ws[:, 1], dw[:, :, 1], dws[:, :, 1], y)


def test_offsets_past_32_bits(td):
    """Rows and matrices that lie past 2^32 bytes."""
    R, E, K, S, B, n_in, n_out = 1, 300, 1, 400, 0, 8192, 4096
    dims = _dims(td, R, E, K, S, B, "bf16")
    w = torch.zeros((E, n_out, n_in // 2), dtype=torch.uint8, device=DEV)
    ws = torch.zeros((E, n_out, scale_cols(n_in)), dtype=torch.uint8, device=DEV)
    w[-1], ws[-1] = (t[0] for t in _mx(td, (1, n_out, n_in), 2))
    x, xs = _mx(td, (R, S, n_in), 1)
    table = make_table([[100] + [0] * (E - 2) + [300]], R, E, 1, S)
    y = torch.zeros((R, S, n_out), dtype=torch.bfloat16, device=DEV)
    td.moonep_expert_matmul_mx(dims, torch.from_numpy(table).to(DEV), x, xs, w, ws, None, None, y)
    a, b = mx_values(x[0, 100:], xs[0, 100:], n_in), mx_values(w[-1], ws[-1], n_in).t().contiguous()
    want, mag = a @ b, a.abs() @ b.abs()
    assert_within(y[0, 100:], want, mag * (n_in * ADD) + want.abs() * half_step(y.dtype) * 1.01, "y")
    assert bool((y[0, :100] == 0).all())


def test_replayed_graph_and_two_streams(td):
    """Quantisation, product and activation to 4 bits captured once and replayed on other rows,
    matrices and segments; and the same calls on two streams at once."""
    R, E, K, S, B, n_in, n_out = 4, 16, 2, 64, 4, 512, 128
    dims = _dims(td, R, E, K, S, B, "bf16")
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731

    class Step:
        def __init__(self, seed):
            self.rows = _rand((R, S * K, n_in), "bf16", seed)
            self.w, self.dw = _mx(td, (E, n_out, n_in), seed + 2), _mx(td, (R, B, n_out, n_in), seed + 4)
            self.seg = torch.from_numpy(_table(KINDS[0], R, E, K, S, B, seed)).to(DEV)
            self.q, self.s = u8(R, S * K, n_in // 2), u8(R, S * K, scale_cols(n_in))
            self.y = torch.zeros((R, S * K, n_out), dtype=torch.bfloat16, device=DEV)
            self.a, self.a_s = u8(R, S * K, n_out // 4), u8(R, S * K, scale_cols(n_out // 2))

        def run(self, stream=None):
            td.moonep_quantize_rows_mx(self.rows, self.q, self.s, stream=stream)
            td.moonep_expert_matmul_mx(dims, self.seg, self.q, self.s, *self.w, *self.dw, self.y, stream=stream)
            td.moonep_swiglu_mx(self.y[..., :n_out // 2], self.y[..., n_out // 2:], self.a, self.a_s, stream=stream)
            return [t.clone() for t in (self.y, self.a, self.a_s)]

    step = Step(1)
    step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for seed in (11, 21, 31):
        new = Step(seed)
        want = new.run()
        for mine, theirs in ((step.rows, new.rows), (step.seg, new.seg), (step.w[0], new.w[0]), (step.w[1], new.w[1]),
                             (step.dw[0], new.dw[0]), (step.dw[1], new.dw[1])):
            mine.copy_(theirs)
        step.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, expected in zip((step.y, step.a, step.a_s), want):
            assert torch.equal(got, expected), f"replay {seed}"
    pair = [Step(41), Step(51)]
    want = [p.run() for p in pair]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    for p in pair:
        p.y.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for p, stream in zip(pair, streams):
            with torch.cuda.stream(stream):
                p.run(stream)
    torch.cuda.synchronize()
    for p, expected in zip(pair, want):
        for got, e in zip((p.y, p.a, p.a_s), expected):
            assert torch.equal(got, e)
