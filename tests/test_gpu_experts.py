"""The experts' products on the GPU against their plain forms in 64 bits.

Tolerances: a sum of n products in binary32 is within n * 2^-23 * sum |products| of the
exact one whatever its order (one step for each addition), and its store is off by half a
step of the output's type. The 8-bit products are exact until their two binary32
factors, and are compared bit for bit.
"""
import numpy as np
import pytest
import torch

from tests.expert_common import (ADD, assert_within, half_step, make_table, plain_matmul,
                                 plain_wgrad, torch_dtype)
from tests.gpu_common import run_plan, say

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


def _dims(td, R, E, K, S, B, dtype, H=64):
    return td.Dims(R, E, K, S, B, td.BF16 if dtype == "bf16" else td.F32, H)


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch_dtype(dtype))


def _split(total, n, seed, zero=0.3):
    """total rows over n segments, some of them empty."""
    rng = np.random.default_rng(seed)
    p = rng.random(n) ** 3 * (rng.random(n) > zero)
    if p.sum() == 0:
        p[0] = 1.0
    return rng.multinomial(total, p / p.sum()).tolist()


def _table(kind, R, E, K, S, B, seed):
    G, SK = E // R, S * K
    dcap = max(1, min(SK, E - G))
    rows = []
    for r in range(R):
        if kind == "full":       # as a plan leaves it: every row in a segment
            rows.append(_split(SK, G + min(B, dcap), seed + r))
        elif kind == "over":     # more duplicates than slots
            rows.append(_split(SK, G + min(B + 2, dcap), seed + r, 0.1))
        elif kind == "one":      # all rows one expert's
            rows.append([0] * (r % G) + [SK])
        elif kind == "behind":   # rows behind the last segment, and an empty rank
            rows.append([] if r == 0 else _split(SK - SK // 3, G, seed + r))
        elif kind == "single":   # one row each
            rows.append([1] * min(SK, G))
    return make_table(rows, R, G, dcap, SK)


# R, E, K, S, B, n_in, n_out: sizes from one row to more than a tile, columns of every tail
SHAPES = [
    (1, 1, 1, 1, 0, 16, 16),
    (1, 2, 1, 3, 1, 8, 8),
    (2, 4, 2, 5, 2, 24, 40),
    (8, 64, 8, 1, 8, 256, 128),
    (3, 21, 5, 33, 2, 264, 136),
    (2, 6, 2, 150, 3, 72, 520),
    (4, 16, 2, 64, 4, 128, 256),
    (1, 3, 3, 400, 1, 1032, 264),
    (2, 2, 2, 600, 1, 64, 1032),
    (2, 8, 4, 700, 4, 512, 512),
    (1, 4, 1, 7, 0, 2048, 24),
    (3, 9, 1, 20, 3, 4104, 48),
]
# enough rows and columns for each of the larger tiles, with ragged segments and tails
LARGE = [
    (8, 32, 2, 600, 2, 72, 776),      # about 240 to 300 rows a segment, wide outputs
    (8, 64, 4, 200, 3, 520, 776),     # about 100
    (8, 64, 4, 400, 2, 264, 104),     # narrow outputs
    (16, 64, 2, 20, 1, 1032, 136),    # about 10 rows, many segments
    (1, 3, 2, 30, 0, 4112, 48),       # few tiles, long rows
    (2, 2, 1, 1500, 0, 136, 72),      # few segments, long
]
# steps and tiles enough for the tiles of 256 columns; few tiles with long segments
TILES = [
    (8, 32, 2, 600, 2, 528, 1160),
    (8, 64, 4, 128, 3, 1040, 712),
    (2, 4, 2, 1100, 1, 264, 520),
]
KINDS = ["full", "over", "one", "behind", "single"]


def _check_matmul(td, shape, kind, dtype, transposed, seed):
    R, E, K, S, B, n_in, n_out = shape
    G, SK = E // R, S * K
    dims = _dims(td, R, E, K, S, B, dtype)
    table = _table(kind, R, E, K, S, B, seed)
    x = _rand((R, SK, n_in), dtype, seed)
    tail = (n_out, n_in) if transposed else (n_in, n_out)
    w, dup_w = _rand((E,) + tail, dtype, seed + 1), _rand((R, B) + tail, dtype, seed + 2)
    y = torch.full((R, SK, n_out), 3.0, dtype=x.dtype, device=DEV)
    seg = torch.from_numpy(table).to(DEV)
    want, mag, written = plain_matmul(table, G, B, x, w, dup_w, transposed)
    # what no segment names may hold anything: it is not read into a result
    x[~written] = float("nan")
    for r in range(R):
        for b in range(min(B, table.shape[1] - 1 - G)):
            if table[r, G + b] < 0 or table[r, G + b + 1] <= table[r, G + b]:
                dup_w[r, b] = float("inf")
    say(f"matmul {shape} {kind} {dtype} transposed={transposed}")
    td.moonep_expert_matmul(dims, seg, x, w, dup_w, y, transposed=transposed)
    torch.cuda.synchronize()
    bound = mag * (n_in * ADD) + want.abs() * half_step(y.dtype) * 1.01
    assert_within(y[written], want[written], bound[written], "y")
    assert bool((y[~written] == 3.0).all()), "a row of no segment was written"
    again = torch.full_like(y, 3.0)
    td.moonep_expert_matmul(dims, seg, x, w, dup_w, again, transposed=transposed)
    assert torch.equal(again, y)


@pytest.mark.parametrize("transposed", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_matmul(td, kind, dtype, transposed):
    for i, shape in enumerate(SHAPES):
        _check_matmul(td, shape, kind, dtype, transposed, 100 + i)


@pytest.mark.parametrize("transposed", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_large(td, shape, dtype, transposed):
    for i, kind in enumerate(("full", "over", "behind")):
        _check_matmul(td, shape, kind, dtype, transposed, 700 + i)
        _check_wgrad(td, shape, kind, dtype, transposed, 710 + i)
        _check_quant(td, shape, kind, dtype, 720 + i)


@pytest.mark.parametrize("transposed", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("kind", ["full", "over", "behind", "single"])
@pytest.mark.parametrize("shape", TILES, ids=lambda s: "x".join(map(str, s)))
def test_wide_tiles_and_shared_steps(td, shape, kind, transposed):
    _check_matmul(td, shape, kind, "bf16", transposed, 800)
    _check_wgrad(td, shape, kind, "bf16", transposed, 810)
    _check_quant(td, shape, kind, "f32" if transposed else "bf16", 820)


def _check_wgrad(td, shape, kind, dtype, transposed, seed):
    R, E, K, S, B, n_in, n_out = shape
    G, SK = E // R, S * K
    dims = _dims(td, R, E, K, S, B, dtype)
    table = _table(kind, R, E, K, S, B, seed)
    x, g = _rand((R, SK, n_in), dtype, seed), _rand((R, SK, n_out), dtype, seed + 1)
    tail = (n_out, n_in) if transposed else (n_in, n_out)
    home = torch.full((E,) + tail, 5.0, device=DEV)
    dup = torch.full((R, B) + tail, 5.0, device=DEV)
    want_h, want_d, mag_h, mag_d, written = plain_wgrad(table, G, B, x, g, transposed)
    _, _, used = plain_matmul(table, G, B, x, torch.zeros((E, n_in, 1), device=DEV),
                              torch.zeros((R, B, n_in, 1), device=DEV), False)
    x[~used] = float("nan")
    g[~used] = float("inf")
    say(f"wgrad {shape} {kind} {dtype} transposed={transposed}")
    seg = torch.from_numpy(table).to(DEV)
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home, dup, transposed=transposed)
    torch.cuda.synchronize()
    eps = SK * ADD + half_step(torch.float32) * 1.01
    assert_within(home, want_h, mag_h * eps, "home")
    assert_within(dup[written], want_d[written], mag_d[written] * eps, "dup")
    assert bool((dup[~written] == 5.0).all()), "a slot without a segment was written"
    home2, dup2 = torch.zeros_like(home), torch.full_like(dup, 5.0)
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home2, dup2, transposed=transposed)
    assert torch.equal(home, home2) and torch.equal(dup, dup2)


@pytest.mark.parametrize("transposed", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_wgrad(td, kind, dtype, transposed):
    for i, shape in enumerate(SHAPES):
        _check_wgrad(td, shape, kind, dtype, transposed, 200 + i)


def _plain_quantise(x):
    """numpy, the header's definition step by step in binary32."""
    x = x.float().cpu().numpy()
    a = np.maximum(np.abs(x).max(axis=-1), np.float32(2.0 ** -100)).astype(np.float32)
    with np.errstate(all="ignore"):
        q = np.rint(x * (np.float32(127.0) / a)[..., None])
    finite = np.isfinite(x).all(axis=-1)
    q[~finite] = 0
    scale = np.where(finite, a / np.float32(127.0), np.float32("nan")).astype(np.float32)
    return q.astype(np.int8), scale


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,cols", [(1, 16), (3, 48), (7, 1024), (65, 7168), (300, 80), (5, 40000)])
def test_quantize_rows(td, n, cols, dtype):
    x = _rand((n, cols), dtype, n + cols)
    x[0, 0] = 0.0
    if n > 5:
        x[1] = 0.0                                     # a row of zeros
        x[2] *= 1e-30                                  # small, but above 2^-100
        x[3] *= 2.0 ** -110                            # below: the scale stays that of 2^-100
        x[4, cols - 1] = float("nan")
        x[5, 3] = float("-inf")
        x[6, 7] = 3.0e38                               # near the largest
    q = torch.full((n, cols), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((n,), 7.0, device=DEV)
    td.moonep_quantize_rows(x, q, scale)
    want_q, want_s = _plain_quantise(x)
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(scale.cpu().numpy(), want_s, equal_nan=True)


def test_quantize_rounds_halves_to_even(td):
    # a row whose largest value is 127 has factor 1: halves are exact ties
    x = torch.arange(-127, 127, dtype=torch.float32, device=DEV)[:252] + 0.5
    x = torch.cat([x, torch.tensor([127.0, -127.0, 0.25, -0.75], device=DEV)]).reshape(1, 256)
    q = torch.empty((1, 256), dtype=torch.int8, device=DEV)
    scale = torch.empty(1, device=DEV)
    td.moonep_quantize_rows(x, q, scale)
    assert torch.equal(q.float(), torch.round(x)) and scale.item() == 1.0


def _check_quant(td, shape, kind, dtype, seed):
    R, E, K, S, B, n_in, n_out = shape
    n_in = (n_in + 15) // 16 * 16
    G, SK = E // R, S * K
    dims = _dims(td, R, E, K, S, B, dtype)
    table = _table(kind, R, E, K, S, B, seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    x, w, dup_w = i8(R, SK, n_in), i8(E, n_out, n_in), i8(R, B, n_out, n_in)
    x[..., 0] = -128
    w[..., 0] = -128
    xs = torch.rand((R, SK), generator=g, device=DEV)
    ws, dws = torch.rand((E, n_out), generator=g, device=DEV), torch.rand((R, B, n_out), generator=g, device=DEV)
    y = torch.full((R, SK, n_out), 3.0, dtype=torch_dtype(dtype), device=DEV)
    sums, _, written = plain_matmul(table, G, B, x, w, dup_w, True)  # exact: below 2^53
    factor = torch.zeros_like(sums)
    for r in range(R):
        for j in range(min(G + B, table.shape[1] - 1)):
            lo, hi = int(table[r, j]), int(table[r, j + 1])
            if lo >= 0 and hi > lo:
                factor[r, lo:hi] = (ws[r * G + j] if j < G else dws[r, j - G]).double()
    want = ((sums.float() * xs[..., None]) * factor.float()).to(y.dtype)
    say(f"quant {shape} {kind} {dtype}")
    td.moonep_expert_matmul_quant(dims, torch.from_numpy(table).to(DEV), x, xs, w, ws, dup_w, dws, y)
    torch.cuda.synchronize()
    assert torch.equal(y[written], want[written])
    assert bool((y[~written] == 3.0).all()), "a row of no segment was written"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_quant(td, kind, dtype):
    for i, shape in enumerate(SHAPES):
        _check_quant(td, shape, kind, dtype, 300 + i)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(td, seed):
    """Seeded random shapes of all four products."""
    rng = np.random.default_rng(seed)
    R, G = int(rng.integers(1, 5)), int(rng.integers(1, 9))
    E, S = R * G, int(2 ** rng.uniform(0, 9))
    K = int(rng.integers(1, min(E, 8) + 1))
    B = int(rng.integers(0, 5))
    n_in, n_out = (8 * int(2 ** rng.uniform(0, 7.5)) for _ in range(2))
    shape = (R, E, K, S, B, n_in, n_out)
    kind = KINDS[seed % 3]
    for transposed in (False, True):
        for dtype in ("bf16", "f32"):
            _check_matmul(td, shape, kind, dtype, transposed, 400 + seed)
            _check_wgrad(td, shape, kind, dtype, transposed, 500 + seed)
    _check_quant(td, shape, kind, "bf16", 600 + seed)


def test_tables_that_no_plan_makes(td):
    """Offsets past the rows, ends before their start and negative starts are empty or
    clamped as documented; nothing else is written."""
    R, E, K, S, B, n = 2, 8, 1, 40, 2, 64
    G = E // R
    dims = _dims(td, R, E, K, S, B, "bf16")
    for row in ([0, 4, -7, 4, 15, 15, 99999, 3, 9], [-1, 3, 9, -5, 12, 40, 41, 41, 50],
                [39, 40, 41, 42, 43, 44, 45, 46, 47], [5] * 9, [-1] * 9,
                [-2 ** 31, 2 ** 31 - 1, 0, 0, 8, 8, 16, 16, 16]):
        table = np.array([row, [0, 3, 3, 9, 20, 40, 40, -1, -1]], dtype=np.int32)
        x = _rand((R, S, n), "bf16", 1)
        w, dup_w = _rand((E, n, n), "bf16", 2), _rand((R, B, n, n), "bf16", 3)
        y = torch.full((R, S, n), 3.0, dtype=torch.bfloat16, device=DEV)
        want, mag, written = plain_matmul(table, G, B, x, w, dup_w, False)
        td.moonep_expert_matmul(dims, torch.from_numpy(table).to(DEV), x, w, dup_w, y)
        bound = mag * (n * ADD) + want.abs() * half_step(y.dtype) * 1.01
        assert_within(y[written], want[written], bound[written], f"{row}")
        assert bool((y[~written] == 3.0).all())
        home, dup = torch.full((E, n, n), 5.0, device=DEV), torch.full((R, B, n, n), 5.0, device=DEV)
        wh, wd, mh, md, wr = plain_wgrad(table, G, B, x, y, False)
        td.moonep_expert_matmul_wgrad(dims, torch.from_numpy(table).to(DEV), x, y, home, dup)
        assert_within(home, wh, mh * (S * ADD + 2.0 ** -23), f"{row} home")
        assert_within(dup[wr], wd[wr], md[wr] * (S * ADD + 2.0 ** -23), f"{row} dup")
        assert bool((dup[~wr] == 5.0).all())


def test_infinities_and_nans_stay_in_their_rows(td):
    R, E, K, S, B, n_in, n_out = 2, 4, 2, 100, 1, 96, 72
    dims = _dims(td, R, E, K, S, B, "bf16")
    table = _table("full", R, E, K, S, B, 5)
    seg = torch.from_numpy(table).to(DEV)
    x, w = _rand((R, S * K, n_in), "bf16", 1), _rand((E, n_in, n_out), "bf16", 2)
    dup_w = _rand((R, B, n_in, n_out), "bf16", 3)
    clean = torch.zeros((R, S * K, n_out), dtype=torch.bfloat16, device=DEV)
    td.moonep_expert_matmul(dims, seg, x, w, dup_w, clean)
    x[0, 7, 95], x[1, 199, 0] = float("nan"), float("inf")
    y = torch.zeros_like(clean)
    td.moonep_expert_matmul(dims, seg, x, w, dup_w, y)
    assert bool(y[0, 7].isnan().all()) and not bool(y[1, 199].isfinite().any())
    y[0, 7], y[1, 199] = clean[0, 7], clean[1, 199]
    assert torch.equal(y, clean)


def test_parts_of_blocks(td):
    """Matrices that are a part of each expert's block, as w[:, 1] of [E, 3, in, out], and
    gradients written into such a part: what lies between is left alone."""
    R, E, K, S, B, n_in, n_out = 2, 8, 2, 70, 3, 128, 64
    dims = _dims(td, R, E, K, S, B, "bf16")
    table = _table("full", R, E, K, S, B, 11)
    seg = torch.from_numpy(table).to(DEV)
    x, g = _rand((R, S * K, n_in), "bf16", 1), _rand((R, S * K, n_out), "bf16", 4)
    w, dup_w = _rand((E, 3, n_in, n_out), "bf16", 2), _rand((R, B, 3, n_in, n_out), "bf16", 3)
    y, y2 = (torch.zeros((R, S * K, n_out), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    td.moonep_expert_matmul(dims, seg, x, w[:, 1], dup_w[:, :, 1], y)
    td.moonep_expert_matmul(dims, seg, x, w[:, 1].contiguous(), dup_w[:, :, 1].contiguous(), y2)
    assert torch.equal(y, y2) and bool((y != 0).any())
    home, dup = torch.full((E, 3, n_in, n_out), 5.0, device=DEV), torch.full((R, B, 3, n_in, n_out), 5.0, device=DEV)
    home2, dup2 = torch.full((E, n_in, n_out), 5.0, device=DEV), torch.full((R, B, n_in, n_out), 5.0, device=DEV)
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home[:, 1], dup[:, :, 1])
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home2, dup2)
    assert torch.equal(home[:, 1], home2) and torch.equal(dup[:, :, 1], dup2)
    for part in (0, 2):
        assert bool((home[:, part] == 5.0).all()) and bool((dup[:, :, part] == 5.0).all())


def test_gradient_against_differences(td):
    """The product is linear in x and in the matrices, so differences along a direction
    equal the gradient's products with it, up to the outputs' own rounding."""
    R, E, K, S, B, n_in, n_out = 2, 6, 2, 60, 2, 96, 64
    dims = _dims(td, R, E, K, S, B, "f32")
    table = _table("full", R, E, K, S, B, 21)
    seg = torch.from_numpy(table).to(DEV)
    x, g = _rand((R, S * K, n_in), "f32", 1), _rand((R, S * K, n_out), "f32", 2)
    w, dup_w = _rand((E, n_in, n_out), "f32", 3), _rand((R, B, n_in, n_out), "f32", 4)
    dx, dw, ddw = _rand(x.shape, "f32", 5), _rand(w.shape, "f32", 6), _rand(dup_w.shape, "f32", 7)
    gx = torch.zeros_like(x)
    td.moonep_expert_matmul(dims, seg, g, w, dup_w, gx, transposed=True)  # w read as [out, in]
    home, dup = torch.zeros_like(w), torch.zeros_like(dup_w)
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home, dup)

    def loss(x, w, dup_w):
        y = torch.zeros((R, S * K, n_out), device=DEV)
        td.moonep_expert_matmul(dims, seg, x, w, dup_w, y)
        _, mag, _ = plain_matmul(table, E // R, B, x, w, dup_w, False)
        return (y.double() * g.double()).sum().item(), (mag * g.double().abs()).sum().item()

    (a, ma), (b, mb) = loss(x + dx, w, dup_w), loss(x - dx, w, dup_w)
    want = 2 * (gx.double() * dx.double()).sum().item()
    # sums of n_in (and, for gx, n_out) products; the rounding of x + dx itself: one step
    assert abs((a - b) - want) <= (ma + mb) * (n_in + n_out + 2) * ADD
    (a, ma), (b, mb) = loss(x, w + dw, dup_w + ddw), loss(x, w - dw, dup_w - ddw)
    want = 2 * ((home.double() * dw.double()).sum() + (dup.double() * ddw.double()).sum()).item()
    assert abs((a - b) - want) <= (ma + mb) * (n_in + S * K + 2) * ADD


def test_on_another_stream_and_in_a_graph(td):
    """The products on a side stream, and captured once and replayed on changed inputs
    between eager calls."""
    R, E, K, S, B, n_in, n_out = 2, 8, 2, 90, 2, 128, 192
    dims = _dims(td, R, E, K, S, B, "bf16")
    seg = torch.from_numpy(_table("full", R, E, K, S, B, 3)).to(DEV)
    x, g = _rand((R, S * K, n_in), "bf16", 1), _rand((R, S * K, n_out), "bf16", 2)
    w, dup_w = _rand((E, n_in, n_out), "bf16", 3), _rand((R, B, n_in, n_out), "bf16", 4)
    xs, q = torch.empty((R, S * K), device=DEV), torch.empty((R, S * K, n_in), dtype=torch.int8, device=DEV)
    wq, ws = torch.empty((E, n_out, n_in), dtype=torch.int8, device=DEV), torch.empty((E, n_out), device=DEV)
    dq, dws = torch.empty((R, B, n_out, n_in), dtype=torch.int8, device=DEV), torch.empty((R, B, n_out), device=DEV)
    td.moonep_quantize_rows(w.transpose(1, 2).contiguous(), wq, ws)
    td.moonep_quantize_rows(dup_w.transpose(2, 3).contiguous(), dq, dws)

    def outputs():
        return (torch.zeros((R, S * K, n_out), dtype=torch.bfloat16, device=DEV),
                torch.zeros((E, n_in, n_out), device=DEV), torch.zeros((R, B, n_in, n_out), device=DEV),
                torch.zeros((R, S * K, n_out), dtype=torch.bfloat16, device=DEV))

    def step(o):
        td.moonep_expert_matmul(dims, seg, x, w, dup_w, o[0])
        td.moonep_expert_matmul_wgrad(dims, seg, x, g, o[1], o[2])
        td.moonep_quantize_rows(x, q, xs)
        td.moonep_expert_matmul_quant(dims, seg, q, xs, wq, ws, dq, dws, o[3])

    eager, side = outputs(), outputs()
    step(eager)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(side)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, side))
    captured, graph = outputs(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for i in range(4):
        x.copy_(_rand(x.shape, "bf16", 10 + i))
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = outputs()
        step(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, captured)), f"replay {i}"


def test_a_table_from_the_plan(td):
    """Both plans' own tables: y of every row is its entry's row times its expert, and rows
    of duplicates without a slot (the water-fill needs more than B here) stay as they were."""
    R, E, K, S, B, n_in, n_out = 4, 16, 2, 64, 4, 64, 32
    for bounded in (False, True):
        dims = _dims(td, R, E, K, S, B, "f32", H=n_in)
        rng = np.random.default_rng(4)
        score = rng.normal(size=(R * S, E)) + rng.normal(size=E) * 1.5
        ids = np.argsort(-score, axis=1)[:, :K].reshape(R, S, K).astype(np.int32)
        plan, ids_d = run_plan(td, dims, ids, DEV, bounded=bounded)
        v = td.plan_views(dims, plan)
        w = _rand((E, n_in, n_out), "f32", 1)
        dup_w = torch.zeros((R, B, n_in, n_out), device=DEV)
        td.moonep_replicate(dims, plan, w, dup_w, 4 * n_in * n_out)
        hidden = _rand((R, S, n_in), "f32", 2)
        x = torch.zeros((R, S * K, n_in), device=DEV)
        td.moonep_dispatch(dims, plan, hidden, x)
        y = torch.zeros((R, S * K, n_out), device=DEV)
        td.moonep_expert_matmul(dims, v["seg_ptr"], x, w, dup_w, y)
        got = y.reshape(-1, n_out)[v["dst"].long()].reshape(R * S, K, n_out)
        rows, we = hidden.reshape(R * S, 1, n_in).double(), w.double()[ids_d.long().reshape(R * S, K)]
        want = (rows.unsqueeze(-1) * we).sum(2)
        mag = (rows.unsqueeze(-1) * we).abs().sum(2)
        table = v["seg_ptr"].cpu().numpy()
        _, _, written = plain_matmul(table, E // R, B, x, w, dup_w, False)
        has = written.reshape(-1)[v["dst"].long()].reshape(R * S, K)
        assert bool(has.all()) == (int(v["n_dup"].max()) <= B)
        bound = mag * (n_in * ADD) + want.abs() * 2.0 ** -23
        assert_within(got[has], want[has], bound[has], f"bounded={bounded}")
        assert bool((got[~has] == 0).all())


def test_offsets_past_32_bits(td):
    """Rows, outputs and gradients whose byte offsets pass 2^32 and element offsets 2^31."""
    R, E, K, S, B, wide, n = 2, 2, 1, 160000, 0, 7168, 64
    dims = _dims(td, R, E, K, S, B, "bf16")
    table = make_table([[S], [S]], R, 1, 1, S)
    seg = torch.from_numpy(table).to(DEV)
    x = torch.empty((R, S, wide), dtype=torch.bfloat16, device=DEV)
    assert x.numel() > 2 ** 31
    for r in range(R):
        x[r] = _rand((S, wide), "bf16", 1 + r)
    w = _rand((E, wide, n), "bf16", 3)
    y = torch.zeros((R, S, n), dtype=torch.bfloat16, device=DEV)
    say(f"wide rows: {x.numel() * 2} bytes")
    td.moonep_expert_matmul(dims, seg, x, w, None, y)
    rows = torch.tensor([0, 1, 77777, S - 257, S - 2, S - 1], device=DEV)
    for r in range(R):
        a, m = x[r, rows].double(), w[r].double()
        want, mag = a @ m, a.abs() @ m.abs()
        assert_within(y[r, rows], want, mag * (wide * ADD) + want.abs() * half_step(y.dtype) * 1.01, "y")
    # the gradient of the rows: wide outputs
    gx = torch.zeros_like(x)
    td.moonep_expert_matmul(dims, seg, y, w, None, gx, transposed=True)
    for r in range(R):
        a, m = y[r, rows].double(), w[r].double().t().contiguous()
        want, mag = a @ m, a.abs() @ m.abs()
        assert_within(gx[r, rows], want, mag * (n * ADD) + want.abs() * half_step(y.dtype) * 1.01, "gx")
    del gx
    home = torch.zeros((E, wide, n), device=DEV)
    td.moonep_expert_matmul_wgrad(dims, seg, x, y, home, None)
    cols = torch.tensor([0, 3000, 7100, 7167], device=DEV)
    for r in range(R):
        a, g = x[r][:, cols].double(), y[r].double()
        want, mag = a.t().contiguous() @ g, a.abs().t().contiguous() @ g.abs()
        assert_within(home[r, cols], want, mag * (S * ADD + 2.0 ** -23), "home")
    q, scale = torch.empty(x.shape, dtype=torch.int8, device=DEV), torch.empty((R, S), device=DEV)
    td.moonep_quantize_rows(x, q, scale)
    for r in range(R):
        want_q, want_s = _plain_quantise(x[r, rows])
        assert np.array_equal(q[r, rows].cpu().numpy(), want_q)
        assert np.array_equal(scale[r, rows].cpu().numpy(), want_s)


def test_two_calls_at_once(td):
    """Calls on two streams share nothing but their inputs."""
    R, E, K, S, B, n_in, n_out = 8, 32, 2, 300, 2, 264, 520
    dims = _dims(td, R, E, K, S, B, "bf16")
    tables = [torch.from_numpy(_table("full", R, E, K, S, B, i)).to(DEV) for i in (1, 2)]
    x, g = _rand((R, S * K, n_in), "bf16", 1), _rand((R, S * K, n_out), "bf16", 2)
    w, dup_w = _rand((E, n_in, n_out), "bf16", 3), _rand((R, B, n_in, n_out), "bf16", 4)

    def outputs():
        return (torch.zeros((R, S * K, n_out), dtype=torch.bfloat16, device=DEV),
                torch.zeros((E, n_in, n_out), device=DEV), torch.zeros((R, B, n_in, n_out), device=DEV))

    def step(seg, o):
        td.moonep_expert_matmul(dims, seg, x, w, dup_w, o[0])
        td.moonep_expert_matmul_wgrad(dims, seg, x, g, o[1], o[2])

    alone, both = [outputs() for _ in tables], [outputs() for _ in tables]
    for seg, o in zip(tables, alone):
        step(seg, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in tables]
    for _ in range(5):
        for s, seg, o in zip(streams, tables, both):
            with torch.cuda.stream(s):
                step(seg, o)
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_binding_refusals(td):
    """What the binding refuses before the library is called: nothing is written."""
    R, E, K, S, B, n_in, n_out = 2, 8, 2, 16, 2, 64, 32
    dims = _dims(td, R, E, K, S, B, "bf16")
    bf, f32 = torch.bfloat16, torch.float32
    seg = torch.from_numpy(_table("full", R, E, K, S, B, 1)).to(DEV)
    good = dict(seg_ptr=seg, x=_rand((R, S * K, n_in), "bf16", 1), w=_rand((E, n_in, n_out), "bf16", 2),
                dup_w=_rand((R, B, n_in, n_out), "bf16", 3),
                y=torch.full((R, S * K, n_out), 3.0, dtype=bf, device=DEV))
    td.moonep_expert_matmul(dims, **dict(good, y=good["y"].clone()))
    bad = [("x", good["x"].float(), TypeError), ("x", good["x"][:, :-1], ValueError),
           ("x", good["x"].cpu(), ValueError), ("y", good["y"].transpose(0, 1), ValueError),
           ("y", good["y"].cpu(), ValueError), ("y", None, TypeError), ("x", [1], TypeError),
           ("w", good["w"][:-1], ValueError), ("w", good["w"].transpose(1, 2), ValueError),
           ("w", good["w"].transpose(1, 2).contiguous().transpose(1, 2), ValueError),
           ("dup_w", None, TypeError), ("dup_w", good["dup_w"][:, :1], ValueError),
           ("dup_w", torch.zeros((R, B, 3, n_in, n_out), dtype=bf, device=DEV)[:, :, 0], ValueError),
           ("seg_ptr", seg.long(), TypeError), ("seg_ptr", seg[:, :-1], ValueError),
           ("seg_ptr", seg.cpu(), ValueError)]
    for name, value, error in bad:
        with pytest.raises(error):
            td.moonep_expert_matmul(dims, **dict(good, **{name: value}))
    with pytest.raises(td.MoonEPError) as err:  # rows that are not whole 16 bytes
        td.moonep_expert_matmul(dims, seg, _rand((R, S * K, 12), "bf16", 1), _rand((E, 12, n_out), "bf16", 2),
                                _rand((R, B, 12, n_out), "bf16", 3), good["y"])
    assert err.value.rc == td.ERR_SIZE
    home, dup = torch.zeros((E, n_in, n_out), device=DEV), torch.zeros((R, B, n_in, n_out), device=DEV)
    for args in ((good["x"], good["y"], home.to(bf), dup), (good["x"], good["y"], home, dup[:1]),
                 (good["x"], good["y"][:, 1:], home, dup)):
        with pytest.raises((TypeError, ValueError)):
            td.moonep_expert_matmul_wgrad(dims, seg, *args)
    q, scale = torch.empty((4, 64), dtype=torch.int8, device=DEV), torch.empty(4, device=DEV)
    for args in ((torch.zeros((4, 64), dtype=torch.float16, device=DEV), q, scale),
                 (torch.zeros((4, 128), device=DEV)[:, ::2], q, scale),
                 (torch.zeros((4, 64), device=DEV), q.float(), scale),
                 (torch.zeros((4, 64), device=DEV), q, scale[:3]), (torch.zeros((4, 64)), q, scale)):
        with pytest.raises((TypeError, ValueError)):
            td.moonep_quantize_rows(*args)
    g = torch.zeros(8, device=DEV)
    for grads, outs in (([g, g], None), ([g], [g.to(bf)]), ([g], [g[:4]]), ([g, g.cpu()], None),
                        ([torch.zeros((4, 4), device=DEV).t()], None), ([g.half()], None)):
        with pytest.raises((TypeError, ValueError)):
            td.GradList(grads, outs)
    with pytest.raises(ValueError):
        td.moonep_grad_sumsq([g], torch.zeros(16, dtype=torch.float64, device=DEV))
    with pytest.raises(td.MoonEPError):
        td.moonep_grad_clip([g], td.new_norm_buffer(DEV), -1.0)
    torch.cuda.synchronize()
    assert bool((good["y"] == 3.0).all()) and f32 == scale.dtype


def _whole(shape, dtype, seed):
    """Whole numbers from -2 to 2: their products' sums are whole and, below 2^24, exact in
    binary32 in every order, so that one lost or repeated row or chunk shows."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = torch.empty(shape, dtype=torch_dtype(dtype), device=DEV)
    for part in out:
        part.copy_(torch.randint(-2, 3, part.shape, generator=g, device=DEV, dtype=torch.int8))
    return out


def _check_exact(td, shape, kind, dtype, transposed, seed):
    R, E, K, S, B, n_in, n_out = shape
    G, SK = E // R, S * K
    assert 4 * max(n_in, SK) < 2 ** 24
    dims = _dims(td, R, E, K, S, B, dtype)
    table = _table(kind, R, E, K, S, B, seed)
    seg = torch.from_numpy(table).to(DEV)
    tail = (n_out, n_in) if transposed else (n_in, n_out)
    x, g = _whole((R, SK, n_in), dtype, seed), _whole((R, SK, n_out), dtype, seed + 1)
    w, dup_w = _whole((E,) + tail, dtype, seed + 2), _whole((R, B) + tail, dtype, seed + 3)
    y = torch.full((R, SK, n_out), 3.0, dtype=x.dtype, device=DEV)
    home, dup = torch.full((E,) + tail, 5.0, device=DEV), torch.full((R, B) + tail, 5.0, device=DEV)
    say(f"exact {shape} {kind} {dtype} transposed={transposed}")
    td.moonep_expert_matmul(dims, seg, x, w, dup_w, y, transposed=transposed)
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home, dup, transposed=transposed)
    want, _, written = plain_matmul(table, G, B, x, w, dup_w, transposed)
    assert torch.equal(y[written], want[written].to(y.dtype)) and bool((y[~written] == 3.0).all())
    del want
    want_h, want_d, _, _, slots = plain_wgrad(table, G, B, x, g, transposed)
    assert torch.equal(home, want_h.float())
    assert torch.equal(dup[slots], want_d[slots].float()) and bool((dup[~slots] == 5.0).all())


# long rows and long segments, beside the shapes above
LONG = [
    (1, 2, 1, 64, 1, 16392, 72),
    (2, 4, 2, 40, 2, 7176, 264),
    (2, 2, 1, 20011, 0, 72, 136),
    (8, 8, 1, 6007, 0, 264, 264),
    (1, 1, 1, 3, 0, 40008, 24),
]


@pytest.mark.parametrize("transposed", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + LARGE + TILES + LONG, ids=lambda s: "x".join(map(str, s)))
def test_exact_sums(td, shape, dtype, transposed):
    for kind in ("full", "behind"):
        _check_exact(td, shape, kind, dtype, transposed, 900)


def test_exact_sums_past_32_bits(td):
    """Every sum of a gradient over 160000 rows whose byte offsets pass 2^32, and every
    output of the products over them, bit for bit."""
    R, E, K, S, B, wide, n = 2, 2, 1, 160000, 0, 7168, 64
    dims = _dims(td, R, E, K, S, B, "bf16")
    seg = torch.from_numpy(make_table([[S], [S]], R, 1, 1, S)).to(DEV)
    x, g = _whole((R, S, wide), "bf16", 1), _whole((R, S, n), "bf16", 2)
    assert x.numel() > 2 ** 31
    home = torch.full((E, wide, n), 5.0, device=DEV)
    other = torch.full((E, n, wide), 5.0, device=DEV)
    say(f"wide gradient: {x.numel() * 2} bytes")
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home, None)
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, other, None, transposed=True)
    for r in range(R):
        b = g[r].double()
        for c in range(0, wide, 1024):
            want = x[r, :, c:c + 1024].double().t().contiguous() @ b
            assert torch.equal(home[r, c:c + 1024], want.float()), (r, c)
            assert torch.equal(other[r, :, c:c + 1024], want.float().t()), (r, c)
    w = _whole((E, wide, n), "bf16", 3)
    y = torch.full((R, S, n), 9.0, dtype=torch.bfloat16, device=DEV)
    td.moonep_expert_matmul(dims, seg, x, w, None, y)
    gx = torch.full_like(x, 9.0)
    td.moonep_expert_matmul(dims, seg, g, w, None, gx, transposed=True)
    for r in range(R):
        m = w[r].double()
        for at in range(0, S, 20000):
            part = slice(at, at + 20000)
            assert torch.equal(y[r, part], (x[r, part].double() @ m).bfloat16()), (r, at)
            want = g[r, part].double() @ m.t().contiguous()
            assert torch.equal(gx[r, part], want.bfloat16()), (r, at)


@pytest.mark.parametrize("transposed", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_outputs_past_the_caches(td, dtype, transposed):
    """Outputs and gradients of 256 MB and more, which are stored past the caches, in the
    widest tiles and in narrow ones."""
    gradients = [(2, 16, 2, 300, 1, 2056, 2104), (2, 256, 1, 60, 0, 520, 520)]
    outputs = [(2, 16, 2, 18000, 1, 40, 2104), (8, 64, 4, 4500, 2, 1032, 1032), (4, 32, 4, 9000, 2, 24, 936)]
    for shape in gradients + outputs:
        R, E, K, S, B, n_in, n_out = shape
        if shape in gradients:
            assert 4 * E * n_in * n_out >= 1 << 28
        else:
            assert 2 * R * S * K * n_out >= 1 << 28
        _check_exact(td, shape, "full", dtype, transposed, 950)


# both sides of each change of the rows' width: 32, 128, 256, 512 and 1024 chunks of 16 bytes
WIDTHS = {"bf16": [256, 272, 1024, 1040, 2032, 2048, 2064, 4080, 4096, 4112, 8176, 8192, 8208],
          "f32": [112, 128, 144, 512, 528, 1008, 1024, 1040, 2032, 2048, 2064, 4080, 4096, 4112]}


@pytest.mark.parametrize("dtype,cols", [(d, c) for d in WIDTHS for c in WIDTHS[d]])
def test_quantize_at_every_width(td, dtype, cols):
    for n in (1, 19, 130):
        x = _rand((n, cols), dtype, n + cols, 3.0)
        x[0, cols - 1] = -50.0          # the largest magnitude in the last chunk
        if n > 10:
            x[1] = 0.0
            x[2, cols - 2] = float("nan")
            x[3, 0] = float("inf")
            x[4] *= 2.0 ** -112
            x[n - 1, cols // 2] = 3.0e38
        q = torch.full((n + 1, cols), 77, dtype=torch.int8, device=DEV)
        scale = torch.full((n + 4,), 7.0, device=DEV)
        td.moonep_quantize_rows(x, q[:n], scale[:n])
        want_q, want_s = _plain_quantise(x)
        assert np.array_equal(q[:n].cpu().numpy(), want_q), (n, cols)
        assert np.array_equal(scale[:n].cpu().numpy(), want_s, equal_nan=True), (n, cols)
        assert bool((q[n] == 77).all()) and bool((scale[n:] == 7.0).all())


@pytest.mark.parametrize("dtype,n,cols", [("bf16", 100003, 2736), ("f32", 40001, 6720), ("bf16", 8003, 40016)])
def test_quantize_past_the_caches(td, dtype, n, cols):
    """256 MB of 8-bit values and more, every one of them."""
    assert n * cols >= 1 << 28
    x = _rand((n, cols), dtype, cols)
    q, scale = torch.empty((n, cols), dtype=torch.int8, device=DEV), torch.empty((n,), device=DEV)
    td.moonep_quantize_rows(x, q, scale)
    a = np.maximum(x.float().abs().amax(dim=1).cpu().numpy(), np.float32(2.0 ** -100))
    assert np.array_equal(scale.cpu().numpy(), a / np.float32(127.0))
    inv = torch.from_numpy(np.float32(127.0) / a).to(DEV)  # divided on the host, correctly rounded
    for at in range(0, n, 10000):
        part = slice(at, at + 10000)
        want = torch.round(x[part].float() * inv[part, None]).to(torch.int8)
        assert torch.equal(q[part], want), at


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_rank_by_itself(td, dtype):
    """A rank that has a GPU of its own makes its part alone: one rank whose experts are the
    home experts and then the duplicates, their matrices in one array. Exact sums, so the
    parts are the same bits as the call for all ranks."""
    R, E, K, S, B, n_in, n_out = 4, 16, 2, 90, 3, 264, 136
    G, SK = E // R, S * K
    dims = _dims(td, R, E, K, S, B, dtype)
    table = _table("over", R, E, K, S, B, 31)
    seg = torch.from_numpy(table).to(DEV)
    x, g = _whole((R, SK, n_in), dtype, 1), _whole((R, SK, n_out), dtype, 2)
    w, dup_w = _whole((E, n_in, n_out), dtype, 3), _whole((R, B, n_in, n_out), dtype, 4)
    y = torch.full((R, SK, n_out), 3.0, dtype=x.dtype, device=DEV)
    home, dup = torch.full((E, n_in, n_out), 5.0, device=DEV), torch.full((R, B, n_in, n_out), 5.0, device=DEV)
    td.moonep_expert_matmul(dims, seg, x, w, dup_w, y)
    td.moonep_expert_matmul_wgrad(dims, seg, x, g, home, dup)
    alone = _dims(td, 1, G + B, 1, SK, 0, dtype)
    for r in range(R):
        own = torch.full((1, G + B + 2), -1, dtype=torch.int32, device=DEV)
        own[0, :G + B + 1] = seg[r, :G + B + 1]
        held = torch.cat([w[r * G:(r + 1) * G], dup_w[r]])
        yr = torch.full((1, SK, n_out), 3.0, dtype=x.dtype, device=DEV)
        grads = torch.full((G + B, n_in, n_out), 5.0, device=DEV)
        td.moonep_expert_matmul(alone, own, x[r:r + 1], held, None, yr)
        td.moonep_expert_matmul_wgrad(alone, own, x[r:r + 1], g[r:r + 1], grads, None)
        assert torch.equal(yr[0], y[r])
        assert torch.equal(grads[:G], home[r * G:(r + 1) * G])
        used = seg[r, G + 1:G + B + 1] >= 0
        assert bool(used.any()) and torch.equal(grads[G:][used], dup[r][used])
        assert bool((grads[G:][~used] == 0).all())  # home experts without rows here: zeros
