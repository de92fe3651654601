"""The norm, the gated activation and rows in 4 bits on the GPU, against their plain forms.

Tolerances, with U = 2^-24 (half a step of binary32): the norm's inverse and its two products
are off by U each (its sum is binary64), and a store by half a step of its type. What goes to
8 or 4 bits follows a rule given in binary32, and is compared bit for bit. The activation's
bounds stand with its plain form; the gradients' sums of n terms in binary32 are within
n 2^-23 sum |terms| whatever their order.
"""
import pytest
import torch

from tests.expert_common import ADD, assert_within, half_step, torch_dtype
from tests.gpu_common import say
from tests.layer_common import (U, mx_pack, mx_quantise, plain_norm, plain_swiglu,
                                plain_swiglu_backward, quantise8, scale_cols)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-6


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


def _small(dtype):
    """The least magnitude a type holds: what a rounding below its normal numbers is off by."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def same_bits(a, b, what):
    """Equal values, NaN alike and zeros of one sign."""
    a, b = a.contiguous(), b.contiguous()
    assert a.dtype == b.dtype and a.shape == b.shape, what
    raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    nan = torch.isnan(a) & torch.isnan(b) if a.is_floating_point() else torch.zeros_like(a, dtype=torch.bool)
    bad = (a.view(raw) != b.view(raw)) & ~nan
    if bool(bad.any()):
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {i}: "
                             f"{a.reshape(-1)[i].item()} for {b.reshape(-1)[i].item()}")


# rows, cols of the smallest unit (8, 16 or 32) times this: from one chunk to rows read twice
SHAPES = [(1, 1), (3, 2), (1, 28), (2, 33), (7, 64), (65, 5), (5, 129), (2, 224), (300, 16), (1, 512),
          (9, 513), (3, 1024), (2, 2200)]
# rows enough that a wave takes one each
MANY = [(2048, 70), (2500, 40)]


def _norm_inputs(shape, dtype, seed, residual):
    rows, cols = shape
    x = _rand((rows, cols), dtype, seed) * torch.exp2(
        torch.randint(-6, 7, (rows, 1), device=DEV, generator=torch.Generator(DEV).manual_seed(seed))).to(
        torch_dtype(dtype))
    gamma = 1 + 0.3 * _rand((cols,), dtype, seed + 1)
    return x, gamma, _rand((rows, cols), dtype, seed + 2) if residual else None


def _check_norm(td, shape, dtype, residual, out, seed):
    x, gamma, res = _norm_inputs(shape, dtype, seed, residual)
    say(f"norm {shape} {dtype} residual={residual} {out}")
    h, v32, want, inv = plain_norm(x, gamma, EPS, res)
    s = torch.full_like(x, 7.0)
    got_inv = torch.empty(shape[0], dtype=torch.float32, device=DEV)
    args = dict(residual=res, sum_out=s, inv_rms=got_inv)
    if out == "same":
        y = torch.empty_like(x)
        td.moonep_rmsnorm(x, gamma, y, EPS, **args)
        bound = want.abs() * (3.1 * U + half_step(x.dtype) * 1.01) + _small(x.dtype)
        assert_within(y, want, bound, "out")
    elif out == "int8":
        q, scale = torch.empty_like(x, dtype=torch.int8), torch.empty_like(got_inv)
        td.moonep_rmsnorm_quant(x, gamma, q, scale, EPS, **args)
        wq, ws = quantise8(v32)
        same_bits(scale, ws, "scale")
        same_bits(q, wq, "q")
    else:
        q = torch.empty((shape[0], shape[1] // 2), dtype=torch.uint8, device=DEV)
        scale = torch.full((shape[0], scale_cols(shape[1])), 9, dtype=torch.uint8, device=DEV)
        td.moonep_rmsnorm_mx(x, gamma, q, scale, EPS, **args)
        wq, ws = mx_pack(*mx_quantise(v32))
        same_bits(scale, ws, "scale")
        same_bits(q, wq, "q")
    same_bits(s, h, "sum")
    assert_within(got_inv, inv, inv * (1.01 * U), "inv_rms")


@pytest.mark.parametrize("out,unit", [("same", 8), ("int8", 16), ("mx", 32)])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm(td, dtype, residual, out, unit):
    for i, (rows, n) in enumerate(SHAPES + MANY):
        _check_norm(td, (rows, n * unit), dtype, residual, out, 10 * i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place(td, dtype):
    """sum_out where the residual lies and out where x does, and the other way round; rows in
    registers and rows read again."""
    for rows, cols in ((3, 512), (2500, 1024), (2, 40960)):
        x, gamma, res = _norm_inputs((rows, cols), dtype, rows, True)
        want, s = torch.empty_like(x), torch.empty_like(x)
        td.moonep_rmsnorm(x, gamma, want, EPS, residual=res, sum_out=s)
        a, b = x.clone(), res.clone()
        td.moonep_rmsnorm(a, gamma, a, EPS, residual=b, sum_out=b)
        same_bits(a, want, "out over x")
        same_bits(b, s, "sum over residual")
        a, b = x.clone(), res.clone()
        td.moonep_rmsnorm(a, gamma, b, EPS, residual=b, sum_out=a)
        same_bits(b, want, "out over residual")
        same_bits(a, s, "sum over x")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_extremes(td, dtype):
    """Zeros, values whose squares pass binary32's range and fall below it, infinities, NaN."""
    cols = 64
    x = _rand((8, cols), dtype, 3)
    x[0] = 0
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -100
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5] = torch.finfo(x.dtype).max / 4
    x[6] = torch.finfo(x.dtype).tiny
    gamma = torch.ones(cols, dtype=x.dtype, device=DEV)
    for eps in (EPS, 0.0):
        h, v32, want, inv = plain_norm(x, gamma, eps)
        y, got = torch.empty_like(x), torch.empty(8, dtype=torch.float32, device=DEV)
        td.moonep_rmsnorm(x, gamma, y, eps, inv_rms=got)
        for r in (0, 1, 2, 5, 6, 7):
            if r == 0 and eps == 0:
                assert bool(torch.isnan(y[0]).all()) and bool(torch.isinf(got[0]))
                continue
            bound = want[r].abs() * (3.1 * U + half_step(x.dtype) * 1.01) + _small(x.dtype)
            assert_within(y[r], want[r], bound, f"row {r}")
        assert got[3] == 0 and bool(torch.isnan(y[3, 5])) and bool((y[3, :5] == 0).all())
        assert bool(torch.isnan(y[4]).all()) and bool(torch.isnan(got[4]))
    q, s = torch.empty_like(x, dtype=torch.int8), torch.empty(8, device=DEV)
    td.moonep_rmsnorm_quant(x, gamma, q, s, EPS)
    wq, ws = quantise8(plain_norm(x, gamma, EPS)[1])
    same_bits(s, ws, "scale")
    same_bits(q, wq, "q")
    q, s = (torch.empty((8, n), dtype=torch.uint8, device=DEV) for n in (32, 4))
    td.moonep_rmsnorm_mx(x, gamma, q, s, EPS)
    wq, ws = mx_pack(*mx_quantise(plain_norm(x, gamma, EPS)[1]))
    same_bits(s, ws, "scale")
    same_bits(q, wq, "q")


def _check_backward(td, shape, dtype, with_sum, seed):
    rows, cols = shape
    x, gamma, _ = _norm_inputs(shape, dtype, seed, False)
    go = _rand(shape, dtype, seed + 3)
    gs = _rand(shape, dtype, seed + 4) if with_sum else None
    say(f"norm backward {shape} {dtype} grad_sum={with_sum}")
    inv32 = plain_norm(x, gamma, EPS)[3].float()
    inv, t = inv32.double()[:, None], go.double() * gamma.double()
    xh = x.double() * inv
    mean = (t * xh).mean(1, keepdim=True)
    want = inv * (t - xh * mean) + (gs.double() if with_sum else 0)
    # mean: cols additions and four roundings a term; then six roundings of what is added
    off = (t * xh).abs().sum(1, keepdim=True) * (ADD + 5 * U / cols)
    bound = inv * (xh.abs() * off + (t.abs() + (xh * mean).abs()) * (6 * U))
    bound = bound + (gs.double().abs() if with_sum else 0) * U + want.abs() * half_step(x.dtype) * 1.01 + _small(x.dtype)
    terms = go.double() * xh
    gg_bound = terms.abs().sum(0) * (rows * ADD + 3 * U)
    gx, gg = torch.empty_like(x), torch.full((cols,), 5.0, device=DEV)
    work = td.new_norm_workspace(cols, DEV).fill_(float("nan"))
    td.moonep_rmsnorm_backward(go, x, gamma, inv32, gx, gg, work, grad_sum=gs)
    assert_within(gx, want, bound, "grad_x")
    assert_within(gg, terms.sum(0), gg_bound, "grad_gamma")
    again, gg2 = go.clone(), torch.empty_like(gg)
    td.moonep_rmsnorm_backward(again, x, gamma, inv32, again, gg2, work, grad_sum=gs)
    same_bits(again, gx, "grad_x where grad_out lies")
    same_bits(gg2, gg, "grad_gamma again")
    if with_sum:
        over = gs.clone()
        td.moonep_rmsnorm_backward(go, x, gamma, inv32, over, None, None, grad_sum=over)
        same_bits(over, gx, "grad_x where grad_sum lies")


@pytest.mark.parametrize("with_sum", [False, True], ids=["plain", "sum"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_backward(td, dtype, with_sum):
    for i, shape in enumerate([(1, 8), (3, 40), (1, 2048), (5, 1032), (700, 520), (1500, 64), (9000, 136),
                               (40, 4104), (13, 8192), (6, 16392), (3, 40000)]):
        _check_backward(td, shape, dtype, with_sum, 20 * i)


def test_norm_backward_of_no_rows(td):
    x, g = torch.empty((0, 64), device=DEV), torch.ones(64, device=DEV)
    gg = torch.full((64,), 3.0, device=DEV)
    td.moonep_rmsnorm_backward(x, x, g, torch.empty(0, device=DEV), x, gg, td.new_norm_workspace(64, DEV))
    assert bool((gg == 0).all())
    td.moonep_rmsnorm(x, g, x, EPS)
    td.moonep_swiglu(x, x, x)


def test_norm_gradient_by_differences(td):
    """grad_x and grad_gamma against central differences of the library's own forward pass, in
    binary32: with a step of 2^-6 the third derivative adds less than 2^-12 of a unit-sized
    function's slope, and the sum's rounding 2^-24 * 64 / 2^-6."""
    rows, cols = 2, 16
    x, gamma, go = _rand((rows, cols), "f32", 1), 1 + 0.2 * _rand((cols,), "f32", 2), _rand((rows, cols), "f32", 3)
    y, inv = torch.empty_like(x), torch.empty(rows, device=DEV)

    def loss(x, gamma):
        td.moonep_rmsnorm(x, gamma, y, EPS, inv_rms=inv)
        return float((y.double() * go.double()).sum())

    loss(x, gamma)
    gx, gg = torch.empty_like(x), torch.empty(cols, device=DEV)
    td.moonep_rmsnorm_backward(go, x, gamma, inv.clone(), gx, gg, td.new_norm_workspace(cols, DEV))
    step = 2.0 ** -6
    for r, c in ((0, 0), (0, 7), (1, 15)):
        d = torch.zeros_like(x)
        d[r, c] = step
        slope = (loss(x + d, gamma) - loss(x - d, gamma)) / (2 * step)
        assert abs(slope - float(gx[r, c])) < 5e-3, (r, c)
    for c in (0, 9):
        d = torch.zeros_like(gamma)
        d[c] = step
        slope = (loss(x, gamma + d) - loss(x, gamma - d)) / (2 * step)
        assert abs(slope - float(gg[c])) < 1e-3, c


# ------------------------------------------------------------------ activation

def _halves(rows, n, dtype, seed, kind):
    if kind == "apart":
        return _rand((rows, n), dtype, seed, 2.0), _rand((rows, n), dtype, seed + 1, 2.0)
    h = _rand((rows, 2 * n), dtype, seed, 2.0)
    return h[:, :n], h[:, n:]


@pytest.mark.parametrize("out,unit", [("same", 8), ("int8", 16), ("mx", 32)])
@pytest.mark.parametrize("kind", ["apart", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu(td, dtype, kind, out, unit):
    for i, (rows, n) in enumerate(SHAPES + MANY):
        cols = n * unit
        g, u = _halves(rows, cols, dtype, 7 * i, kind)
        say(f"swiglu {(rows, cols)} {dtype} {kind} {out}")
        want, bound = plain_swiglu(g, u)
        y = torch.empty((rows, cols), dtype=g.dtype, device=DEV)
        td.moonep_swiglu(g, u, y)
        assert_within(y, want, bound + want.abs() * half_step(y.dtype) * 1.01 + _small(y.dtype), "out")
        if out == "same":
            continue
        # what is quantised is the binary32 value, which rows of binary32 show
        v32 = torch.empty((rows, cols), dtype=torch.float32, device=DEV)
        td.moonep_swiglu(g.float().contiguous(), u.float().contiguous(), v32)
        if out == "int8":
            q, s = torch.empty_like(v32, dtype=torch.int8), torch.empty(rows, device=DEV)
            td.moonep_swiglu_quant(g, u, q, s)
            wq, ws = quantise8(v32)
        else:
            q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
            s = torch.full((rows, scale_cols(cols)), 9, dtype=torch.uint8, device=DEV)
            td.moonep_swiglu_mx(g, u, q, s)
            wq, ws = mx_pack(*mx_quantise(v32))
        same_bits(s, ws, "scale")
        same_bits(q, wq, "q")


@pytest.mark.parametrize("kind", ["apart", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_backward(td, dtype, kind):
    for i, (rows, n) in enumerate(SHAPES + MANY):
        cols = 8 * n
        g, u = _halves(rows, cols, dtype, 9 * i, kind)
        go = _rand((rows, cols), dtype, 9 * i + 5)
        dg, du = _halves(rows, cols, dtype, 1, kind)
        td.moonep_swiglu_backward(go, g, u, dg, du)
        wg, bg, wu, bu = plain_swiglu_backward(go, g, u)
        for got, want, bound, what in ((dg, wg, bg, "grad_gate"), (du, wu, bu, "grad_up")):
            assert_within(got, want, bound + want.abs() * half_step(got.dtype) * 1.01 + _small(got.dtype), what)
        td.moonep_swiglu_backward(go, g, u, g, u)  # where the values lie
        same_bits(g, dg, "grad_gate over gate")
        same_bits(u, du, "grad_up over up")


def test_swiglu_of_extremes(td):
    g = torch.tensor([0.0, -0.0, 90.0, -90.0, 1e30, -1e30, float("inf"), float("nan"), 88.0, -88.0, -104.0, 1e-40] + [1.0] * 4, device=DEV)
    u = torch.ones_like(g)
    y = torch.empty_like(g)
    td.moonep_swiglu(g, u, y)
    want = torch.nan_to_num(g.double() * torch.sigmoid(g.double()), nan=0.0, posinf=0.0)
    fine = torch.isfinite(g)
    assert_within(y[fine], want[fine], want[fine].abs() * (8 * U) + 2.0 ** -119, "out")
    assert float(y[6]) == float("inf") and bool(torch.isnan(y[7]))


def test_swiglu_rows_of_more_dims(td):
    """[R, S, n] rows at one distance, as halves of a product's output; others are refused."""
    h = _rand((3, 5, 48), "bf16", 1)
    y, want = torch.empty((3, 5, 24), dtype=h.dtype, device=DEV), torch.empty((15, 24), dtype=h.dtype, device=DEV)
    td.moonep_swiglu(h[..., :24], h[..., 24:], y)
    td.moonep_swiglu(h.view(15, 48)[:, :24].contiguous(), h.view(15, 48)[:, 24:].contiguous(), want)
    same_bits(y.view(15, 24), want, "out")
    big = _rand((3, 8, 48), "bf16", 1)
    for gate, up in ((big[:, :5, :24], big[:, :5, 24:]),     # rows at two distances
                     (h[..., :24], h[..., 24:].contiguous()),  # gate and up at different ones
                     (h[..., ::2], h[..., 1::2])):
        with pytest.raises(ValueError):
            td.moonep_swiglu(gate, up, y)


# ------------------------------------------------------------------ rows in 4 bits

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_mx(td, dtype):
    for i, (rows, n) in enumerate(SHAPES + MANY):
        cols = 32 * n
        x = _rand((rows, cols), dtype, 5 * i, 3.0)
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
        s = torch.full((rows, scale_cols(cols)), 9, dtype=torch.uint8, device=DEV)
        td.moonep_quantize_rows_mx(x, q, s)
        wq, ws = mx_pack(*mx_quantise(x.float()))
        same_bits(s, ws, f"scale of {(rows, cols)}")
        same_bits(q, wq, f"q of {(rows, cols)}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_mx_of_extremes(td, dtype):
    """Every exponent the type has, ties, the border where the scale doubles, infinities."""
    m = torch.tensor([0.0, 0.25, 0.26, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 5.01, 6.0,
                      6.5, 6.96875, 7.0, 7.5, -0.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0, -7.0, 0.125],
                     dtype=torch.float64, device=DEV)
    rows = []
    for e in range(-152, 126):
        rows.append(m * 2.0 ** e)
        rows.append(torch.where(m.abs() < 7, m, torch.zeros_like(m)) * 2.0 ** e)
    x = torch.stack(rows).to(torch_dtype(dtype))
    x = torch.cat([x, torch.full_like(x[:1], torch.finfo(x.dtype).max), torch.zeros_like(x[:1])])
    for bad in (float("inf"), float("-inf"), float("nan")):
        row = x[300:301].clone()
        row[0, 17] = bad
        x = torch.cat([x, row])
    q = torch.empty((x.shape[0], 16), dtype=torch.uint8, device=DEV)
    s = torch.empty((x.shape[0], 4), dtype=torch.uint8, device=DEV)
    td.moonep_quantize_rows_mx(x, q, s)
    wq, ws = mx_pack(*mx_quantise(x.float()))
    same_bits(s, ws, "scale")
    same_bits(q, wq, "q")
    assert bool((s[-3:, 0] == 255).all()) and bool((q[-3:] == 0).all())


def test_offsets_past_32_bits(td):
    """Rows whose elements and bytes lie past 2^32: the last ones are right."""
    rows, cols = 300000, 16384
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    last = _rand((4, cols), "bf16", 1)
    x[-4:] = last
    gamma = torch.ones(cols, dtype=x.dtype, device=DEV)
    x[:-4] = 1
    y, want = torch.empty_like(x), torch.empty_like(last)
    td.moonep_rmsnorm(x, gamma, y, EPS)
    td.moonep_rmsnorm(last, gamma, want, EPS)
    same_bits(y[-4:], want, "norm")
    td.moonep_swiglu(x, x, y)
    td.moonep_swiglu(last, last, want)
    same_bits(y[-4:], want, "swiglu")
    q, s = (torch.empty((rows, n), dtype=torch.uint8, device=DEV) for n in (cols // 2, scale_cols(cols)))
    td.moonep_quantize_rows_mx(x, q, s)
    wq, ws = mx_pack(*mx_quantise(last.float()))
    same_bits(q[-4:], wq, "q")
    same_bits(s[-4:], ws, "scale")


def test_on_a_side_stream_and_in_a_graph(td):
    """The calls on a stream of their own, then captured together and replayed on other values
    with eager work between the replays."""
    rows, cols = 40, 1024
    gamma = 1 + 0.2 * _rand((cols,), "bf16", 1)
    x, res, go = (_rand((rows, cols), "bf16", s) for s in (2, 3, 4))
    half = cols // 2
    work = td.new_norm_workspace(cols, DEV)

    def buffers():
        e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
        return dict(s=e(rows, cols), y=e(rows, cols), inv=e(rows, dt=torch.float32), a=e(rows, half),
                    gx=e(rows, cols), gg=e(cols, dt=torch.float32), dh=e(rows, cols),
                    q=e(rows, half // 2, dt=torch.uint8), qs=e(rows, scale_cols(half), dt=torch.uint8))

    def step(b, work, stream=None):
        td.moonep_rmsnorm(x, gamma, b["y"], EPS, residual=res, sum_out=b["s"], inv_rms=b["inv"], stream=stream)
        td.moonep_swiglu(b["y"][:, :half], b["y"][:, half:], b["a"], stream=stream)
        td.moonep_swiglu_mx(b["y"][:, :half], b["y"][:, half:], b["q"], b["qs"], stream=stream)
        td.moonep_rmsnorm_backward(go, b["s"], gamma, b["inv"], b["gx"], b["gg"], work, stream=stream)
        td.moonep_swiglu_backward(b["a"], b["y"][:, :half], b["y"][:, half:], b["dh"][:, :half],
                                  b["dh"][:, half:], stream=stream)

    want, got = buffers(), buffers()
    step(want, work)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(got, td.new_norm_workspace(cols, DEV), stream=side)
    side.synchronize()
    for k in want:
        same_bits(got[k], want[k], k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got, work)
    for seed in (11, 12, 13):
        x.copy_(_rand((rows, cols), "bf16", seed))
        go.copy_(_rand((rows, cols), "bf16", seed + 50))
        for t in got.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        step(want, td.new_norm_workspace(cols, DEV))
        torch.cuda.synchronize()
        for k in want:
            same_bits(got[k], want[k], f"{k}, replay {seed}")


# ------------------------------------------------------------------ every length of row

# in chunks of 16 bytes: each side of where lanes and registers of a row change
CHUNKS = [1, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_every_length(td, dtype):
    for i, n in enumerate(CHUNKS):
        cols = n * (8 if dtype == "bf16" else 4)
        for rows in (3, 70 if n <= 64 else 5):
            _check_norm(td, (rows, cols), dtype, i % 2 == 0, "same", 3 * i)
            if cols % 16 == 0:
                _check_norm(td, (rows, cols), dtype, i % 2 == 1, "int8", 3 * i)
            if cols % 32 == 0:
                _check_norm(td, (rows, cols), dtype, i % 2 == 0, "mx", 3 * i)
    _check_norm(td, (2049, 2040 if dtype == "bf16" else 1020), dtype, True, "same", 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_backward_of_every_length(td, dtype):
    for i, n in enumerate(CHUNKS):
        cols = n * (8 if dtype == "bf16" else 4)
        _check_backward(td, (5000 if n <= 33 else 11, cols), dtype, i % 2 == 0, 5 * i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activation_of_every_length(td, dtype):
    for i, n in enumerate(CHUNKS):
        cols, rows = n * (8 if dtype == "bf16" else 4), 70 if n <= 64 else 5
        g, u = _halves(rows, cols, dtype, 11 * i, "halves")
        say(f"activation {(rows, cols)} {dtype}")
        want, bound = plain_swiglu(g, u)
        y, v32 = torch.empty((rows, cols), dtype=g.dtype, device=DEV), torch.empty((rows, cols), device=DEV)
        td.moonep_swiglu(g, u, y)
        assert_within(y, want, bound + want.abs() * half_step(y.dtype) * 1.01 + _small(y.dtype), "out")
        td.moonep_swiglu(g.float().contiguous(), u.float().contiguous(), v32)
        if cols % 16 == 0:
            q, s = torch.empty_like(v32, dtype=torch.int8), torch.empty(rows, device=DEV)
            td.moonep_swiglu_quant(g, u, q, s)
            for got, expected in zip((q, s), quantise8(v32)):
                same_bits(got, expected, "8 bits")
        if cols % 32 == 0:
            q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
            s = torch.full((rows, scale_cols(cols)), 9, dtype=torch.uint8, device=DEV)
            td.moonep_swiglu_mx(g, u, q, s)
            for got, expected in zip((q, s), mx_pack(*mx_quantise(v32))):
                same_bits(got, expected, "4 bits")
            x = g.contiguous()
            td.moonep_quantize_rows_mx(x, q, s)
            for got, expected in zip((q, s), mx_pack(*mx_quantise(x.float()))):
                same_bits(got, expected, "rows in 4 bits")
        go, dg, du = _rand((rows, cols), dtype, 11 * i + 5), torch.empty_like(y), torch.empty_like(y)
        td.moonep_swiglu_backward(go, g, u, dg, du)
        wg, bg, wu, bu = plain_swiglu_backward(go, g, u)
        for got, want, bound, what in ((dg, wg, bg, "grad_gate"), (du, wu, bu, "grad_up")):
            assert_within(got, want, bound + want.abs() * half_step(got.dtype) * 1.01 + _small(got.dtype), what)
