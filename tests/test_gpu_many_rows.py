"""Rows by the million: calls that take more than one launch, and rows whose offsets pass 32 bits.
A call over all rows has to give what calls over parts of them give, bit for bit; those are
compared with the plain forms elsewhere.

A launch takes 2^22 workgroups at most and fewer than 2^32 threads, so the rows here are just past
what one launch takes: of 32 rows to a workgroup, of one, and of one that 1024 lanes share.
"""
import pytest
import torch

from tests.gpu_common import say
from tests.layer_common import scale_cols

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-6
F32, BF16 = torch.float32, torch.bfloat16
STEP = 1 << 20  # rows of a part: one launch at every length here


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    torch.cuda.empty_cache()  # what other tests have left
    return td


def _values(rows, cols, dtype, seed):
    x = torch.empty((rows, cols), dtype=dtype, device=DEV)
    return x.normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


def _outputs(out, rows, cols, dtype):
    u8 = lambda n: torch.full((rows, n), 7, dtype=torch.uint8, device=DEV)  # noqa: E731
    if out == "int8":
        return [torch.full((rows, cols), 7, dtype=torch.int8, device=DEV), torch.full((rows,), 7.0, device=DEV)]
    if out == "mx":
        return [u8(cols // 2), u8(scale_cols(cols))]
    return [torch.full((rows, cols), 7.0, dtype=dtype, device=DEV)]


def _same_as_parts(call, rows, inputs, outs, what):
    """call(inputs, outs) over all rows against the same over parts of them."""
    say(what)
    call(inputs, outs)
    for lo in range(0, rows, STEP):
        part = [t[lo:lo + STEP] for t in inputs]
        own = [torch.full_like(t[lo:lo + STEP], 3) for t in outs]
        call(part, own)
        for i, (a, b) in enumerate(zip(own, outs)):
            assert torch.equal(a, b[lo:lo + STEP]), f"{what}: output {i}, rows {lo} on"


PAST = 5  # rows past the last launch's
# (form of the result, columns, rows): columns in binary32, 4 to a chunk
NORM = [("same", 4, (1 << 27) + PAST), ("same", 1028, (1 << 22) + PAST), ("int8", 1040, (1 << 22) + PAST),
        ("mx", 1056, (1 << 22) + PAST), ("same", 4100, (1 << 20) + PAST), ("int8", 4112, (1 << 22) + PAST)]


@pytest.mark.parametrize("out,cols,rows", NORM)
def test_norm(td, out, cols, rows):
    name = {"same": "moonep_rmsnorm", "int8": "moonep_rmsnorm_quant", "mx": "moonep_rmsnorm_mx"}[out]
    gamma = 1 + 0.2 * _values(1, cols, F32, 2)[0]
    x, outs = _values(rows, cols, F32, 1), _outputs(out, rows, cols, F32)
    inv = torch.full((rows,), 7.0, device=DEV)
    _same_as_parts(lambda i, o: getattr(td, name)(i[0], gamma, *o[:-1], EPS, inv_rms=o[-1]), rows, [x], outs + [inv],
                   f"norm {out} {(rows, cols)}")


SWIGLU = [("same", 4, (1 << 27) + PAST), ("same", 1028, (1 << 22) + PAST), ("int8", 16, (1 << 27) + PAST),
          ("mx", 1056, (1 << 22) + PAST), ("int8", 4112, (1 << 22) + PAST)]


@pytest.mark.parametrize("out,cols,rows", SWIGLU)
def test_swiglu(td, out, cols, rows):
    name = {"same": "moonep_swiglu", "int8": "moonep_swiglu_quant", "mx": "moonep_swiglu_mx"}[out]
    x = _values(rows, cols, F32, 3)  # gate and up alike: half the memory
    _same_as_parts(lambda i, o: getattr(td, name)(i[0], i[0], *o), rows, [x], _outputs(out, rows, cols, F32),
                   f"swiglu {out} {(rows, cols)}")


@pytest.mark.parametrize("cols,rows", [(4, (1 << 27) + PAST), (132, (1 << 22) + PAST), (260, (1 << 22) + PAST)])
def test_swiglu_backward(td, cols, rows):
    go, gate, up = (_values(rows, cols, F32, s) for s in (4, 5, 6))
    _same_as_parts(lambda i, o: td.moonep_swiglu_backward(*i, *o), rows, [go, gate, up],
                   [torch.full_like(go, 7.0) for _ in range(2)], f"swiglu backward {(rows, cols)}")


@pytest.mark.parametrize("cols,rows", [(32, (1 << 27) + PAST), (1056, (1 << 22) + PAST)])
def test_quantize_mx(td, cols, rows):
    x = _values(rows, cols, F32, 7)
    _same_as_parts(lambda i, o: td.moonep_quantize_rows_mx(i[0], *o), rows, [x], _outputs("mx", rows, cols, F32),
                   f"quantize mx {(rows, cols)}")


def test_offsets_past_32_bits(td):
    """The gradients and the 8-bit results of rows past 2^32 elements."""
    rows, cols = 300000, 16384
    x, go = _values(rows, cols, BF16, 1), _values(rows, cols, BF16, 2)
    gamma = (1 + 0.2 * _values(1, cols, F32, 3)[0]).to(BF16)
    inv = torch.rand(rows, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV) + 0.5
    _same_as_parts(lambda i, o: td.moonep_rmsnorm_quant(i[0], gamma, *o, EPS), rows, [x],
                   _outputs("int8", rows, cols, BF16), "norm to 8 bits")
    _same_as_parts(lambda i, o: td.moonep_swiglu_quant(*i, *o), rows, [x, go], _outputs("int8", rows, cols, BF16),
                   "swiglu to 8 bits")
    _same_as_parts(lambda i, o: td.moonep_rmsnorm_backward(*i[:2], gamma, i[2], o[0], None, None), rows, [go, x, inv],
                   [torch.empty_like(x)], "norm backward")
    dg, du = torch.empty_like(x), torch.empty_like(x)
    td.moonep_swiglu_backward(go, x, go, dg, du)
    for lo in (0, rows // 2, rows - 40000):
        part = [torch.empty_like(x[lo:lo + 40000]) for _ in range(2)]
        td.moonep_swiglu_backward(go[lo:lo + 40000], x[lo:lo + 40000], go[lo:lo + 40000], *part)
        assert torch.equal(part[0], dg[lo:lo + 40000]) and torch.equal(part[1], du[lo:lo + 40000]), lo
