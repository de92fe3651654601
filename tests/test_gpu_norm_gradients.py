"""The norm's gradients over more rows than the kernels have workgroups for, so that every form
walks from row to row, against 64 bits.

grad_gamma, with U = 2^-24: a term g (x inv) is rounded twice, sums are binary64 but for the at most
512 partial sums, rounded once each, and the result: 3 U of the magnitudes and U of the sum, and
some slack for binary64. Not one row of distinct values can be lost or doubled within that.
"""
import pytest
import torch

from tests.expert_common import assert_within
from tests.gpu_common import say
from tests.layer_common import U
from tests.test_gpu_rowops import _check_backward, _rand

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


def _gamma_gradient(td, go, x, inv):
    cols = x.shape[1]
    gx, gg = torch.empty_like(x), torch.full((cols,), 5.0, device=DEV)
    work = td.new_norm_workspace(cols, DEV).fill_(float("nan"))
    td.moonep_rmsnorm_backward(go, x, torch.ones(cols, dtype=x.dtype, device=DEV), inv, gx, gg, work)
    return gg


# chunks of 16 bytes to a row, and rows past 512 workgroups: 32, 16, 4 and 1 rows to one
WALKS = [(1, 40000), (8, 40000), (16, 20000), (32, 20000), (64, 5000), (128, 5000), (256, 5000),
         (257, 1300), (512, 1300), (513, 1300), (1024, 1300), (1025, 1300), (2048, 1300), (2049, 1300), (4096, 1300),
         (4097, 1300)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_form_walks_its_rows(td, dtype):
    for i, (chunks, rows) in enumerate(WALKS):
        cols = chunks * (8 if dtype == "bf16" else 4)
        _check_backward(td, (rows, cols), dtype, i % 2 == 0, 40 * i)
        say(f"grad_gamma {(rows, cols)} {dtype}")
        x, go = _rand((rows, cols), dtype, 40 * i + 1), _rand((rows, cols), dtype, 40 * i + 2)
        inv = torch.rand(rows, generator=torch.Generator(DEV).manual_seed(i), device=DEV) + 0.5
        want = torch.zeros(cols, dtype=torch.float64, device=DEV)
        mag = torch.zeros_like(want)
        for lo in range(0, rows, 512):
            terms = go[lo:lo + 512].double() * x[lo:lo + 512].double() * inv[lo:lo + 512, None].double()
            want += terms.sum(0)
            mag += terms.abs().sum(0)
        assert_within(_gamma_gradient(td, go, x, inv), want, mag * (3.01 * U) + want.abs() * (1.01 * U), "grad_gamma")


@pytest.mark.parametrize("chunks", [8, 257, 4097])
def test_grad_gamma_of_many_rows(td, chunks):
    """Equal rows, whose roundings in a long binary32 sum would all be to one side: the error does
    not grow with the rows."""
    cols, rows = 4 * chunks, {8: 1 << 22, 257: 1 << 19, 4097: 1 << 15}[chunks]
    row = _rand((1, cols), "f32", 3).abs() + 0.5
    x, go = row.expand(rows, cols).contiguous(), torch.ones((rows, cols), device=DEV)
    want = row[0].double() * rows
    got = _gamma_gradient(td, go, x, torch.ones(rows, device=DEV))
    assert_within(got, want, want * (2.01 * U), "grad_gamma")
