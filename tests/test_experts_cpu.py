"""What the experts' products and the gradients' clipping refuse, checked on the host:
every error comes back before anything is enqueued, so no GPU is needed."""
import ctypes

import numpy as np
import pytest

from tests.expert_common import make_table, segments


@pytest.fixture(scope="module")
def td():
    import token_dispatch_amd as td
    return td


OK = ctypes.c_void_p(1 << 20)         # aligned, never dereferenced: calls fail first
MIS = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned


def _dims(td, **kw):
    d = dict(R=4, E=16, K=2, S=64, B=4, dtype=1, H=128)
    d.update(kw)
    return td.Dims(d["R"], d["E"], d["K"], d["S"], d["B"], d["dtype"], d["H"])


def _matmul(td, d, ptrs=(OK,) * 5, n_in=64, n_out=32, block=None, transposed=0):
    block = n_in * n_out if block is None else block
    return td._lib.moonep_expert_matmul(ctypes.byref(d), *ptrs, n_in, n_out, block, transposed, None)


def _wgrad(td, d, ptrs=(OK,) * 5, n_in=64, n_out=32, block=None, transposed=0):
    block = n_in * n_out if block is None else block
    return td._lib.moonep_expert_matmul_wgrad(ctypes.byref(d), *ptrs, n_in, n_out, block, transposed, None)


def _quant(td, d, ptrs=(OK,) * 8, n_in=64, n_out=32, block=None, sblock=None):
    block = n_in * n_out if block is None else block
    return td._lib.moonep_expert_matmul_quant(ctypes.byref(d), *ptrs, n_in, n_out, block,
                                              n_out if sblock is None else sblock, None)


@pytest.mark.parametrize("call", [_matmul, _wgrad, _quant])
def test_products_refuse_bad_dims(td, call):
    for bad in (dict(R=0), dict(E=18), dict(K=65), dict(S=0), dict(B=-1), dict(dtype=2), dict(H=0)):
        assert call(td, _dims(td, **bad)) == td.ERR_DIMS, bad


def test_products_refuse_a_missing_dims(td):
    lib = td._lib
    assert lib.moonep_expert_matmul(None, *(OK,) * 5, 64, 32, 2048, 0, None) == td.ERR_PTR
    assert lib.moonep_expert_matmul_wgrad(None, *(OK,) * 5, 64, 32, 2048, 0, None) == td.ERR_PTR
    assert lib.moonep_expert_matmul_quant(None, *(OK,) * 8, 64, 32, 2048, 32, None) == td.ERR_PTR


@pytest.mark.parametrize("call,n", [(_matmul, 5), (_wgrad, 5), (_quant, 8)])
def test_products_refuse_bad_pointers(td, call, n):
    d = _dims(td)
    for i in range(n):
        for bad in (None, MIS):
            ptrs = [OK] * n
            ptrs[i] = bad
            assert call(td, d, tuple(ptrs)) == td.ERR_PTR, (i, bad)


@pytest.mark.parametrize("call", [_matmul, _wgrad, _quant])
def test_products_refuse_bad_columns_and_blocks(td, call):
    d = _dims(td)
    for kw in (dict(n_in=0), dict(n_out=0), dict(n_in=-16), dict(n_out=(1 << 20) + 16),
               dict(n_in=(1 << 20) + 16), dict(n_in=1 << 40), dict(n_out=4), dict(n_in=4),
               dict(block=64 * 32 - 16), dict(block=64 * 32 + 1), dict(block=-16),
               dict(block=1 << 41)):
        assert call(td, d, **kw) == td.ERR_SIZE, kw


def test_products_refuse_other_options(td):
    d = _dims(td)
    for transposed in (-1, 2):
        assert _matmul(td, d, transposed=transposed) == td.ERR_SIZE
        assert _wgrad(td, d, transposed=transposed) == td.ERR_SIZE
    assert _quant(td, d, n_in=24) == td.ERR_SIZE            # 8-bit rows of whole 16 bytes
    assert _quant(td, d, n_in=131072) == td.ERR_SIZE        # sums could pass int32
    assert _quant(td, d, sblock=16) == td.ERR_SIZE
    assert _quant(td, d, sblock=34) == td.ERR_SIZE
    assert _quant(td, d, sblock=(1 << 40) + 4) == td.ERR_SIZE
    f = _dims(td, dtype=0)
    assert _matmul(td, f, n_in=6) == td.ERR_SIZE
    assert _matmul(td, f, n_out=34) == td.ERR_SIZE


def test_quantize_refusals(td):
    q = td._lib.moonep_quantize_rows
    assert q(4, 64, OK, 2, OK, OK, None) == td.ERR_DIMS
    for n, cols in ((-1, 64), (1 << 31, 64), (4, 0), (4, 24), (4, (1 << 20) + 16), (4, -16)):
        assert q(n, cols, OK, 1, OK, OK, None) == td.ERR_SIZE, (n, cols)
    for i in range(3):
        for bad in (None, MIS):
            p = [OK] * 3
            p[i] = bad
            assert q(4, 64, p[0], 1, p[1], p[2], None) == td.ERR_PTR
    assert q(0, 64, None, 1, None, None, None) == td.OK


def _lists(ptrs, numel, dtypes):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*dtypes))


def test_clip_refusals(td):
    s, c = td._lib.moonep_grad_sumsq, td._lib.moonep_grad_clip
    p, n, t = _lists([1 << 20, 1 << 20], [8, 8], [0, 1])

    def both(count, p, n, t, rc, acc=OK):
        assert s(count, p, n, t, acc, None) == rc
        assert c(count, p, p, n, t, acc, 1.0, None, None) == rc

    both(-1, p, n, t, td.ERR_SIZE)
    both(2, None, n, t, td.ERR_PTR)
    both(2, p, None, t, td.ERR_PTR)
    both(2, p, n, None, td.ERR_PTR)
    both(2, p, n, t, td.ERR_PTR, None)
    both(2, p, n, t, td.ERR_PTR, MIS)
    both(2, *_lists([1 << 20, 1 << 20], [8, -1], [0, 1]), td.ERR_SIZE)
    both(2, *_lists([1 << 20, 1 << 20], [8, (1 << 40) + 1], [0, 1]), td.ERR_SIZE)
    both(2, *_lists([1 << 20, 1 << 20], [8, 8], [0, 2]), td.ERR_DIMS)
    both(2, *_lists([1 << 20, None], [8, 8], [0, 1]), td.ERR_PTR)
    both(2, *_lists([(1 << 20) + 2, 1 << 20], [8, 8], [0, 1]), td.ERR_PTR)  # not a float's address
    both(2, *_lists([1 << 20, (1 << 20) + 1], [8, 8], [0, 1]), td.ERR_PTR)
    bad = _lists([1 << 20, None], [8, 8], [0, 1])[0]
    assert c(2, p, bad, n, t, OK, 1.0, None, None) == td.ERR_PTR
    for max_norm in (-1.0, float("nan")):
        assert c(2, p, p, n, t, OK, max_norm, None, None) == td.ERR_SIZE
    assert c(2, p, p, n, t, OK, 1.0, ctypes.c_void_p((1 << 20) + 2), None) == td.ERR_PTR


def test_binding_refuses_tensors(td):
    import torch
    d = _dims(td)
    seg = torch.zeros((4, 17), dtype=torch.int32)
    x, y = torch.zeros((4, 128, 64)), torch.zeros((4, 128, 32))
    with pytest.raises((TypeError, ValueError)):
        td.moonep_expert_matmul(d, seg, x, torch.zeros((16, 64, 32)), None, y)
    with pytest.raises(TypeError):
        td.GradList([1, 2])
    with pytest.raises(ValueError):
        td.GradList([torch.zeros(3)])
    with pytest.raises(ValueError):
        td.GradList([], outs=[torch.zeros(3)])
    with pytest.raises(TypeError):
        td.moonep_quantize_rows(torch.zeros((2, 16), dtype=torch.float16), None, None)
    assert td.GradList([]).n == 0


def test_the_constants_match_the_header(td):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moonep.h")).read()
    assert td.NORM_DOUBLES == int(re.search(r"#define MOONEP_NORM_DOUBLES (\d+)", text).group(1))


def test_the_tests_own_tables():
    """The oracle's reading of a table, by hand."""
    t = make_table([[2, 0, 3], []], 2, 2, 3, 8)
    assert t.tolist() == [[0, 2, 2, 5, -1, -1], [0, -1, -1, -1, -1, -1]]
    got = [s for s in segments(t, 2, 1, 8) if s[2] >= 0 and s[3] > s[2]]
    assert got == [(0, 0, 0, 2), (0, 2, 2, 5)]
    got = [s for s in segments(np.array([[7, 9, 3, -1]], dtype=np.int32), 3, 0, 8)]
    assert got == [(0, 0, 7, 8), (0, 1, 9, 9), (0, 2, 3, 3)]


def test_the_epilogue_orders_its_lanes(tmp_path):
    """Lanes of a wave hand the tile's values to one another through shared memory: whatever
    order the compiler chooses, a fence stands between the writes and the reads of a pass,
    and between its reads and the next pass's writes. The loads into shared memory name the
    register that they change."""
    import re
    import subprocess

    from token_dispatch_amd import build
    src = tmp_path / "epilogue.hip"
    src.write_text("""
#include "tiles.h"
using namespace moonep;
template <typename P> __device__ void store(char *lds, char *out, int rows, int cols, int n) {
    typename P::X x;
    typename P::W w;
    x.init(out, 128, rows, 0);
    w.init(out, 128, cols, 0);
    typename P::Sums acc;
    P::run(x, w, n, rows, lds, acc);
    asm volatile("; the epilogue" ::: "memory");
    P::template put<false>(lds, acc, rows, cols, out, n, false, [](int, int, float *) {});
}
typedef tiles::Product<2, false, false, 256, 256, 2, 4, 1, 5, 128, true> Wide;
extern "C" __global__ __launch_bounds__(Wide::kThreads) void probe(char *out, int rows, int cols, int n) {
    __shared__ __align__(1024) char lds[Wide::kLds];
    store<Wide>(lds, out, rows, cols, n);
}
""")
    ir = subprocess.run([build.HIPCC] + build.FLAGS + ["--offload-device-only", "-S", "-emit-llvm", "-o", "-", str(src)],
                        check=True, capture_output=True, text=True).stdout
    body = ir[ir.index("; the epilogue"):]
    body = body[:body.index("\n}")]
    last, fenced, turns = None, True, 0
    for line in body.splitlines():
        if "fence" in line and 'syncscope("wavefront")' in line:
            fenced = True
        m = re.search(r"(store|= load) .*addrspace\(3\)", line)
        if m is None:
            continue
        kind = m.group(1)
        if last is not None and kind != last:
            assert fenced, line
            turns += 1
        last, fenced = kind, False
    assert turns >= 3, "two passes of writes and reads"
    loads = [line for line in ir.splitlines() if "buffer_load_dwordx4" in line]
    assert loads and all(re.search(r"[,\"]~?\{m0\}", line) for line in loads)


def test_every_kernel_has_a_launch(td):
    """The compiler drops a kernel's host handle where no launch of it can be reached, but
    builds the kernel itself all the same: each one in the library has its handle."""
    import re
    import subprocess
    with open(td.LIB_PATH, "rb") as f:
        kernels = {m.decode() for m in re.findall(rb"(_Z\w+)\.kd\0", f.read())}
    symbols = subprocess.run(["nm", td.LIB_PATH], check=True, capture_output=True, text=True).stdout
    assert len(kernels) > 50
    assert kernels <= {line.split()[-1] for line in symbols.splitlines() if line}
