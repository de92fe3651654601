"""What the norm, the activation, the 4-bit rows and products and the layer for a few tokens
refuse, checked on the host (every error comes back before anything is enqueued), and the
4-bit rule of the tests' own oracle by hand."""
import ctypes
import os
import re

import pytest
import torch

from tests.layer_common import mx_pack, mx_quantise, mx_values

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def td():
    import token_dispatch_amd as td
    return td


OK = ctypes.c_void_p(1 << 20)         # aligned, never dereferenced: calls fail first
MIS = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned


def _norm(td, n=4, cols=64, dtype=1, eps=1e-6, x=OK, res=None, gamma=OK, s=None, out=OK, inv=None):
    return td._lib.moonep_rmsnorm(n, cols, x, dtype, res, gamma, eps, s, out, inv, None)


def _norm_q(td, n=4, cols=64, dtype=1, eps=1e-6, x=OK, res=None, gamma=OK, s=None, out=OK, inv=None,
            scale=OK, call="moonep_rmsnorm_quant"):
    return getattr(td._lib, call)(n, cols, x, dtype, res, gamma, eps, s, out, scale, inv, None)


def _norm_mx(td, **kw):
    return _norm_q(td, call="moonep_rmsnorm_mx", **kw)


def _act(td, n=4, cols=64, dtype=1, ld=None, gate=OK, up=OK, out=OK):
    return td._lib.moonep_swiglu(n, cols, gate, up, cols if ld is None else ld, dtype, out, None)


def _act_q(td, n=4, cols=64, dtype=1, ld=None, gate=OK, up=OK, out=OK, scale=OK,
           call="moonep_swiglu_quant"):
    return getattr(td._lib, call)(n, cols, gate, up, cols if ld is None else ld, dtype, out, scale, None)


def _act_mx(td, **kw):
    return _act_q(td, call="moonep_swiglu_mx", **kw)


def _quant_mx(td, n=4, cols=64, dtype=1, x=OK, q=OK, scale=OK):
    return td._lib.moonep_quantize_rows_mx(n, cols, x, dtype, q, scale, None)


def _norm_bwd(td, n=4, cols=64, dtype=1, go=OK, gs=None, x=OK, gamma=OK, inv=OK, gx=OK, gg=OK, work=OK):
    return td._lib.moonep_rmsnorm_backward(n, cols, go, dtype, gs, x, gamma, inv, gx, gg, work, None)


def _act_bwd(td, n=4, cols=64, dtype=1, ld=None, gld=None, go=OK, gate=OK, up=OK, dg=OK, du=OK):
    return td._lib.moonep_swiglu_backward(n, cols, go, gate, up, cols if ld is None else ld, dtype, dg,
                                          du, cols if gld is None else gld, None)


ROWS = [(_norm, 8, ("x", "gamma", "out"), ("res", "s", "inv")),
        (_norm_q, 16, ("x", "gamma", "out", "scale"), ("res", "s", "inv")),
        (_norm_mx, 32, ("x", "gamma", "out", "scale"), ("res", "s", "inv")),
        (_act, 8, ("gate", "up", "out"), ()),
        (_act_q, 16, ("gate", "up", "out", "scale"), ()),
        (_act_mx, 32, ("gate", "up", "out", "scale"), ()),
        (_quant_mx, 32, ("x", "q", "scale"), ()),
        (_norm_bwd, 8, ("go", "x", "gamma", "inv", "gx", "gg", "work"), ("gs",)),
        (_act_bwd, 8, ("go", "gate", "up", "dg", "du"), ())]


@pytest.mark.parametrize("call,unit,needs,may", ROWS, ids=lambda v: getattr(v, "__name__", None))
def test_rows_refusals(td, call, unit, needs, may):
    for dtype in (-1, 2):
        assert call(td, dtype=dtype) == td.ERR_DIMS
    for n, cols in ((-1, 64), (1 << 31, 64), (4, 0), (4, -64), (4, unit // 2), (4, 64 + unit // 2),
                    (4, (1 << 20) + 32), (4, 1 << 40)):
        assert call(td, n=n, cols=cols) == td.ERR_SIZE, (n, cols)
    for name in needs:
        for bad in (None, MIS):
            if (name, bad) == ("gg", None):  # the gradient of gamma may be skipped
                continue
            assert call(td, **{name: bad}) == td.ERR_PTR, (name, bad)
    for name in may:
        assert call(td, **{name: MIS}) == td.ERR_PTR, name
    if call is not _norm_bwd:
        assert call(td, n=0, **{name: None for name in needs}) == td.OK


def test_norm_refuses_other_eps(td):
    for call in (_norm, _norm_q, _norm_mx):
        for eps in (-1e-6, float("nan"), float("inf")):
            assert call(td, eps=eps) == td.ERR_SIZE


def test_activation_refuses_bad_distances(td):
    for call in (_act, _act_q, _act_mx, _act_bwd):
        for ld in (32, 68, -64, (1 << 40) + 8):
            assert call(td, ld=ld) == td.ERR_SIZE, ld
    assert _act_bwd(td, gld=32) == td.ERR_SIZE and _act_bwd(td, gld=68) == td.ERR_SIZE


def _dims(td, **kw):
    d = dict(R=4, E=16, K=2, S=4, B=4, dtype=1, H=128)
    d.update(kw)
    return td.Dims(d["R"], d["E"], d["K"], d["S"], d["B"], d["dtype"], d["H"])


def _matmul_mx(td, d, ptrs=(OK,) * 8, n_in=64, n_out=32, block=None, sblock=None):
    block = n_out * n_in // 2 if block is None else block
    sblock = n_out * td.mx_scale_cols(n_in) if sblock is None else sblock
    return td._lib.moonep_expert_matmul_mx(ctypes.byref(d) if d else None, *ptrs, n_in, n_out, block,
                                           sblock, None)


def test_product_refusals(td):
    for bad in (dict(R=0), dict(E=18), dict(K=65), dict(S=0), dict(B=-1), dict(dtype=2), dict(H=0)):
        assert _matmul_mx(td, _dims(td, **bad)) == td.ERR_DIMS, bad
    assert _matmul_mx(td, None) == td.ERR_PTR
    d = _dims(td)
    for i in range(8):
        for bad in (None, MIS):
            ptrs = [OK] * 8
            ptrs[i] = bad
            assert _matmul_mx(td, d, tuple(ptrs)) == td.ERR_PTR, (i, bad)
    for kw in (dict(n_in=0), dict(n_out=0), dict(n_in=48), dict(n_in=-32), dict(n_out=4),
               dict(n_in=(1 << 20) + 32), dict(n_out=(1 << 20) + 8), dict(block=1008), dict(block=1032),
               dict(sblock=124), dict(sblock=130), dict(block=1 << 41), dict(sblock=1 << 41)):
        assert _matmul_mx(td, d, **kw) == td.ERR_SIZE, kw
    assert _matmul_mx(td, _dims(td, dtype=0), n_out=6) == td.ERR_SIZE


def _few(td, d, ptrs=(OK,) * 8, inner=64, ib=None, ob=None):
    n = inner * (d.H if d else 128)
    return td._lib.moonep_expert_layer(ctypes.byref(d) if d else None, *ptrs, inner,
                                       n if ib is None else ib, n if ob is None else ob, None)


def _few_mx(td, d, ptrs=(OK,) * 11, inner=64, ib=None, isb=None, ob=None, osb=None):
    H = d.H if d else 128
    return td._lib.moonep_expert_layer_mx(
        ctypes.byref(d) if d else None, *ptrs, inner, inner * H // 2 if ib is None else ib,
        inner * td.mx_scale_cols(H) if isb is None else isb, inner * H // 2 if ob is None else ob,
        H * td.mx_scale_cols(inner) if osb is None else osb, None)


@pytest.mark.parametrize("call,n", [(_few, 8), (_few_mx, 11)])
def test_few_tokens_refusals(td, call, n):
    for bad in (dict(R=0), dict(E=18), dict(K=65), dict(S=0), dict(B=-1), dict(dtype=2), dict(H=0)):
        assert call(td, _dims(td, **bad)) == td.ERR_DIMS, bad
    assert call(td, None) == td.ERR_PTR
    d = _dims(td)
    for i in range(n):
        for bad in (None, MIS):
            ptrs = [OK] * n
            ptrs[i] = bad
            assert call(td, d, tuple(ptrs)) == td.ERR_PTR, (i, bad)
    assert call(td, _dims(td, S=17)) == td.ERR_SIZE               # 68 tokens
    assert call(td, _dims(td, H=(1 << 20) + 32)) == td.ERR_SIZE
    for kw in (dict(inner=0), dict(inner=-64), dict(inner=4), dict(inner=(1 << 20) + 32),
               dict(ib=16), dict(ob=16), dict(ib=64 * 128 + 4), dict(ob=64 * 128 + 4),
               dict(ib=1 << 41), dict(ob=1 << 41)):
        assert call(td, d, **kw) == td.ERR_SIZE, kw
    # the workspace would pass 2^31 bytes: 64 tokens of 64 experts, 2^20 columns
    assert call(td, _dims(td, R=1, E=64, K=64, S=64), inner=1 << 20) == td.ERR_SIZE
    if call is _few_mx:
        for kw in (dict(inner=48), dict(isb=16), dict(osb=16), dict(isb=64 * 4 + 2), dict(osb=128 * 4 + 2)):
            assert call(td, d, **kw) == td.ERR_SIZE, kw
        assert call(td, _dims(td, H=144)) == td.ERR_SIZE


def test_workspace_bytes(td):
    d = _dims(td)
    # slots, map, and three planes of 16-bit values for every (token, k)
    assert td.moonep_expert_layer_bytes(d, 64) == 4 * 1024 + 64 * 1024 + 16 * 2 * 64 * 6
    for bad in (dict(S=17), dict(H=0), dict(dtype=3)):
        with pytest.raises(td.MoonEPError):
            td.moonep_expert_layer_bytes(_dims(td, **bad), 64)
    with pytest.raises(td.MoonEPError):
        td.moonep_expert_layer_bytes(d, 0)
    assert td._lib.moonep_expert_layer_bytes(ctypes.byref(d), 64, None) == td.ERR_PTR


def test_the_constants_match_the_header(td):
    text = open(os.path.join(ROOT, "include", "moonep.h")).read()
    for name in ("NORM_GRAD_ROWS", "FEW_TOKENS"):
        assert getattr(td, name) == int(re.search(rf"#define MOONEP_{name} (\d+)", text).group(1))
    assert re.search(r"#define MOONEP_MX_SCALE_BYTES\(cols\) \(\(\(cols\) / 32 \+ 3\) / 4 \* 4\)", text)
    for cols, want in ((32, 4), (128, 4), (160, 8), (7168, 224)):
        assert td.mx_scale_cols(cols) == want


def test_binding_refuses_tensors(td):
    x, g = torch.zeros((2, 64)), torch.zeros(64)
    for call in (lambda: td.moonep_rmsnorm(x, g, torch.zeros((2, 64)), 1e-6),
                 lambda: td.moonep_quantize_rows_mx(x, x, x),
                 lambda: td.moonep_swiglu(x, x, x),
                 lambda: td.moonep_swiglu_backward(x, x, x, x, x),
                 lambda: td.moonep_rmsnorm_backward(x, x, g, g, x, None, None)):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(TypeError):
        td.moonep_rmsnorm([1.0], g, x, 1e-6)
    d = _dims(td)
    with pytest.raises((TypeError, ValueError)):
        td.moonep_expert_layer(d, None, None, None, torch.zeros((16, 64, 128)), None, None, None, None)
    with pytest.raises(TypeError):
        td.moonep_expert_layer(d, None, None, None, 3, None, None, None, None)
    with pytest.raises(ValueError):
        td.moonep_expert_layer(d, None, None, None, torch.zeros((16, 64)), None, None, None, None)


def test_the_oracles_rule_of_4_bits():
    """By hand: scales and codes of blocks whose largest magnitude decides them."""
    def one(values):
        v = torch.zeros(32)
        v[:len(values)] = torch.tensor(values)
        c, b = mx_quantise(v)
        return c[:len(values)].tolist(), int(b[0])

    assert one([6.0, -0.25, 0.75, 5.0, -0.0, 1.25]) == ([7, 8, 2, 6, 8, 2], 127)
    assert one([6.99, 2.5, 3.5, 1.75]) == ([7, 4, 6, 4], 127)      # ties: 2.5 to 2, 3.5 to 4
    assert one([7.0, 1.0, 0.5]) == ([6, 1, 0], 128)                # 3.5 to 4, .5, .25 to 0
    assert one([4.0]) == ([6], 127) and one([3.99]) == ([6], 127)  # over 0.5 it would be 7.98
    assert one([3.4999]) == ([7], 126)
    assert one([0.0]) == ([0], 0)
    assert one([2.0 ** -149]) == ([0], 0)
    assert one([2.0 ** -126]) == ([4], 0)                          # 2^-126 / 2^-127 = 2
    assert one([3.0e38])[1] == 253 and one([3.4e38])[1] == 253
    assert one([float("inf"), 1.0]) == ([0, 0], 255) and one([1.0, float("nan")]) == ([0, 0], 255)
    v = torch.randn(3, 160)
    c, b = mx_quantise(v)
    q, s = mx_pack(c, b)
    assert q.shape == (3, 80) and s.shape == (3, 8) and bool((s[:, 5:] == 0).all())
    back = mx_values(q, s, 160)
    size = torch.exp2(b.double() - 127).repeat_interleave(32, -1)
    assert bool(((back - v.double()).abs() <= size).all())          # half of the widest step
