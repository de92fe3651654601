"""The gradients' norm and clipping on the GPU against their plain forms in 64 bits.

Tolerances: the sum of n squares in binary64 is within n * 2^-53 of the exact one
(relative, all terms are positive; n counts the squares' own roundings twice). A clipped
value has three roundings: the factor's and the product's binary32 ones and the store's.
"""
import math

import pytest
import torch

from tests.expert_common import half_step, torch_dtype
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


def _tensors(sizes, dtypes, seed, scale=0.1, offset=0):
    """Tensors that begin `offset` elements into their storage, so at any alignment."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = torch_dtype(dtypes[i % len(dtypes)])
        at = offset * (1 + i % 5)
        out.append((torch.randn(n + at, generator=g, device=DEV) * scale).to(dt)[at:])
    return out


def _sum64(ts):
    return math.fsum(t.double().square().sum().item() for t in ts)


def _check(td, grads, max_norm, outs=None):
    before = [t.clone() for t in grads]
    acc = torch.full((td.NORM_DOUBLES,), float("nan"), dtype=torch.float64, device=DEV)
    norm = torch.full((1,), -1.0, device=DEV)
    gl = td.GradList(grads, outs)
    td.moonep_grad_sumsq(gl, acc)
    td.moonep_grad_clip(gl, acc, max_norm, norm)
    torch.cuda.synchronize()
    n, want = sum(t.numel() for t in grads), _sum64(before)
    assert abs(acc[0].item() - want) <= want * (2 * n + 4) * 2.0 ** -53
    assert abs(norm.item() - math.sqrt(want)) <= math.sqrt(want) * 2.0 ** -23
    c = max_norm / math.sqrt(want) if math.sqrt(want) > max_norm else 1.0
    for b, o, g in zip(before, gl.outs, grads):
        ref = b.double() * c
        # below the smallest normal number a step no longer shrinks with the value
        tiny = torch.finfo(b.dtype).smallest_normal * torch.finfo(b.dtype).eps
        tol = ref.abs() * (2 * 2.0 ** -24 + half_step(b.dtype)) * 1.01 + tiny
        if c == 1.0:
            assert torch.equal(o, b)
        else:
            assert bool(((o.double() - ref).abs() <= tol).all())
        if outs is not None:
            assert torch.equal(g, b)


@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f32", "bf16")], ids=["f32", "bf16", "both"])
@pytest.mark.parametrize("sizes", [[1], [5], [16384], [16385, 3], [1, 0, 7, 0], [100000, 1, 65537],
                                   [17] * 129, [33, 4097] * 200, [3_000_001]],
                         ids=["1", "5", "chunk", "two", "empty", "odd", "129", "400", "large"])
def test_clip(td, sizes, dtypes):
    for offset in (0, 1, 3):
        for rel in (0.3, 3.0):
            grads = _tensors(sizes, dtypes, 7, offset=offset)
            max_norm = rel * math.sqrt(_sum64(grads)) + 1e-30
            say(f"clip {len(sizes)} tensors {dtypes} offset {offset} rel {rel}")
            _check(td, grads, max_norm)
            grads = _tensors(sizes, dtypes, 8, offset=offset)
            _check(td, grads, max_norm, _tensors(sizes, dtypes, 9, offset=1 - offset % 2))


def test_equal_bits_and_order(td):
    grads = _tensors([4099, 70001, 12] * 60, ("f32", "bf16"), 3)
    acc = [td.new_norm_buffer(DEV) for _ in range(3)]
    for a in acc:
        td.moonep_grad_sumsq(grads, a)
    assert acc[0][0].item() == acc[1][0].item() == acc[2][0].item()


def test_no_tensors(td):
    acc, norm = td.new_norm_buffer(DEV), torch.full((1,), 5.0, device=DEV)
    for grads in ([], [torch.empty(0, device=DEV)]):
        td.moonep_grad_sumsq(grads, acc)
        norm.fill_(5.0)
        td.moonep_grad_clip(grads, acc, 1.0, norm)
        assert acc[0].item() == 0.0 and norm.item() == 0.0


def test_large_and_small_values(td):
    """Squares that leave binary32's range on either side."""
    for v in (1e30, 1e-30):
        grads = [torch.full((1000,), v, device=DEV), torch.full((24,), -v, device=DEV, dtype=torch.bfloat16)]
        want = math.sqrt(_sum64(grads))
        acc, norm = td.new_norm_buffer(DEV), torch.zeros(1, device=DEV)
        td.moonep_grad_sumsq(grads, acc)
        td.moonep_grad_clip(grads, acc, 1.0, norm)
        assert abs(norm.item() - want) <= want * 2.0 ** -23
        assert abs(math.sqrt(_sum64(grads)) - min(want, 1.0)) <= min(want, 1.0) * 2.0 ** -8


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(td, bad):
    grads = _tensors([1000, 20000], ("f32", "bf16"), 5)
    grads[1][777] = bad
    before = [t.clone() for t in grads]
    outs = [torch.zeros_like(t) for t in grads]
    acc, norm = td.new_norm_buffer(DEV), torch.zeros(1, device=DEV)
    for gl in (td.GradList(grads), td.GradList(grads, outs)):
        td.moonep_grad_sumsq(gl, acc)
        td.moonep_grad_clip(gl, acc, 0.5, norm)
        assert not math.isfinite(norm.item())
        for b, o in zip(before, gl.outs):
            assert torch.equal(b.nan_to_num(nan=9.0), o.nan_to_num(nan=9.0))


def test_zero_and_infinite_max_norm(td):
    grads = _tensors([1000, 3], ("f32", "bf16"), 5)
    before = [t.clone() for t in grads]
    acc = td.new_norm_buffer(DEV)
    td.moonep_grad_sumsq(grads, acc)
    td.moonep_grad_clip(grads, acc, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    td.moonep_grad_clip(grads, acc, 0.0)
    assert all(bool((a == 0).all()) for a in grads)


def test_ranks_add_their_sums(td):
    """Two ranks' gradients: the sums added before clipping give the norm of all."""
    a, b = _tensors([5000, 31], ("f32",), 1), _tensors([777], ("f32",), 2)
    want = math.sqrt(_sum64(a + b))
    accs = [td.new_norm_buffer(DEV) for _ in range(2)]
    for ts, acc in zip((a, b), accs):
        td.moonep_grad_sumsq(ts, acc)
    accs[0][:1] += accs[1][:1]
    accs[1][:1] = accs[0][:1]
    for ts, acc in zip((a, b), accs):
        td.moonep_grad_clip(ts, acc, 0.25 * want)
    assert abs(math.sqrt(_sum64(a + b)) - 0.25 * want) <= 0.25 * want * 2.0 ** -22


def test_captured_and_replayed(td):
    grads = _tensors([5000, 70001, 9], ("f32", "bf16"), 1)
    outs = [torch.zeros_like(t) for t in grads]
    gl = td.GradList(grads, outs)
    acc, norm = td.new_norm_buffer(DEV), torch.zeros(1, device=DEV)

    def step():
        td.moonep_grad_sumsq(gl, acc)
        td.moonep_grad_clip(gl, acc, 1.0, norm)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for t, n in zip(grads, _tensors([t.numel() for t in grads], ("f32", "bf16"), 20 + i)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        got, got_norm = [o.clone() for o in outs], norm.item()
        step()
        torch.cuda.synchronize()
        assert got_norm == norm.item() and all(torch.equal(p, q) for p, q in zip(got, outs)), f"replay {i}"
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert got_norm == norm.item()


# value, elements, max_norm: norms past binary32's range, factors below its normal numbers,
# clipped values that are subnormal or round to zero, and a factor just above the border
RANGES = [(3e38, 1_000_000, 1.0), (3e38, 1_000_000, 1e-30), (3e38, 300_001, 1e30), (1e30, 4097, 1e-20),
          (1e38, 33, 1e-8), (1e20, 1000, 1e-24), (1.0, 1000, 2.0 ** -120), (1e10, 77, 1e-33),
          (3e38, 20_000, 1e-40), (1e-5, 50, 1e-300)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value,n,max_norm", RANGES)
def test_norms_and_factors_outside_binary32(td, value, n, max_norm, dtype):
    """The factor keeps its digits wherever it lies: two binary32 roundings (factor and
    product), a third where the value lands below the normal numbers, and the store's. The
    reported norm is the nearest binary32 number, the largest finite one for a finite norm
    beyond, so that only a norm that leaves the gradients alone is reported as infinite."""
    dt = torch_dtype(dtype)
    grads = [torch.full((n,), value, device=DEV, dtype=dt), torch.full((7,), -value / 3, device=DEV, dtype=dt)]
    before = [t.clone() for t in grads]
    want = math.sqrt(_sum64(before))
    acc, norm = td.new_norm_buffer(DEV), torch.zeros(1, device=DEV)
    td.moonep_grad_sumsq(grads, acc)
    td.moonep_grad_clip(grads, acc, max_norm, norm)
    most = torch.finfo(torch.float32).max
    assert abs(norm.item() - min(want, most)) <= min(want, most) * 2.0 ** -23 and math.isfinite(norm.item())
    for b, g in zip(before, grads):
        ref = b.double() * (max_norm / want)
        # below the normal numbers a step is 2^-149 (bf16: 2^-133): half of one for the
        # product, which is binary32 in both types, and half of one for the store
        step = 2.0 ** -149 + (2.0 ** -133 if dtype == "bf16" else 0.0)
        tol = ref.abs() * (2 * 2.0 ** -24 + half_step(dt)) * 1.01 + step
        assert bool(((g.double() - ref).abs() <= tol).all()), (g[0].item(), ref[0].item())


def test_large_sets_past_the_caches(td):
    """256 MB and more, whose outputs are stored past the caches, at every alignment."""
    sizes = [30_000_003, 5, 40_000_001, 16_385]
    for dtypes, offset in ((("f32",), 0), (("f32", "bf16"), 1)):
        grads = _tensors(sizes, dtypes, 11, offset=offset)
        if len(dtypes) > 1:
            grads += _tensors([50_000_001], ("f32",), 12, offset=3)
        assert sum(t.numel() * t.element_size() for t in grads) >= 1 << 28
        max_norm = 0.3 * math.sqrt(_sum64(grads))
        outs = [torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:] for t in grads]
        _check(td, grads, max_norm, outs)
        _check(td, grads, max_norm)


def test_a_kept_list_follows_its_tensors(td):
    """A GradList works on what its tensors hold at the call: a tensor that was given other
    storage since is read and written there, and one that no longer fits is refused."""
    for other in (False, True):
        grads = _tensors([5000, 33, 70001], ("f32", "bf16"), 1)
        outs = [torch.zeros_like(t) for t in grads] if other else None
        kept = td.GradList(grads, outs)
        acc, norm = td.new_norm_buffer(DEV), torch.zeros(1, device=DEV)
        first = [t.detach() for t in grads]  # keeps the first storages, which stay as they are
        held = [t.clone() for t in first]
        for t, n in zip(grads, _tensors([5000, 33, 70001], ("f32", "bf16"), 2)):
            t.data = n.clone()
        if other:
            outs[1].data = torch.full_like(outs[1], 4.0)
        fresh = [t.clone() for t in grads]
        want = [torch.zeros_like(t) for t in grads]
        plain = td.GradList(fresh, want)
        td.moonep_grad_sumsq(plain, acc)
        td.moonep_grad_clip(plain, acc, 1.0, norm)
        acc2, norm2 = td.new_norm_buffer(DEV), torch.zeros(1, device=DEV)
        td.moonep_grad_sumsq(kept, acc2)
        td.moonep_grad_clip(kept, acc2, 1.0, norm2)
        assert norm.item() == norm2.item() > 1.0
        assert all(torch.equal(a, b) for a, b in zip(want, outs if other else grads))
        assert all(torch.equal(a, b) for a, b in zip(first, held)), "a storage given up was written"


def test_a_kept_list_refuses_what_no_longer_fits(td):
    """Storage on the host, freed storage, other dtypes and outs of another size are refused
    before anything is enqueued; a size that changed on both sides is followed."""
    def lists(seed, outs):
        grads = _tensors([5000, 300], ("f32",), seed)
        return td.GradList(grads, [torch.zeros_like(t) for t in grads] if outs else None)

    acc = torch.zeros(td.NORM_DOUBLES, dtype=torch.float64, device=DEV)

    def host(t):
        t.data = t.data.cpu()

    def freed(t):
        t.untyped_storage().resize_(0)

    def half(t):
        t.data = t.data.half()

    def strided(t):
        t.data = torch.zeros((t.numel(), 2), device=DEV)[:, 0]

    errors = (TypeError, ValueError, td.MoonEPError)
    for change in (host, freed, half, strided):
        for outs in (False, True):
            gl = lists(1, outs)
            change(gl.grads[1])
            with pytest.raises(errors):
                td.moonep_grad_sumsq(gl, acc)
            gl = lists(1, outs)
            change(gl.outs[1])
            with pytest.raises(errors):
                td.moonep_grad_clip(gl, acc, 1.0)
    gl = lists(2, True)
    gl.outs[0].data = torch.zeros(4999, device=DEV)
    with pytest.raises(ValueError):
        td.moonep_grad_clip(gl, acc, 1.0)
    gl = lists(2, True)
    gl.outs[0].data = gl.outs[1].data  # two gradients' values in one place, and one too small
    with pytest.raises(ValueError):
        td.moonep_grad_clip(gl, acc, 1.0)
    torch.cuda.synchronize()
    assert bool((acc == 0).all())
    gl = lists(3, False)
    gl.grads[0].data = gl.grads[0].data[:100].clone()
    gl.grads[1].resize_(40000).fill_(0.25)
    want = _sum64(gl.grads)
    td.moonep_grad_sumsq(gl, acc)
    assert abs(acc[0].item() - want) <= want * (2 * 40100 + 4) * 2.0 ** -53
    td.moonep_grad_clip(gl, acc, 0.5 * math.sqrt(want))
    assert abs(_sum64(gl.grads) - 0.25 * want) <= 0.25 * want * 2.0 ** -21
