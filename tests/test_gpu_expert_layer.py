"""The expert layer run from end to end, as a training step and as a serving step use it.

Each stage is held against its plain 64-bit form on the values that the stage before it
left, so every tolerance is that of one operator: n * 2^-23 * sum |products| for a
binary32 sum of n products and half a step of the output's type for its store.
"""
import math

import numpy as np
import pytest
import torch

from tests.expert_common import (ADD, assert_within, half_step, plain_matmul, plain_wgrad,
                                 torch_dtype)
from tests.gpu_common import run_plan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import token_dispatch_amd as td
    torch.cuda.set_device(DEV)
    return td


def _ids(R, E, K, S, seed, skew):
    rng = np.random.default_rng(seed)
    score = rng.normal(size=(R * S, E)) + skew * rng.normal(size=E)
    return np.argsort(-score, axis=1)[:, :K].reshape(R, S, K).astype(np.int32)


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch_dtype(dtype))


def _product(got, table, G, B, x, w, dup_w, transposed, what):
    want, mag, written = plain_matmul(table, G, B, x, w, dup_w, transposed)
    assert bool(written.all())
    bound = mag * (x.shape[-1] * ADD) + want.abs() * half_step(got.dtype) * 1.01
    assert_within(got, want, bound, what)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step(td, dtype):
    """plan, replicate, dispatch, gate/up products, activation, down product, combine; the
    same backwards; duplicates' gradients reduced home; the norm of all, clipped."""
    R, E, K, S, B, H, N = 4, 16, 2, 64, 4, 128, 64
    G, SK = E // R, S * K
    dims = td.Dims(R, E, K, S, B, td.BF16 if dtype == "bf16" else td.F32, H)
    dt, es = torch_dtype(dtype), 2 if dtype == "bf16" else 4
    plan, _ = run_plan(td, dims, _ids(R, E, K, S, 3, 1.0), DEV)
    v = td.plan_views(dims, plan)
    assert int(v["status"]) == 0 and int(v["n_dup"].max()) > 0
    seg, table = v["seg_ptr"], v["seg_ptr"].cpu().numpy()
    w = _rand((E, 3, H, N), dtype, 1, H ** -0.5)  # gate, up [H, N] and down [H, N] read the other way
    dup_w = torch.zeros((R, B, 3, H, N), dtype=dt, device=DEV)
    td.moonep_replicate(dims, plan, w, dup_w, 3 * H * N * es)
    hidden, topk_w = _rand((R, S, H), dtype, 2), _rand((R, S, K), "f32", 3).softmax(-1)
    rows = lambda n: torch.zeros((R, SK, n), dtype=dt, device=DEV)  # noqa: E731
    x, gate, up, y = rows(H), rows(N), rows(N), rows(H)
    td.moonep_dispatch(dims, plan, hidden, x)
    td.moonep_expert_matmul(dims, seg, x, w[:, 0], dup_w[:, :, 0], gate)
    td.moonep_expert_matmul(dims, seg, x, w[:, 1], dup_w[:, :, 1], up)
    gf, uf = gate.float().requires_grad_(), up.float().requires_grad_()
    act = torch.nn.functional.silu(gf) * uf
    h = act.detach().to(dt)
    td.moonep_expert_matmul(dims, seg, h, w[:, 2], dup_w[:, :, 2], y, transposed=True)
    out = torch.zeros((R, S, H), dtype=dt, device=DEV)
    td.moonep_combine(dims, plan, y, topk_w, out)
    for got, a, part, tr in ((gate, x, 0, False), (up, x, 1, False), (y, h, 2, True)):
        _product(got, table, G, B, a, w[:, part], dup_w[:, :, part], tr, f"part {part}")

    # backwards: the loss is <out, go>
    go = _rand((R, S, H), dtype, 4)
    gy, gh, gg, gu, gx, gx2 = rows(H), rows(N), rows(N), rows(N), rows(H), rows(H)
    td.moonep_combine_backward(dims, plan, go, topk_w, y, gy, None)
    home, dup = torch.zeros((E, 3, H, N), device=DEV), torch.zeros((R, B, 3, H, N), device=DEV)
    td.moonep_expert_matmul(dims, seg, gy, w[:, 2], dup_w[:, :, 2], gh)
    td.moonep_expert_matmul_wgrad(dims, seg, h, gy, home[:, 2], dup[:, :, 2], transposed=True)
    act.backward(gh.float())
    gg.copy_(gf.grad)
    gu.copy_(uf.grad)
    for part, g in ((0, gg), (1, gu)):
        td.moonep_expert_matmul_wgrad(dims, seg, x, g, home[:, part], dup[:, :, part])
    td.moonep_expert_matmul(dims, seg, gg, w[:, 0], dup_w[:, :, 0], gx, transposed=True)
    td.moonep_expert_matmul(dims, seg, gu, w[:, 1], dup_w[:, :, 1], gx2, transposed=True)
    _product(gh, table, G, B, gy, w[:, 2], dup_w[:, :, 2], False, "grad of h")
    _product(gx, table, G, B, gg, w[:, 0], dup_w[:, :, 0], True, "grad of x by gate")
    _product(gx2, table, G, B, gu, w[:, 1], dup_w[:, :, 1], True, "grad of x by up")
    reduced = home.clone()
    td.moonep_reduce_dup_grads(dims, plan, dup, reduced, 3 * H * N)

    # one gradient per expert whatever the ranks that held it: against all of its rows
    expert = torch.from_numpy(_ids(R, E, K, S, 3, 1.0).reshape(-1)).to(DEV).long()
    slot = v["dst"].long()
    for part, a, g in ((0, x, gg), (1, x, gu), (2, gy, h)):
        a, g = (t.reshape(R * SK, -1)[slot].double() for t in (a, g))
        for e in range(E):
            p, q = a[expert == e], g[expert == e]
            want, mag = p.t().contiguous() @ q, p.abs().t().contiguous() @ q.abs()
            # sums of its rows, the duplicates' additions (at most one per rank) and the stores
            bound = mag * ((p.shape[0] + 2 * R) * ADD)
            assert_within(reduced[e, part], want, bound, f"expert {e} part {part}")

    grads = [reduced[e] for e in range(E)]
    before, acc, norm = reduced.clone(), td.new_norm_buffer(DEV), torch.zeros(1, device=DEV)
    td.moonep_grad_sumsq(grads, acc)
    want = math.sqrt(before.double().square().sum().item())
    td.moonep_grad_clip(grads, acc, want / 3, norm)
    assert abs(norm.item() - want) <= want * 2.0 ** -23
    assert_within(reduced, before.double() / 3, before.double().abs() / 3 * 2.0 ** -22, "clipped")

    # the gradient against differences, through the whole layer in binary32: along a
    # direction of the down matrices the loss is linear
    if dtype == "f32":
        dw = _rand((E, H, N), "f32", 9)

        def loss(sign):
            w2 = w.clone()
            w2[:, 2] += sign * dw
            d2 = torch.zeros_like(dup_w)
            td.moonep_replicate(dims, plan, w2, d2, 3 * H * N * es)
            y2, o2 = rows(H), torch.zeros_like(out)
            td.moonep_expert_matmul(dims, seg, h, w2[:, 2], d2[:, :, 2], y2, transposed=True)
            td.moonep_combine(dims, plan, y2, topk_w, o2)
            _, mag, _ = plain_matmul(table, G, B, h, w2[:, 2], d2[:, :, 2], True)
            each = mag.reshape(R * SK, H)[slot].reshape(R * S, K, H)
            mag = (each * topk_w.reshape(R * S, K, 1).double()).sum(1)
            return (o2.double() * go.double()).sum().item(), (mag * go.reshape(R * S, H).double().abs()).sum().item()

        (a, ma), (b, mb) = loss(1.0), loss(-1.0)
        want = 2 * (before[:, 2].double() * dw.double()).sum().item()
        # N products, K weighted terms, and the gradient's own sums of up to R * SK rows
        assert abs((a - b) - want) <= (ma + mb) * (N + K + R * SK + 2 * R + 4) * ADD


@pytest.mark.parametrize("S", [1, 5, 64])
def test_serving_step_in_8_bits(td, S):
    """The bounded plan, rows and weights in 8 bits, from one token per rank on."""
    R, E, K, B, H, N = 4, 16, 2, 2, 128, 64
    G, SK = E // R, S * K
    dims = td.Dims(R, E, K, S, B, td.BF16, H)
    plan, _ = run_plan(td, dims, _ids(R, E, K, S, 5, 0.5), DEV, bounded=True)
    v = td.plan_views(dims, plan)
    seg, table = v["seg_ptr"], v["seg_ptr"].cpu().numpy()
    hidden, topk_w = _rand((R, S, H), "bf16", 2), _rand((R, S, K), "f32", 3).softmax(-1)
    x = torch.zeros((R, SK, H), dtype=torch.bfloat16, device=DEV)
    td.moonep_dispatch(dims, plan, hidden, x)
    out = torch.zeros((R, S, H), dtype=torch.bfloat16, device=DEV)
    for n_in, n_out, seed in ((H, 2 * N, 1), (N, H, 2)):
        w = _rand((E, n_out, n_in), "bf16", seed, n_in ** -0.5)
        wq, ws = torch.empty((E, n_out, n_in), dtype=torch.int8, device=DEV), torch.empty((E, n_out), device=DEV)
        td.moonep_quantize_rows(w, wq, ws)
        assert_within(wq.double() * ws.double()[..., None], w.double(),
                      (ws.double()[..., None] * (0.5 + 127 * 2.0 ** -22)).expand_as(w), "weights")
        dq, ds = torch.zeros((R, B, n_out, n_in), dtype=torch.int8, device=DEV), torch.zeros((R, B, n_out), device=DEV)
        td.moonep_replicate(dims, plan, wq, dq, n_out * n_in)
        td.moonep_replicate(dims, plan, ws, ds, 4 * n_out)
        q, xs = torch.empty((R, SK, n_in), dtype=torch.int8, device=DEV), torch.empty((R, SK), device=DEV)
        td.moonep_quantize_rows(x, q, xs)
        y = torch.zeros((R, SK, n_out), dtype=torch.bfloat16, device=DEV)
        td.moonep_expert_matmul_quant(dims, seg, q, xs, wq, ws, dq, ds, y)
        want, mag, written = plain_matmul(table, G, B, q.double() * xs.double()[..., None],
                                          wq.double() * ws.double()[..., None],
                                          dq.double() * ds.double()[..., None], True)
        # three binary32 roundings (the sum's conversion and the two factors), the store's, and
        # the plain form's own: its scaled factors and n_in additions, 2^-53 of the magnitude each
        # (the integer sum here is exact, and may be 0 where the 64-bit one is a last digit)
        bound = want.abs() * (4 * 2.0 ** -24 + half_step(y.dtype) * 1.01) + mag * ((n_in + 3) * 2.0 ** -53)
        assert_within(y[written], want[written], bound[written], "y")
        # as far from the unquantised product as half a step of each side's scale
        full, _, _ = plain_matmul(table, G, B, x, w, torch.zeros((R, B, n_out, n_in), device=DEV), True)
        for r in range(R):
            n = int(table[r, G])  # the home experts' rows
            a, fa = x[r, :n].double().abs(), xs[r, :n, None].double()
            for j in range(G):
                lo, hi = int(table[r, j]), int(table[r, j + 1])
                we, fw = w[r * G + j].double().abs(), ws[r * G + j].double()
                off = (0.51 * fa[lo:hi]) * we.sum(1) + a[lo:hi].sum(1, keepdim=True) * (0.51 * fw) \
                    + 0.2601 * n_in * fa[lo:hi] * fw
                off = off + full[r, lo:hi].abs() * 2.0 ** -7 + off * 2.0 ** -7
                assert_within(y[r, lo:hi], full[r, lo:hi], off, "against the product before it")
        if n_in == H:
            g, u = y[..., :N].float(), y[..., N:].float()
            x = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)
        else:
            td.moonep_combine(dims, plan, y, topk_w, out)
    assert bool(out.isfinite().all()) and bool((out != 0).any())
