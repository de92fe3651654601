"""Norm, dispatch, products, activation and combine run together, as a training step and as
serving steps use them. Each stage is held against its plain form on the values that the
stage before it left, with that operator's tolerance."""
import pytest
import torch

from tests.expert_common import (ADD, assert_within, half_step, plain_matmul, torch_dtype)
from tests.gpu_common import run_plan
from tests.layer_common import (U, mx_pack, mx_quantise, mx_values, plain_layer, plain_norm,
                                plain_swiglu, plain_swiglu_backward, scale_cols)
from tests.test_gpu_expert_layer import _ids, _product, _rand
from tests.test_gpu_rowops import _small, same_bits

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


def _mx_of(td, v):
    q = torch.empty(v.shape[:-1] + (v.shape[-1] // 2,), dtype=torch.uint8, device=DEV)
    s = torch.empty(v.shape[:-1] + (scale_cols(v.shape[-1]),), dtype=torch.uint8, device=DEV)
    td.moonep_quantize_rows_mx(v, q, s)
    return q, s


@pytest.mark.parametrize("S", [1, 5, 64])
def test_serving_step_in_4_bits(td, S):
    """Rows are normed straight to 4 bits and dispatched as such: codes and scales are two
    sets of rows that one plan moves."""
    R, E, K, B, H, N = 4, 16, 2, 2, 512, 96
    G, SK = E // R, S * K
    dims = td.Dims(R, E, K, S, B, td.BF16, H)
    plan, _ = run_plan(td, dims, _ids(R, E, K, S, 5, 0.5), DEV, bounded=True)
    v = td.plan_views(dims, plan)
    seg, table = v["seg_ptr"], v["seg_ptr"].cpu().numpy()
    hidden, res, topk_w = _rand((R, S, H), "bf16", 2), _rand((R, S, H), "bf16", 4), _rand((R, S, K), "f32", 3).softmax(-1)
    gamma = 1 + 0.2 * _rand((H,), "bf16", 5)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    q, qs, new = u8(R, S, H // 2), u8(R, S, scale_cols(H)), torch.empty_like(hidden)
    td.moonep_rmsnorm_mx(hidden, gamma, q, qs, EPS, residual=res, sum_out=new)
    h, v32, _, _ = plain_norm(hidden, gamma, EPS, res)
    same_bits(new, h, "sum")
    for got, want in zip((q, qs), mx_pack(*mx_quantise(v32))):
        same_bits(got, want, "rows in 4 bits")
    x, xs = u8(R, SK, H // 2), u8(R, SK, scale_cols(H))
    f32 = torch.float32
    for rows, to in ((q, x), (qs, xs)):  # rows of whole 16 bytes, whatever they hold
        of = td.Dims(R, E, K, S, B, td.F32, rows.shape[-1] // 4)
        td.moonep_dispatch(of, plan, rows.view(f32), to.view(f32))
    token = torch.arange(R * S, device=DEV).repeat_interleave(K)
    slot = v["dst"].long()
    same_bits(x.reshape(R * SK, -1)[slot], q.reshape(R * S, -1)[token], "dispatched codes")
    same_bits(xs.reshape(R * SK, -1)[slot], qs.reshape(R * S, -1)[token], "dispatched scales")
    for n_in, n_out, seed in ((H, 2 * N, 1), (N, H, 2)):
        w, ws = _mx_of(td, _rand((E, n_out, n_in), "bf16", seed, n_in ** -0.5))
        dw, dws = u8(R, B, n_out, n_in // 2), u8(R, B, n_out, scale_cols(n_in))
        td.moonep_replicate(dims, plan, w, dw, n_out * n_in // 2)
        td.moonep_replicate(dims, plan, ws, dws, n_out * scale_cols(n_in))
        y = torch.zeros((R, SK, n_out), dtype=torch.bfloat16, device=DEV)
        td.moonep_expert_matmul_mx(dims, seg, x, xs, w, ws, dw, dws, y)
        want, mag, written = plain_matmul(table, G, B, mx_values(x, xs, n_in), mx_values(w, ws, n_in),
                                          mx_values(dw, dws, n_in), True)
        bound = mag * (n_in * ADD) + want.abs() * half_step(y.dtype) * 1.01
        assert_within(y[written], want[written], bound[written], "y")
        if n_in == H:
            x, xs = u8(R, SK, N // 2), u8(R, SK, scale_cols(N))
            td.moonep_swiglu_mx(y[..., :N], y[..., N:], x, xs)
            a = torch.empty((R, SK, N), device=DEV)
            td.moonep_swiglu(y[..., :N].float().contiguous(), y[..., N:].float().contiguous(), a)
            for got, want in zip((x, xs), mx_pack(*mx_quantise(a))):
                same_bits(got, want, "activation in 4 bits")
    out = torch.zeros((R, S, H), dtype=torch.bfloat16, device=DEV)
    td.moonep_combine(dims, plan, y, topk_w, out)
    assert bool(out.isfinite().all()) and bool((out != 0).any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step(td, dtype):
    """norm with the residual, plan, dispatch, products, activation, combine, and all of it
    backwards to the residual stream and gamma."""
    R, E, K, S, B, H, N = 4, 16, 2, 24, 4, 128, 64
    G, SK = E // R, S * K
    dims = td.Dims(R, E, K, S, B, td.BF16 if dtype == "bf16" else td.F32, H)
    dt, es = torch_dtype(dtype), 2 if dtype == "bf16" else 4
    plan, _ = run_plan(td, dims, _ids(R, E, K, S, 3, 1.0), DEV)
    v = td.plan_views(dims, plan)
    seg, table = v["seg_ptr"], v["seg_ptr"].cpu().numpy()
    w1, w2 = _rand((E, 2 * N, H), dtype, 1, H ** -0.5), _rand((E, H, N), dtype, 2, N ** -0.5)
    d1, d2 = torch.zeros((R, B, 2 * N, H), dtype=dt, device=DEV), torch.zeros((R, B, H, N), dtype=dt, device=DEV)
    td.moonep_replicate(dims, plan, w1, d1, 2 * N * H * es)
    td.moonep_replicate(dims, plan, w2, d2, N * H * es)
    stream, update, gamma = _rand((R, S, H), dtype, 3), _rand((R, S, H), dtype, 4), 1 + 0.2 * _rand((H,), dtype, 5)
    topk_w = _rand((R, S, K), "f32", 6).softmax(-1)
    rows = lambda n: torch.zeros((R, SK, n), dtype=dt, device=DEV)  # noqa: E731
    normed, inv = torch.empty_like(stream), torch.empty((R, S), device=DEV)
    before = stream.clone()
    td.moonep_rmsnorm(update, gamma, normed, EPS, residual=stream, sum_out=stream, inv_rms=inv)
    h, _, want, winv = plain_norm(update, gamma, EPS, before)
    same_bits(stream, h, "residual stream")
    assert_within(normed, want, want.abs() * (3.1 * U + half_step(dt) * 1.01) + _small(dt), "normed")
    x, gu, a, y, out = rows(H), rows(2 * N), rows(N), rows(H), torch.empty_like(stream)
    td.moonep_dispatch(dims, plan, normed, x)
    td.moonep_expert_matmul(dims, seg, x, w1, d1, gu, transposed=True)
    td.moonep_swiglu(gu[..., :N], gu[..., N:], a)
    td.moonep_expert_matmul(dims, seg, a, w2, d2, y, transposed=True)
    td.moonep_combine(dims, plan, y, topk_w, out)
    want, bound = plain_swiglu(gu[..., :N], gu[..., N:])
    assert_within(a, want, bound + want.abs() * half_step(dt) * 1.01 + _small(dt), "activation")
    _product(y, table, G, B, a, w2, d2, True, "down product")

    go = _rand((R, S, H), dtype, 7)
    gy, ga, ggu, gx = rows(H), rows(N), rows(2 * N), rows(H)
    td.moonep_combine_backward(dims, plan, go, topk_w, y, gy, None)
    td.moonep_expert_matmul(dims, seg, gy, w2, d2, ga)
    td.moonep_swiglu_backward(ga, gu[..., :N], gu[..., N:], ggu[..., :N], ggu[..., N:])
    wg, bg, wu, bu = plain_swiglu_backward(ga, gu[..., :N], gu[..., N:])
    for got, want, bound in ((ggu[..., :N], wg, bg), (ggu[..., N:], wu, bu)):
        assert_within(got, want, bound + want.abs() * half_step(dt) * 1.01 + _small(dt), "activation's gradient")
    td.moonep_expert_matmul(dims, seg, ggu, w1, d1, gx)
    _product(gx, table, G, B, ggu, w1, d1, False, "grad of x")
    gn = torch.empty_like(stream)
    td.moonep_dispatch_backward(dims, plan, gx, gn)
    gs, gg = torch.empty_like(stream), torch.empty(H, device=DEV)
    td.moonep_rmsnorm_backward(gn, stream, gamma, inv, gs, gg, td.new_norm_workspace(H, DEV), grad_sum=go)
    # the formula's by autograd in 64 bits on the same gradient
    p, q = stream.double().requires_grad_(), gamma.double().requires_grad_()
    n = p * torch.rsqrt(p.square().mean(-1, keepdim=True) + EPS) * q
    n.backward(gn.double())
    want = p.grad + go.double()
    t, xh = gn.double() * gamma.double(), stream.double() * inv.double()[..., None]
    mean = (t * xh).mean(-1, keepdim=True)
    off = (t * xh).abs().sum(-1, keepdim=True) * (ADD + 5 * U / H)
    # inv itself is off by U, and so is what it scales, three times over
    bound = inv.double()[..., None] * (xh.abs() * off + (t.abs() + (xh * mean).abs()) * (9 * U)) \
        + go.double().abs() * U + want.abs() * half_step(dt) * 1.01
    assert_within(gs, want, bound, "gradient of the residual stream")
    terms = (gn.double() * xh).abs().sum((0, 1))
    assert_within(gg, q.grad, terms * (R * S * ADD + 5 * U), "gradient of gamma")


@pytest.mark.parametrize("S", [1, 16])
def test_few_tokens_agree_with_the_planned_layer(td, S):
    """The same tokens through plan, dispatch, products, activation and combine."""
    R, E, K, B, H, N = 4, 16, 2, 4, 128, 64
    SK = S * K
    dims = td.Dims(R, E, K, S, B, td.BF16, H)
    ids = _ids(R, E, K, S, 9, 0.5)
    plan, ids_d = run_plan(td, dims, ids, DEV)
    seg = td.plan_views(dims, plan)["seg_ptr"]
    w1, w2 = _rand((E, 2 * N, H), "bf16", 1, H ** -0.5), _rand((E, H, N), "bf16", 2, N ** -0.5)
    d1, d2 = (torch.zeros((R, B) + tuple(w.shape[1:]), dtype=w.dtype, device=DEV) for w in (w1, w2))
    td.moonep_replicate(dims, plan, w1, d1, 4 * N * H)
    td.moonep_replicate(dims, plan, w2, d2, 2 * N * H)
    x, topk_w = _rand((R, S, H), "bf16", 3), _rand((R, S, K), "f32", 4).softmax(-1)
    rows = lambda n: torch.zeros((R, SK, n), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    recv, gu, a, y, out = rows(H), rows(2 * N), rows(N), rows(H), torch.empty_like(x)
    td.moonep_dispatch(dims, plan, x, recv)
    td.moonep_expert_matmul(dims, seg, recv, w1, d1, gu, transposed=True)
    td.moonep_swiglu(gu[..., :N], gu[..., N:], a)
    td.moonep_expert_matmul(dims, seg, a, w2, d2, y, transposed=True)
    td.moonep_combine(dims, plan, y, topk_w, out)
    few = torch.empty_like(x)
    td.moonep_expert_layer(dims, ids_d, topk_w, x, w1[:, :N], w1[:, N:], w2, few,
                           td.new_layer_workspace(dims, N, DEV))
    gate, up, down = (t.double() for t in (w1[:, :N], w1[:, N:], w2))
    want, bound = plain_layer(ids_d.reshape(-1, K), topk_w.reshape(-1, K), x.reshape(-1, H), gate, up, down,
                              E, 2.0 ** -16)
    assert_within(few.reshape(-1, H), want, bound + want.abs() * half_step(few.dtype) * 1.01, "few")
    # the planned layer rounds gate, up, the activation and y to bf16 on the way
    step, xd, flat = half_step(few.dtype) * 1.1, x.reshape(-1, H).double(), ids_d.reshape(-1, K).long()
    for t in range(R * S):
        for k in range(K):
            e, wk = int(flat[t, k]), topk_w.reshape(-1, K)[t, k].double()
            g, u = gate[e] @ xd[t], up[e] @ xd[t]
            act = (g * torch.sigmoid(g) * u).abs()
            off = down[e].abs() @ (1.1 * (g * u).abs() + 2 * act) + (down[e] @ (g * torch.sigmoid(g) * u)).abs()
            bound[t] += wk * off * step
    assert_within(out.reshape(-1, H), want, bound * 1.1 + want.abs() * step, "planned")
