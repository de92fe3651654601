"""Cases of the operators around the experts' products: norm, activation, 4-bit products and
the whole layer for a few tokens.

Each operator has its plain form (elementary torch operations) and the library's calls
(taken when `own` is set):

  norm, norm_bwd  root-mean-square norm of rows with the residual's addition, out as the rows
                  are or in 8 bits with a scale for each row; and its gradients
  act, act_bwd    the experts' gated activation silu(gate) * up, and its gradients
  mx4, ffn4       rows quantised to 4-bit floating point (e2m1) in blocks of 32 with a power of
                  two for each, times 4-bit weights, grouped by expert; the second is an
                  expert's whole network in 4 bits
  layer           the whole mixture-of-experts layer for a few tokens

Values that are rounded to 8 or 4 bits are defined in binary32 step by step, after a sum in
binary64 where there is one, so that both forms round the same numbers.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_ES = {"f32": 4, "bf16": 2}
_TINY = 2.0 ** -100  # the least magnitude that an 8-bit row's scale stands for
_EPS = 1e-6          # of the norm
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _rows(name, op, dtype, rows, cols, residual=False, out="same"):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "cols": cols,
            "residual": residual, "out": out}


def _grouped(name, op, R, E, K, S, B, n_in, n_out, skew):
    return {"name": name, "op": op, "dtype": "bf16", "R": R, "E": E, "K": K, "S": S, "B": B,
            "n_in": n_in, "n_out": n_out, "skew": skew}


def _layer(name, dtype, weights, T, E, K, H, F):
    return {"name": name, "op": "layer", "dtype": dtype, "weights": weights, "T": T, "E": E,
            "K": K, "H": H, "F": F}


def listed():
    return [
        # one token of a decode step before its layer: a launch is what it costs
        _rows("norm_token_bf16", "norm", "bf16", 1, 7168, True),
        # a prompt's rows, handed on in 8 bits
        _rows("norm_prompt_int8", "norm", "bf16", 8192, 7168, True, "int8"),
        # a training step's gradients of the norm: rows of 8 ranks
        _rows("norm_bwd_bf16", "norm_bwd", "bf16", 32768, 2048, True),
        # the activation between the products of the decode shape, 2 * 512 columns in
        _rows("act_decode_bf16", "act", "bf16", 64 * 128 * 16, 512),
        # its gradients in training with even routing
        _rows("act_bwd_bf16", "act_bwd", "bf16", 8 * 4096 * 8, 1024),
        # the decode shape's first product in 4 bits: a quarter of the weights' bytes
        _grouped("mx4_decode", "mx4", 64, 896, 16, 128, 4, 7168, 512, 0.75),
        # prompts in 4 bits: long segments
        _grouped("mx4_uniform", "mx4", 8, 64, 8, 4096, 8, 2048, 1024, 0.0),
        # an expert's whole network in 4 bits with skewed routing and ragged sizes
        _grouped("ffn4_skewed", "ffn4", 16, 256, 8, 1023, 16, 4096, 1024, 1.2),
        # serving one token: the weights of its 8 experts are all there is
        _layer("layer_one_token_bf16", "bf16", "same", 1, 64, 8, 2048, 1024),
        # two dozen tokens over 896 experts: most experts have one token
        _layer("layer_decode_bf16", "bf16", "same", 24, 896, 16, 7168, 512),
        # the same layer with weights in 4 bits, fewer tokens
        _layer("layer_decode_mx4", "bf16", "mx4", 8, 896, 16, 7168, 512),
        # odd sizes all round in binary32, more tokens than one tile takes
        _layer("layer_odd_f32", "f32", "same", 37, 21, 5, 1032, 264),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rows", "rows", "grouped", "layer"))
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    if kind == "rows":
        op = rng.choice(("norm", "norm", "norm_bwd", "act", "act_bwd"))
        out = rng.choice(("same", "int8")) if op == "norm" else "same"
        unit = 16 if out == "int8" else 8 if dtype == "bf16" else 4
        while True:
            rows, cols = _log_int(rng, 1, 200000), unit * _log_int(rng, 2, 16384 // unit)
            if rows * cols <= 8192 * 7168:
                break
        return {"op": op, "dtype": dtype, "rows": rows, "cols": cols,
                "residual": op.startswith("norm") and rng.random() < 0.7, "out": out}
    if kind == "grouped":
        while True:
            R, G = _log_int(rng, 1, 64), _log_int(rng, 1, 32)
            E = R * G
            if E > 896:
                continue
            K = _log_int(rng, 1, min(16, E))
            S = _log_int(rng, 1, 4096)
            op = rng.choice(("mx4", "ffn4"))
            B = rng.choice((0, 1, 4, G))
            n_in, n_out = 32 * _log_int(rng, 1, 224), 32 * _log_int(rng, 1, 64)
            rows, held = R * S * K, (E + R * B) * n_in * n_out * (3 if op == "ffn4" else 1)
            flops = 2 * rows * n_in * n_out * (3 if op == "ffn4" else 1)
            if rows <= 1 << 18 and held <= 4 * 10 ** 9 and flops <= 10 ** 12:
                break
        return {"op": op, "dtype": "bf16", "R": R, "E": E, "K": K, "S": S, "B": B, "n_in": n_in,
                "n_out": n_out, "skew": rng.choice((0.0, 0.75, 1.5))}
    weights = rng.choice(("same", "mx4"))
    unit = 32 if weights == "mx4" else 8 if dtype == "bf16" else 4
    while True:
        E = _log_int(rng, 1, 896)
        K, T = _log_int(rng, 1, min(16, E)), _log_int(rng, 1, 64)
        H, F = unit * _log_int(rng, 2, 7168 // unit), unit * _log_int(rng, 2, 4096 // unit)
        if 3 * min(E, T * K) * H * F <= 2 * 10 ** 9 and 3 * E * H * F <= 10 ** 10:
            break
    return {"op": "layer", "dtype": dtype, "weights": weights, "T": T, "E": E, "K": K, "H": H,
            "F": F}


# ------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _generator(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, std):
    return torch.randn(shape, generator=g, device=g.device, dtype=dtype).mul_(std)


def _scale_cols(cols):
    """Bytes of a row's scales: one for each block of 32, whole words."""
    return (cols // 32 + 3) // 4 * 4


def _mx4_weights(g, lead, n_out, n_in, std):
    """(q, scale) of normal weights [lead, n_out, n_in], quantised some matrices at a time."""
    q = torch.empty((lead, n_out, n_in // 2), dtype=torch.uint8, device=g.device)
    scale = torch.zeros((lead, n_out, _scale_cols(n_in)), dtype=torch.uint8, device=g.device)
    step = max(1, (1 << 27) // (n_out * n_in))
    for i in range(0, lead, step):
        n = min(step, lead - i)
        _, codes, e = _mx4(_randn(g, (n, n_out, n_in), torch.float32, std))
        q[i:i + n] = codes[..., 0::2] | codes[..., 1::2] << 4
        scale[i:i + n, :, :n_in // 32] = e
    return q, scale


def _table(case, seed):
    """Segment table int32 [R, G + dcap + 1] (row offsets: the rank's home experts, then its
    duplicates, -1 beyond), each rank's S*K rows cut at random, and the duplicates' experts."""
    R, E, SK, rng = case["R"], case["E"], case["S"] * case["K"], np.random.default_rng(seed)
    G = E // R
    dcap = max(1, min(SK, E - G))
    table = np.full((R, G + dcap + 1), -1, dtype=np.int32)
    experts = np.zeros((R, case["B"]), dtype=np.int64)
    for r in range(R):
        n = G + (min(case["B"], dcap) if R > 1 else 0)
        p = np.exp(case["skew"] * rng.normal(size=n))
        table[r, :n + 1] = np.concatenate([[0], np.cumsum(rng.multinomial(SK, p / p.sum()))])
        away = rng.integers(0, max(1, E - G), case["B"])
        experts[r] = np.where(away < r * G, away, np.minimum(away + G, E - 1))
    return table, experts


def _prepare_grouped(case, seed):
    dev, g, op = _device(), _generator(seed), case["op"]
    R, E, SK, n_in, n_out = case["R"], case["E"], case["S"] * case["K"], case["n_in"], case["n_out"]
    table, experts = _table(case, seed)
    at = torch.from_numpy(experts).to(dev)
    s = {k: case[k] for k in ("op", "R", "E", "K", "S", "B", "n_in", "n_out")}
    s["seg_ptr"] = torch.from_numpy(table).to(dev)
    empty = lambda n, dt: torch.empty((R, SK, n), dtype=dt, device=dev)  # noqa: E731
    s["x"] = _randn(g, (R, SK, n_in), torch.bfloat16, 1.0)
    s["q"], s["x_scale"] = empty(n_in // 2, torch.uint8), empty(_scale_cols(n_in), torch.uint8)
    first = n_out if op == "mx4" else 2 * n_out
    s["w"], s["w_scale"] = _mx4_weights(g, E, first, n_in, n_in ** -0.5)
    s["dup_w"], s["dup_w_scale"] = s["w"][at], s["w_scale"][at]
    # rows of no segment are nobody's: they keep these zeros
    s["y"] = torch.zeros((R, SK, first), dtype=torch.bfloat16, device=dev)
    if op == "ffn4":
        s["a"], s["a_scale"] = empty(n_out // 2, torch.uint8), empty(_scale_cols(n_out), torch.uint8)
        s["w2"], s["w2_scale"] = _mx4_weights(g, E, n_in, n_out, n_out ** -0.5)
        s["dup_w2"], s["dup_w2_scale"] = s["w2"][at], s["w2_scale"][at]
        s["out"] = torch.zeros((R, SK, n_in), dtype=torch.bfloat16, device=dev)
    return s


def _prepare_layer(case, seed):
    dev, g, dt = _device(), _generator(seed), _DT[case["dtype"]]
    T, E, K, H, F = (case[k] for k in ("T", "E", "K", "H", "F"))
    s = {k: case[k] for k in ("op", "dtype", "weights", "T", "E", "K", "H", "F")}
    scores = torch.randn((1, T, E), generator=g, device=dev) + 0.75 * torch.randn(E, generator=g, device=dev)
    top = torch.topk(scores, K, dim=2)
    s["ids"], s["topk_w"] = top.indices.to(torch.int32), torch.softmax(top.values, dim=2)
    s["x"] = _randn(g, (1, T, H), dt, 1.0)
    s["out"] = torch.empty((1, T, H), dtype=dt, device=dev)
    # a program keeps this as long as its weights: slots, the tokens' activations
    s["work"] = torch.empty(_work_bytes(case), dtype=torch.uint8, device=dev)
    for name, n_out, n_in in (("w_gate", F, H), ("w_up", F, H), ("w_down", H, F)):
        if case["weights"] == "mx4":
            s[name], s[name + "_scale"] = _mx4_weights(g, E, n_out, n_in, n_in ** -0.5)
        else:
            s[name] = _randn(g, (E, n_out, n_in), dt, n_in ** -0.5)
    return s


def _work_bytes(case):
    """Bytes that are enough for the layer's workspace."""
    return (1 << 17) + 8 * case["T"] * case["K"] * (case["F"] + 64)


def prepare(case, seed):
    if case["op"] in ("mx4", "ffn4"):
        return _prepare_grouped(case, seed)
    if case["op"] == "layer":
        return _prepare_layer(case, seed)
    dev, g, dt, op = _device(), _generator(seed), _DT[case["dtype"]], case["op"]
    rows, cols = case["rows"], case["cols"]
    s = {"op": op, "out_kind": case["out"]}
    new = lambda n, t=dt: torch.empty((rows, n), dtype=t, device=dev)  # noqa: E731
    if op.startswith("act"):
        s["h"] = _randn(g, (rows, 2 * cols), dt, 1.5)  # gate and up side by side, as one product leaves them
        s["gate"], s["up"] = s["h"][:, :cols], s["h"][:, cols:]
        if op == "act":
            s["out"] = new(cols)
        else:
            s["grad_out"], s["grad_h"] = _randn(g, (rows, cols), dt, 1.0), new(2 * cols)
        return s
    s["gamma"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device=dev)).to(dt)
    # rows of different sizes, as a residual stream has them
    size = torch.exp(torch.randn((rows, 1), generator=g, device=dev))
    s["x"] = (torch.randn((rows, cols), generator=g, device=dev) * size).to(dt)
    if op == "norm":
        s["residual"] = _randn(g, (rows, cols), dt, 1.0) if case["residual"] else None
        s["sum"] = new(cols) if case["residual"] else None
        if case["out"] == "int8":
            s["q"], s["scale"] = new(cols, torch.int8), torch.empty(rows, dtype=torch.float32, device=dev)
        else:
            s["out"], s["inv_rms"] = new(cols), torch.empty(rows, dtype=torch.float32, device=dev)
        return s
    x = s["x"].double()
    s["inv_rms"] = torch.rsqrt(x.square().mean(1) + _EPS).float()  # what the forward pass left
    s["grad_out"] = _randn(g, (rows, cols), dt, 1.0)
    s["grad_sum"] = _randn(g, (rows, cols), dt, 1.0) if case["residual"] else None
    s["grad_x"] = new(cols)
    s["grad_gamma"] = torch.empty(cols, dtype=torch.float32, device=dev)
    s["work"] = torch.empty(1024 * cols, dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _mx4(v):
    """(values, codes, exponents) of binary32 v [..., n] in blocks of 32: the block's scale is
    2^(e - 127), with e - 127 two less than the exponent of its largest magnitude, which
    counts as the next power of two from 1.75 of one on; the values are v / scale to the
    nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code)."""
    b = v.reshape(v.shape[:-1] + (-1, 32))
    bits = b.abs().amax(dim=-1).view(torch.int32)
    e = (((bits + 0x200000) >> 23) - 2).clamp_min(0)
    half = (e + 127 - 2 * 127).neg()  # 127 - (e - 127 + 127): the inverse's exponent, in two halves
    inv = torch.ldexp(torch.ones_like(b[..., 0]), half // 2), torch.ldexp(torch.ones_like(b[..., 0]), half - half // 2)
    a = b.abs() * inv[0][..., None] * inv[1][..., None]
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_max(6.0)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | torch.signbit(b).to(torch.uint8) << 3
    scale = torch.ldexp(torch.ones_like(b[..., 0]), e - 127)
    return (torch.copysign(a, b) * scale[..., None]).reshape(v.shape), code.reshape(v.shape), e.to(torch.uint8)


def _mx4_values(q, scale, n, dtype=torch.float32):
    """The values [..., n] that 4-bit codes and their blocks' scales stand for."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=dtype, device=q.device)
    codes = torch.stack([q & 15, q >> 4], dim=-1).reshape(q.shape[:-1] + (n // 32, 32))
    exponent = scale[..., :n // 32].to(torch.int32) - 127
    return torch.ldexp(table[codes.int()], exponent[..., None]).reshape(q.shape[:-1] + (n,))


def _segments(s):
    """(rank, first row, end, expert or None, slot or None) of each segment that has weights."""
    R, G, B = s["R"], s["E"] // s["R"], s["B"]
    for r, row in enumerate(s["seg_ptr"].tolist()):
        for j, (lo, hi) in enumerate(zip(row, row[1:])):
            if hi > lo >= 0 and j < G + B:
                yield (r, lo, hi, r * G + j, None) if j < G else (r, lo, hi, None, j - G)


def _plain_product(s, x, w, n_in, y):
    """y's rows: x (values, binary32) times the 4-bit matrix of each segment."""
    for r, lo, hi, e, b in _segments(s):
        q, scale = (s[w][e], s[w + "_scale"][e]) if b is None else (s["dup_" + w][r, b], s["dup_" + w + "_scale"][r, b])
        y[r, lo:hi] = (x[r, lo:hi] @ _mx4_values(q, scale, n_in).t()).to(y.dtype)


def _silu(g):
    return g / (1 + torch.exp(-g))


def _plain_grouped(s):
    _plain_product(s, _mx4(s["x"].float())[0], "w", s["n_in"], s["y"])
    if s["op"] == "mx4":
        return {"y": s["y"]}
    h = s["y"].float()
    a = _mx4(_silu(h[..., :s["n_out"]]) * h[..., s["n_out"]:])[0]
    _plain_product(s, a, "w2", s["n_out"], s["out"])
    return {"out": s["out"]}


def _plain_layer(s):
    H, F = s["H"], s["F"]

    def of(name, ids, n):
        if s["weights"] == "mx4":
            return _mx4_values(s[name][ids], s[name + "_scale"][ids], n)
        return s[name][ids].float()

    for t in range(s["T"]):  # a token at a time: its experts' matrices in binary32
        ids, x = s["ids"][0, t].long(), s["x"][0, t].float()
        h = _silu(of("w_gate", ids, H) @ x) * (of("w_up", ids, H) @ x)
        y = (of("w_down", ids, F) @ h[:, :, None])[:, :, 0]
        s["out"][0, t] = (s["topk_w"][0, t][:, None] * y).sum(0).to(s["out"].dtype)
    return {"out": s["out"]}


def _plain_norm(s):
    h = s["x"] if s["residual"] is None else torch.add(s["x"].float(), s["residual"].float()).to(s["x"].dtype)
    inv = (1 / torch.sqrt(h.double().square().mean(1) + _EPS)).float()
    v = h.float() * inv[:, None] * s["gamma"].float()
    got = {} if s["residual"] is None else {"sum": h}
    if s["out_kind"] == "int8":
        a = v.abs().amax(dim=1).clamp_min(_TINY)
        most = torch.full_like(a, 127.0)
        got["out"] = torch.round(v * (most / a)[:, None]) * (a / most)[:, None]
        return got
    return {**got, "out": v.to(h.dtype), "inv_rms": inv}


def _plain_norm_bwd(s):
    x, go, inv = s["x"].float(), s["grad_out"].float(), s["inv_rms"][:, None]
    t = go * s["gamma"].float()
    grad = inv * t - x * (inv * inv * inv * (t * x).mean(1, keepdim=True))
    if s["grad_sum"] is not None:
        grad = grad + s["grad_sum"].float()
    return {"grad_x": grad.to(s["x"].dtype), "grad_gamma": (go * (x * inv)).sum(0)}


def _plain_act(s):
    return {"out": (_silu(s["gate"].float()) * s["up"].float()).to(s["gate"].dtype)}


def _plain_act_bwd(s):
    g, u, go = s["gate"].float(), s["up"].float(), s["grad_out"].float()
    sig = 1 / (1 + torch.exp(-g))
    both = torch.cat([go * u * sig * (1 + g * (1 - sig)), go * g * sig], dim=1)
    return {"grad_h": both.to(s["gate"].dtype)}


# ------------------------------------------------------------------ one pass

def _own(s):
    import token_dispatch_amd as td
    op = s["op"]
    if op == "norm" and s["out_kind"] == "int8":
        td.moonep_rmsnorm_quant(s["x"], s["gamma"], s["q"], s["scale"], _EPS,
                                residual=s["residual"], sum_out=s["sum"])
        got = {} if s["residual"] is None else {"sum": s["sum"]}
        return {**got, "out": s["q"] * s["scale"][:, None]}
    if op == "norm":
        td.moonep_rmsnorm(s["x"], s["gamma"], s["out"], _EPS, residual=s["residual"],
                          sum_out=s["sum"], inv_rms=s["inv_rms"])
        got = {} if s["residual"] is None else {"sum": s["sum"]}
        return {**got, "out": s["out"], "inv_rms": s["inv_rms"]}
    if op == "norm_bwd":
        td.moonep_rmsnorm_backward(s["grad_out"], s["x"], s["gamma"], s["inv_rms"], s["grad_x"],
                                   s["grad_gamma"], s["work"], grad_sum=s["grad_sum"])
        return {"grad_x": s["grad_x"], "grad_gamma": s["grad_gamma"]}
    if op == "act":
        td.moonep_swiglu(s["gate"], s["up"], s["out"])
        return {"out": s["out"]}
    if op == "act_bwd":
        n = s["gate"].shape[1]
        td.moonep_swiglu_backward(s["grad_out"], s["gate"], s["up"], s["grad_h"][:, :n],
                                  s["grad_h"][:, n:])
        return {"grad_h": s["grad_h"]}
    if op == "layer":
        dt = td.BF16 if s["dtype"] == "bf16" else td.F32
        dims = td.Dims(1, s["E"], s["K"], s["T"], 0, dt, s["H"])
        if s["weights"] == "mx4":
            td.moonep_expert_layer_mx(dims, s["ids"], s["topk_w"], s["x"], s["w_gate"],
                                      s["w_gate_scale"], s["w_up"], s["w_up_scale"], s["w_down"],
                                      s["w_down_scale"], s["out"], s["work"])
        else:
            td.moonep_expert_layer(dims, s["ids"], s["topk_w"], s["x"], s["w_gate"], s["w_up"],
                                   s["w_down"], s["out"], s["work"])
        return {"out": s["out"]}
    dims = td.Dims(s["R"], s["E"], s["K"], s["S"], s["B"], td.BF16, s["n_in"])
    td.moonep_quantize_rows_mx(s["x"], s["q"], s["x_scale"])
    td.moonep_expert_matmul_mx(dims, s["seg_ptr"], s["q"], s["x_scale"], s["w"], s["w_scale"],
                               s["dup_w"], s["dup_w_scale"], s["y"])
    if op == "mx4":
        return {"y": s["y"]}
    n = s["n_out"]
    td.moonep_swiglu_mx(s["y"][..., :n], s["y"][..., n:], s["a"], s["a_scale"])
    td.moonep_expert_matmul_mx(dims, s["seg_ptr"], s["a"], s["a_scale"], s["w2"], s["w2_scale"],
                               s["dup_w2"], s["dup_w2_scale"], s["out"])
    return {"out": s["out"]}


def run(s):
    if own:
        return _own(s)
    plain = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "act": _plain_act,
             "act_bwd": _plain_act_bwd, "mx4": _plain_grouped, "ffn4": _plain_grouped,
             "layer": _plain_layer}
    return plain[s["op"]](s)


# ------------------------------------------------------------------ what it cannot do without

def _chosen(case):
    """Distinct experts that a few tokens' routing names, as a seed has it."""
    rng = np.random.default_rng(case["T"] * 1009 + case["E"])
    scores = rng.normal(size=(case["T"], case["E"])) + 0.75 * rng.normal(size=case["E"])
    return len(np.unique(np.argsort(-scores, axis=1)[:, :case["K"]]))


def work(case):
    op, es = case["op"], _ES[case["dtype"]]
    if op == "layer":
        T, K, H, F = case["T"], case["K"], case["H"], case["F"]
        matrix = 3 * H * F * es
        if case["weights"] == "mx4":
            matrix = 3 * H * F / 2 + 2 * F * (H // 32) + H * (F // 32)
        return {"bytes": _chosen(case) * matrix + 2 * T * H * es + 8 * T * K,
                "flops": 6.0 * T * K * H * F}
    if op in ("mx4", "ffn4"):
        n_in, n_out = case["n_in"], case["n_out"]
        table, _ = _table(case, 0)
        G = case["E"] // case["R"]
        full = (np.diff(table, axis=1) > 0)[:, :G + case["B"]]
        rows, segs = int(np.diff(table, axis=1)[:, :G + case["B"]][full].sum()), int(full.sum())
        each = n_in * n_out * 17 / 32  # bytes of a 4-bit matrix and its scales
        if op == "mx4":
            return {"bytes": 2.0 * rows * (n_in + n_out) + segs * each, "flops": 2.0 * rows * n_in * n_out}
        return {"bytes": 4.0 * rows * n_in + 3 * segs * each, "flops": 6.0 * rows * n_in * n_out}
    rows, n = case["rows"], case["rows"] * case["cols"]
    if op == "norm":
        moved = n * es * (3 if case["residual"] else 1) + case["cols"] * es
        return {"bytes": moved + (n if case["out"] == "int8" else n * es) + 4 * rows, "flops": 6.0 * n}
    if op == "norm_bwd":
        return {"bytes": n * es * (4 if case["residual"] else 3) + case["cols"] * (es + 4) + 4 * rows,
                "flops": 10.0 * n}
    return {"bytes": n * es * (3 if op == "act" else 5), "flops": (6.0 if op == "act" else 14.0) * n}


# ------------------------------------------------------------------ in 64 bits

def _exact_fp4(v):
    """Binary32 v in 4 bits as binary64 values: by the blocks' exponents and the nearest entry
    of the table, ties to the entry of even place."""
    b = v.double().unflatten(-1, (-1, 32))
    mantissa, exponent = torch.frexp(b.abs().amax(-1))  # mantissa in [0.5, 1)
    exponent = torch.where(mantissa >= 0.875, exponent + 1, exponent) - 3
    exponent = torch.where(mantissa == 0, torch.full_like(exponent, -127), exponent.clamp(-127))
    unit = torch.exp2(exponent.double())[..., None]
    levels = torch.tensor(_E2M1, dtype=torch.float64, device=v.device)
    borders = (levels[1:] + levels[:-1]) / 2
    y = b.abs() / unit
    place = torch.bucketize(y, borders)  # of a border itself: the lower place
    up = (y == borders[place.clamp(max=6)]) & (place % 2 == 1)
    return (torch.sign(b) * levels[(place + up).clamp(max=7)] * unit).flatten(-2)


def _exact_weights(q, scale, n_in):
    lo, hi = torch.bitwise_and(q, 15), torch.bitwise_right_shift(q, 4)
    codes = torch.empty(q.shape[:-1] + (n_in,), dtype=torch.int64, device=q.device)
    codes[..., 0::2], codes[..., 1::2] = lo.long(), hi.long()
    size = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)[codes % 8] * (1 - 2 * (codes // 8)).double()
    return size * torch.exp2(scale[..., :n_in // 32].double() - 127).repeat_interleave(32, dim=-1)


def _exact_grouped(case, s):
    R, G, B, n_in, n_out = case["R"], case["E"] // case["R"], case["B"], case["n_in"], case["n_out"]
    table = s["seg_ptr"].cpu().numpy()
    last = s["out"] if case["op"] == "ffn4" else s["y"]
    got = torch.zeros(last.shape, dtype=torch.float64, device=last.device)
    for r in range(R):
        for j in range(min(G + B, table.shape[1] - 1)):
            lo, hi = int(table[r, j]), int(table[r, j + 1])
            if lo < 0 or hi <= lo:
                continue
            pick = lambda name: (s[name][r * G + j], s[name + "_scale"][r * G + j]) if j < G else (  # noqa: E731
                s["dup_" + name][r, j - G], s["dup_" + name + "_scale"][r, j - G])
            y = _exact_fp4(s["x"][r, lo:hi]) @ _exact_weights(*pick("w"), n_in).T
            if case["op"] == "ffn4":  # the first product is held in bf16 between the two
                gate, up = y.to(torch.bfloat16).double().chunk(2, dim=-1)
                y = _exact_fp4((gate * torch.sigmoid(gate) * up).float()) @ _exact_weights(*pick("w2"), n_out).T
            got[r, lo:hi] = y
    return {"out": got} if case["op"] == "ffn4" else {"y": got}


def _exact_layer(case, s):
    H, F, ids, w = case["H"], case["F"], s["ids"][0].long(), s["topk_w"][0].double()
    x = s["x"][0].double()
    out = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        t, k = torch.nonzero(ids == e, as_tuple=True)
        m = {}
        for name, n in (("w_gate", H), ("w_up", H), ("w_down", F)):
            m[name] = _exact_weights(s[name][e], s[name + "_scale"][e], n) if case["weights"] == "mx4" else s[name][e].double()
        gate = x[t] @ m["w_gate"].T
        y = (gate * torch.sigmoid(gate) * (x[t] @ m["w_up"].T)) @ m["w_down"].T
        out.index_add_(0, t, y * w[t, k][:, None])
    return {"out": out[None]}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("mx4", "ffn4"):
        return _exact_grouped(case, s)
    if op == "layer":
        return _exact_layer(case, s)
    if op.startswith("act"):
        g, u = s["gate"].double(), s["up"].double()
        sig = torch.sigmoid(g)
        if op == "act":
            return {"out": g * sig * u}
        go = s["grad_out"].double()
        return {"grad_h": torch.cat([go * u * (sig + g * sig * (1 - sig)), go * g * sig], dim=1)}
    gamma = s["gamma"].double()
    if op == "norm_bwd":
        x, go, inv = s["x"].double(), s["grad_out"].double(), s["inv_rms"].double()[:, None]
        hat = x * inv
        grad = inv * (go * gamma - hat * (go * gamma * hat).sum(1, keepdim=True) / x.shape[1])
        if s["grad_sum"] is not None:
            grad = grad + s["grad_sum"].double()
        return {"grad_x": grad, "grad_gamma": (go * hat).sum(0)}
    h, got = s["x"], {}
    if s["residual"] is not None:
        h = (s["x"].double() + s["residual"].double()).to(h.dtype)  # as it is stored
        got["sum"] = h.double()
    inv = (torch.linalg.vector_norm(h.double(), dim=1).square() / case["cols"] + _EPS).rsqrt()
    if case["out"] == "int8":  # the 8-bit values are defined by their binary32 rounding
        v = torch.mul(torch.mul(h.float(), inv.float()[:, None]), s["gamma"].float())
        a = torch.maximum(v.abs().max(dim=1).values, torch.full((1,), _TINY, device=v.device))
        q = torch.round(v * torch.div(torch.full_like(a, 127.0), a)[:, None])
        return {**got, "out": q.double() * (a.double() / 127)[:, None]}
    return {**got, "out": h.double() * inv[:, None] * gamma, "inv_rms": inv}
