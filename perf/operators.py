"""Cases of the experts' products, their 8-bit form and gradient clipping.

Three operators, each with its plain form (elementary torch operations) and the library's
calls (taken when `own` is set):

  matmul, wgrad   the products grouped by expert of the rows that dispatch wrote, and the
                  gradient of their weights
  int8            rows quantised to 8 bits with a scale each, times 8-bit weights with a
                  scale for each output channel
  clip            the norm of many gradient tensors together, and their clipping

A case of the first two holds the shape of an expert-parallel layer: R ranks, E experts, K
experts per token, S tokens per rank, B duplicate slots per rank. Its segment table is a
plan's: every rank has exactly S*K rows, cut into its home experts' and its duplicates'.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_ES = {"f32": 4, "bf16": 2}
_TINY = 2.0 ** -100  # the least magnitude that a row's scale stands for


# ------------------------------------------------------------------ cases

def _layer(name, op, dtype, R, E, K, S, B, n_in, n_out, transposed, skew):
    return {"name": name, "op": op, "dtype": dtype, "R": R, "E": E, "K": K, "S": S, "B": B,
            "n_in": n_in, "n_out": n_out, "transposed": transposed, "skew": skew}


def listed():
    return [
        # the smallest layer there is, in binary32: a launch is what it costs
        _layer("tiny_f32", "matmul", "f32", 4, 16, 2, 64, 4, 128, 256, False, 1.0),
        # serving one token per rank: a row or two for each expert, so all of it is weights
        _layer("one_token_bf16", "matmul", "bf16", 8, 64, 8, 1, 8, 2048, 1024, True, 0.0),
        # the decode shape's first product: about a hundred rows for each of 896 experts
        _layer("decode_bf16", "matmul", "bf16", 64, 896, 16, 128, 4, 7168, 512, False, 0.75),
        # training with even routing: long segments, bound by the matrix units
        _layer("uniform_bf16", "matmul", "bf16", 8, 64, 8, 4096, 8, 2048, 1024, False, 0.0),
        # training with skewed routing, the product back to the hidden size: a million rows
        _layer("zipf_down_bf16", "matmul", "bf16", 16, 256, 8, 8192, 16, 1024, 4096, True, 1.2),
        # the weights' gradient of the evenly routed layer
        _layer("wgrad_uniform_bf16", "wgrad", "bf16", 8, 64, 8, 4096, 8, 2048, 1024, False, 0.0),
        # and of four ranks of the 896-expert layer, where the gradients' own size counts
        _layer("wgrad_k3_bf16", "wgrad", "bf16", 4, 112, 16, 2048, 28, 7168, 512, False, 1.5),
        # odd sizes all round in binary32, and more duplicates than slots
        _layer("wgrad_odd_f32", "wgrad", "f32", 3, 21, 5, 333, 2, 264, 520, True, 1.5),
        # the decode shape in 8 bits: half the weights' bytes
        _layer("int8_decode", "int8", "bf16", 64, 896, 16, 128, 4, 7168, 512, True, 0.75),
        # prompts in 8 bits
        _layer("int8_uniform", "int8", "bf16", 8, 64, 8, 4096, 8, 2048, 1024, True, 0.0),
        # gradients of a layer's home experts, one tensor each: 1.6 GB
        {"name": "clip_experts_f32", "op": "clip", "dtype": "f32", "tensors": 64,
         "least": 3 * 2048 * 1024, "most": 3 * 2048 * 1024, "clips": True},
        # many small odd tensors: norms, biases, routers
        {"name": "clip_small_bf16", "op": "clip", "dtype": "bf16", "tensors": 48,
         "least": 1, "most": 20000, "clips": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.2:
        dtype = rng.choice(("f32", "bf16"))
        tensors = _log_int(rng, 1, 400)
        most = _log_int(rng, 1, min(1 << 25, (1 << 28) // tensors))
        return {"op": "clip", "dtype": dtype, "tensors": tensors, "least": max(1, most // 16),
                "most": most, "clips": rng.random() < 0.75}
    op = rng.choice(("matmul", "matmul", "wgrad", "int8"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    unit = 16 if op == "int8" else 8 if dtype == "bf16" else 4
    while True:
        R, G = _log_int(rng, 1, 32), _log_int(rng, 1, 32)
        E = R * G
        if E > 896:
            continue
        K = _log_int(rng, 1, min(16, E))
        S = _log_int(rng, 1, 8192)
        B = rng.choice((0, 1, 4, G))
        n_in = unit * _log_int(rng, 2, 7168 // unit)
        n_out = unit * _log_int(rng, 2, 7168 // unit)
        rows, held = R * S * K, (E + R * B) * n_in * n_out
        cells = rows * (n_in + n_out) + held * (2 if op == "wgrad" else 1)
        if rows <= 1 << 20 and cells <= 2 * 10 ** 9 and 2 * rows * n_in * n_out <= 4 * 10 ** 12:
            break
    return {"op": op, "dtype": dtype, "R": R, "E": E, "K": K, "S": S, "B": B, "n_in": n_in,
            "n_out": n_out, "transposed": op == "int8" or rng.random() < 0.5,
            "skew": rng.choice((0.0, 0.75, 1.5))}


# ------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _counts(case, seed):
    """Assignments routed to each expert: top-K of normal logits with a bias per expert."""
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(2 * seed + 1)
    E, K, n = case["E"], case["K"], case["R"] * case["S"]
    bias = case["skew"] * torch.randn(E, generator=g, device=dev)
    T = torch.zeros(E, dtype=torch.int64, device=dev)
    for t0 in range(0, n, 1 << 16):
        m = min(1 << 16, n - t0)
        scores = torch.randn((m, E), generator=g, device=dev) + bias
        T += torch.bincount(torch.topk(scores, K, dim=1).indices.reshape(-1), minlength=E)
    return T.cpu().numpy()


def _table(case, seed):
    """Segment table int32 [R, G + dcap + 1] (row offsets: the rank's home experts, then its
    duplicates, -1 beyond) and the experts of its duplicates [R][n_dup]."""
    R, E, SK = case["R"], case["E"], case["S"] * case["K"]
    G = E // R
    dcap = max(1, min(SK, E - G))
    T = _counts(case, seed)
    kept, over = T.copy(), {}
    lack = np.zeros(R, dtype=np.int64)
    for r in range(R):
        home = range(r * G, (r + 1) * G)
        left = int(T[r * G:(r + 1) * G].sum()) - SK
        lack[r] = max(0, -left)
        for e in sorted(home, key=lambda e: -T[e]):
            if left <= 0:
                break
            take = min(left, int(T[e]))
            kept[e] -= take
            over[e] = take
            left -= take
    held = [[] for _ in range(R)]
    for r in sorted(range(R), key=lambda r: -lack[r]):
        need = int(lack[r])
        while need > 0:
            enough = [e for e in over if over[e] >= need]
            last = len(held[r]) + 1 >= case["B"] and enough
            e = min(enough, key=lambda e: (over[e], e)) if last else max(over, key=lambda e: (over[e], -e))
            take = min(need, over[e])
            held[r].append((e, take))
            over[e] -= take
            need -= take
            if over[e] == 0:
                del over[e]
    table = np.full((R, G + dcap + 1), -1, dtype=np.int32)
    for r in range(R):
        rows = np.concatenate([kept[r * G:(r + 1) * G], [c for _, c in held[r]]])
        table[r, 0] = 0
        table[r, 1:len(rows) + 1] = np.cumsum(rows)
    return table, [[e for e, _ in h] for h in held]


def _randn(g, shape, dtype, std):
    return torch.randn(shape, generator=g, device=g.device, dtype=dtype).mul_(std)


def _duplicates(case, w, experts):
    """[R, B, ...]: the home weights of each duplicate that has a slot."""
    R, B = case["R"], case["B"]
    out = torch.zeros((R, B) + tuple(w.shape[1:]), dtype=w.dtype, device=w.device)
    for r in range(R):
        for b, e in enumerate(experts[r][:B]):
            out[r, b] = w[e]
    return out


def _sizes(case):
    """Elements of each gradient tensor: a model's own, the same for every seed."""
    rng = np.random.default_rng(case["tensors"] + case["most"])
    return rng.integers(case["least"], case["most"] + 1, case["tensors"])


def _prepare_clip(case, seed):
    dev, dt = _device(), _DT[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    sizes = _sizes(case)
    grads = [_randn(g, (int(n),), dt, 0.01) for n in sizes]
    flat = torch.empty(int(sizes.sum()), dtype=dt, device=dev)  # one buffer, a view for each
    norm = 0.01 * math.sqrt(float(sizes.sum()))
    return {"op": "clip", "grads": grads, "flat": flat, "outs": list(flat.split(sizes.tolist())),
            "max_norm": norm / 4 if case["clips"] else norm * 4,
            "acc": torch.empty(4096, dtype=torch.float64, device=dev),
            "norm": torch.empty(1, dtype=torch.float32, device=dev)}


def prepare(case, seed):
    if case["op"] == "clip":
        return _prepare_clip(case, seed)
    dev, op, dt = _device(), case["op"], _DT[case["dtype"]]
    R, E, B, SK = case["R"], case["E"], case["B"], case["S"] * case["K"]
    n_in, n_out = case["n_in"], case["n_out"]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    table, experts = _table(case, seed)
    s = {k: case[k] for k in ("op", "R", "E", "K", "S", "B", "n_in", "n_out", "transposed", "dtype")}
    s["seg_ptr"] = torch.from_numpy(table).to(dev)
    s["x"] = _randn(g, (R, SK, n_in), dt, 1.0)
    shape = (n_out, n_in) if case["transposed"] else (n_in, n_out)
    if op == "wgrad":
        s["g"] = _randn(g, (R, SK, n_out), dt, 1.0)
        s["home"] = torch.zeros((E,) + shape, dtype=torch.float32, device=dev)
        s["dup"] = torch.zeros((R, B) + shape, dtype=torch.float32, device=dev)
        return s
    if op == "int8":
        s["w"] = torch.randint(-127, 128, (E,) + shape, generator=g, device=dev, dtype=torch.int8)
        s["w_scale"] = torch.rand((E, n_out), generator=g, device=dev) * (2.0 / 127 / n_in ** 0.5)
        s["dup_w_scale"] = _duplicates(case, s["w_scale"], experts)
        s["q"] = torch.empty((R, SK, n_in), dtype=torch.int8, device=dev)
        s["x_scale"] = torch.empty((R, SK), dtype=torch.float32, device=dev)
    else:
        s["w"] = _randn(g, (E,) + shape, dt, n_in ** -0.5)
    s["dup_w"] = _duplicates(case, s["w"], experts)
    # rows of duplicates without a slot are nobody's: they keep these zeros
    s["y"] = torch.zeros((R, SK, n_out), dtype=dt, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def _segments(s):
    """(rank, first row, end, expert or None, slot or None) of each segment that has weights."""
    R, G, B = s["R"], s["E"] // s["R"], s["B"]
    for r, row in enumerate(s["seg_ptr"].tolist()):
        for j, (lo, hi) in enumerate(zip(row, row[1:])):
            if hi >= lo >= 0 and j < G + B:
                yield (r, lo, hi, r * G + j, None) if j < G else (r, lo, hi, None, j - G)


def _plain_matmul(s):
    y = s["y"]
    for r, lo, hi, e, b in _segments(s):
        w = (s["w"][e] if b is None else s["dup_w"][r, b]).float()
        y[r, lo:hi] = (s["x"][r, lo:hi].float() @ (w.t() if s["transposed"] else w)).to(y.dtype)
    return {"y": y}


def _plain_wgrad(s):
    for r, lo, hi, e, b in _segments(s):
        x, g = s["x"][r, lo:hi].float(), s["g"][r, lo:hi].float()
        into = s["home"][e] if b is None else s["dup"][r, b]
        torch.mm(g.t(), x, out=into) if s["transposed"] else torch.mm(x.t(), g, out=into)
    return {"home": s["home"], "dup": s["dup"]}


def _quantise(x):
    """(q, scale) of rows in binary32: q = rint(x * (127 / a)), scale = a / 127 with a the
    row's largest magnitude, 2^-100 at least."""
    x = x.float()
    a = x.abs().amax(dim=-1).clamp_min(_TINY)
    most = torch.full_like(a, 127.0)
    return torch.round(x * (most / a).unsqueeze(-1)), a / most


def _plain_int8(s):
    y = s["y"]
    for r in range(s["R"]):
        q, scale = _quantise(s["x"][r])
        s["q"][r], s["x_scale"][r] = q.to(torch.int8), scale
    for r, lo, hi, e, b in _segments(s):
        w, ws = (s["w"][e], s["w_scale"][e]) if b is None else (s["dup_w"][r, b], s["dup_w_scale"][r, b])
        sums = s["q"][r, lo:hi].float() @ w.float().t()
        y[r, lo:hi] = (sums * s["x_scale"][r, lo:hi, None] * ws).to(y.dtype)
    return {"y": y, "x_scale": s["x_scale"]}


def _plain_clip(s):
    norm = torch.stack([t.double().square().sum() for t in s["grads"]]).sum().sqrt()
    c = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * c)
    return {"norm": norm.float().reshape(1), "grads": s["flat"]}


def _own(s):
    import token_dispatch_amd as td
    if s["op"] == "clip":
        grads = td.GradList(s["grads"], outs=s["outs"])
        td.moonep_grad_sumsq(grads, s["acc"])
        td.moonep_grad_clip(grads, s["acc"], s["max_norm"], s["norm"])
        return {"norm": s["norm"], "grads": s["flat"]}
    dt = td.BF16 if s["dtype"] == "bf16" else td.F32
    dims = td.Dims(s["R"], s["E"], s["K"], s["S"], s["B"], dt, s["n_out"])
    if s["op"] == "matmul":
        td.moonep_expert_matmul(dims, s["seg_ptr"], s["x"], s["w"], s["dup_w"], s["y"],
                                transposed=s["transposed"])
        return {"y": s["y"]}
    if s["op"] == "wgrad":
        td.moonep_expert_matmul_wgrad(dims, s["seg_ptr"], s["x"], s["g"], s["home"], s["dup"],
                                      transposed=s["transposed"])
        return {"home": s["home"], "dup": s["dup"]}
    td.moonep_quantize_rows(s["x"], s["q"], s["x_scale"])
    td.moonep_expert_matmul_quant(dims, s["seg_ptr"], s["q"], s["x_scale"], s["w"], s["w_scale"],
                                  s["dup_w"], s["dup_w_scale"], s["y"])
    return {"y": s["y"], "x_scale": s["x_scale"]}


def run(s):
    if own:
        return _own(s)
    plain = {"matmul": _plain_matmul, "wgrad": _plain_wgrad, "int8": _plain_int8, "clip": _plain_clip}
    return plain[s["op"]](s)


# ------------------------------------------------------------------ what it cannot do without

def work(case):
    if case["op"] == "clip":
        n = int(_sizes(case).sum())
        return {"bytes": 2 * n * _ES[case["dtype"]], "flops": 3 * n}
    R, G, B = case["R"], case["E"] // case["R"], case["B"]
    n_in, n_out, es = case["n_in"], case["n_out"], _ES[case["dtype"]]
    table, _ = _table(case, 0)  # segments with rows, as routing of this skew leaves them
    full = (np.diff(table, axis=1) > 0) & (np.arange(table.shape[1] - 1) < G + B)[None, :]
    rows = int(np.diff(table, axis=1)[full].sum())
    segs, flops = int(full.sum()), 2.0 * rows * n_in * n_out
    if case["op"] == "wgrad":
        segs += R * G - int(full[:, :G].sum())  # an expert without rows has a gradient of zeros
        return {"bytes": rows * (n_in + n_out) * es + 4.0 * segs * n_in * n_out, "flops": flops}
    ws = 1 if case["op"] == "int8" else es
    return {"bytes": rows * (n_in + n_out) * es + float(segs) * n_in * n_out * ws, "flops": flops}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        flat = torch.cat([t.double() for t in s["grads"]])
        norm = torch.linalg.vector_norm(flat)
        factor = s["max_norm"] / norm if norm > s["max_norm"] else torch.ones_like(norm)
        return {"norm": norm.reshape(1), "grads": flat * factor}
    R, G, B, tr = case["R"], case["E"] // case["R"], case["B"], case["transposed"]
    table = s["seg_ptr"].cpu().numpy()
    where = [(r, j, int(table[r, j]), int(table[r, j + 1])) for r in range(R) for j in range(G + B)
             if j + 1 < table.shape[1] and table[r, j + 1] > table[r, j] >= 0]
    if case["op"] == "wgrad":
        home, dup = s["home"].double(), s["dup"].double()
        for r, j, lo, hi in where:
            d = torch.matmul(s["x"][r, lo:hi].double().t(), s["g"][r, lo:hi].double())
            d = d.t() if tr else d
            if j < G:
                home[r * G + j] = d
            else:
                dup[r, j - G] = d
        return {"home": home, "dup": dup}
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=s["y"].device)
    scale = None
    if case["op"] == "int8":
        scale = torch.empty(s["x_scale"].shape, dtype=torch.float64, device=y.device)
    for r in range(R):
        x = s["x"][r]
        if scale is not None:  # the 8-bit values are defined by their binary32 rounding
            a = torch.maximum(x.float().abs().max(dim=1).values, torch.full((1,), _TINY, device=x.device))
            x = torch.round(x.float() * torch.div(torch.full_like(a, 127.0), a)[:, None])
            scale[r] = a.double() / 127.0
        for _, j, lo, hi in (t for t in where if t[0] == r):
            w = (s["w"][r * G + j] if j < G else s["dup_w"][r, j - G]).double()
            z = torch.matmul(x[lo:hi].double(), w.t() if tr else w)
            if scale is not None:
                ws = s["w_scale"][r * G + j] if j < G else s["dup_w_scale"][r, j - G]
                z = z * scale[r, lo:hi, None] * ws.double()
            y[r, lo:hi] = z
    return {"y": y} if scale is None else {"y": y, "x_scale": scale}
