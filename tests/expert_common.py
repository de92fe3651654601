"""Plain 64-bit forms of the experts' products and the tables their tests use."""
import numpy as np
import torch

# One binary32 rounding is off by at most 2^-24 relative. A matrix unit may round each
# partial sum less carefully than to nearest: a whole step, 2^-23, is allowed for each.
ADD = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def torch_dtype(dtype):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]


def make_table(rows, R, G, dcap, SK):
    """Segment table [R, G + dcap + 1] from each rank's list of segment lengths."""
    t = np.full((R, G + dcap + 1), -1, dtype=np.int32)
    for r, lens in enumerate(rows):
        assert len(lens) <= G + dcap and sum(lens) <= SK
        t[r, 0] = 0
        t[r, 1:len(lens) + 1] = np.cumsum(lens)
    return t


def segments(table, G, B, SK):
    """(rank, segment, first row, end) of the segments that have a matrix, as the header
    defines them: negative offsets and ends not past their start are empty."""
    n = table.shape[1] - 1
    for r in range(table.shape[0]):
        for j in range(min(G + B, n)):
            lo, hi = int(table[r, j]), min(int(table[r, j + 1]), SK)
            yield r, j, lo, max(lo, hi) if lo >= 0 else lo


def plain_matmul(table, G, B, x, w, dup_w, transposed):
    """(y, magnitude, written) in 64 bits: sum x w, sum |x w|, and the rows of a segment."""
    R, SK = x.shape[:2]
    n_out = w.shape[-2] if transposed else w.shape[-1]
    y = torch.zeros((R, SK, n_out), dtype=torch.float64, device=x.device)
    mag, written = torch.zeros_like(y), torch.zeros((R, SK), dtype=torch.bool, device=x.device)
    for r, j, lo, hi in segments(table, G, B, SK):
        if lo < 0 or hi <= lo:
            continue
        m = (w[r * G + j] if j < G else dup_w[r, j - G]).double()
        m = m.t().contiguous() if transposed else m
        a = x[r, lo:hi].double()
        y[r, lo:hi], mag[r, lo:hi], written[r, lo:hi] = a @ m, a.abs() @ m.abs(), True
    return y, mag, written


def plain_wgrad(table, G, B, x, g, transposed):
    """(home, dup, magnitudes, which duplicate slots are written) in 64 bits."""
    R, SK = x.shape[:2]
    shape = (g.shape[-1], x.shape[-1]) if transposed else (x.shape[-1], g.shape[-1])
    new = lambda *lead: torch.zeros(lead + shape, dtype=torch.float64, device=x.device)  # noqa: E731
    home, dup, mh, md = new(R * G), new(R, B), new(R * G), new(R, B)
    written = torch.zeros((R, B), dtype=torch.bool, device=x.device)
    n = table.shape[1] - 1
    for r, j, lo, hi in segments(table, G, B, SK):
        if j >= G:
            written[r, j - G] = lo >= 0 and int(table[r, j + 1]) >= lo
        if lo < 0 or hi <= lo:
            continue
        a, b = x[r, lo:hi].double(), g[r, lo:hi].double()
        a, b = (b, a) if transposed else (a, b)
        d, m = a.t().contiguous() @ b, a.abs().t().contiguous() @ b.abs()
        if j < G:
            home[r * G + j], mh[r * G + j] = d, m
        else:
            dup[r, j - G], md[r, j - G] = d, m
    assert n >= G
    return home, dup, mh, md, written


def assert_within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
            f"{got.reshape(-1)[i].item()} for {want.reshape(-1)[i].item()} "
            f"(allowed {bound.reshape(-1)[i].item():.3g})")
