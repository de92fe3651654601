"""Plain forms, in 64 bits, of what stands around the experts' products: rows in 4 bits, the
norm, the gated activation, and the whole layer for a few tokens."""
import torch

U = 2.0 ** -24       # half a step of binary32, relative
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def scale_cols(cols):
    return (cols // 32 + 3) // 4 * 4


def mx_quantise(v):
    """(codes int64 [..., n], bytes int64 [..., n / 32]) of binary32 v, by the header's rule: the
    block's exponent from frexp, the codes by counting the borders that a value passes."""
    b = v.double().unflatten(-1, (-1, 32))
    m = b.abs().amax(-1)
    finite = torch.isfinite(b).all(-1)
    m = torch.where(finite, m, torch.ones_like(m))
    mantissa, exponent = torch.frexp(m)  # m = mantissa * 2^exponent, mantissa in [0.5, 1)
    biased = (exponent.long() - 1 + 127).clamp(min=0)  # binary32's field; 0 for its small numbers
    # in the small numbers' range the field grows by one at 1.75 * 2^-127 only
    up = torch.where(biased > 0, mantissa >= 0.875, m >= 1.75 * 2.0 ** -127)
    biased = torch.where(m < 2.0 ** -126, torch.zeros_like(biased), biased) + up.long()
    byte = (biased - 2).clamp(min=0)
    y = torch.where(finite[..., None], b, torch.zeros_like(b)).abs() / torch.exp2(byte.double() - 127)[..., None]
    code = torch.zeros_like(y, dtype=torch.int64)
    for i in range(7):
        border = (LEVELS[i] + LEVELS[i + 1]) / 2
        # a tie goes to the even code: up from odd ones
        code += (y >= border).long() if i % 2 else (y > border).long()
    code += 8 * torch.signbit(b).long()
    code = torch.where(finite[..., None], code, torch.zeros_like(code))
    byte = torch.where(finite, byte, torch.full_like(byte, 255))
    return code.flatten(-2), byte


def mx_pack(codes, byte):
    """(q, scale) uint8 as the library lays them out."""
    q = (codes[..., 0::2] + 16 * codes[..., 1::2]).to(torch.uint8)
    scale = torch.zeros(byte.shape[:-1] + (scale_cols(codes.shape[-1]),), dtype=torch.uint8, device=q.device)
    scale[..., :byte.shape[-1]] = byte.to(torch.uint8)
    return q, scale


def mx_values(q, scale, n):
    """The binary64 values of codes [..., n / 2] and scales; NaN where a scale is 255."""
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    level = torch.tensor(LEVELS, dtype=torch.float64, device=q.device)[codes % 8] * (1 - 2 * (codes // 8))
    byte = scale[..., :n // 32].double()
    size = torch.where(byte == 255, torch.full_like(byte, float("nan")), torch.exp2(byte - 127))
    return level * size.repeat_interleave(32, -1)


def plain_norm(x, gamma, eps, residual=None):
    """(h as stored, v in binary32 by the header's steps, v in 64 bits, inv in 64 bits)."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    inv = 1 / torch.sqrt(h.double().square().sum(-1, keepdim=True) / h.shape[-1] + eps)
    v32 = h.float() * inv.float() * gamma.float()
    return h, v32, h.double() * inv * gamma.double(), inv[..., 0]


def quantise8(v):
    """(q, scale) of binary32 v by the header's rule."""
    finite = torch.isfinite(v).all(-1)
    a = v.abs().amax(-1).clamp_min(2.0 ** -100)
    inv = torch.where(finite, torch.div(torch.full_like(a, 127.0), a), torch.zeros_like(a))
    q = torch.where(finite[..., None], torch.round(v * inv[..., None]), torch.zeros_like(v))
    return q.to(torch.int8), torch.where(finite, torch.div(a, torch.full_like(a, 127.0)),
                                         torch.full_like(a, float("nan")))


def plain_swiglu(g, u):
    """(value, bound) in 64 bits; the bound is binary32's: exp within a step (2 U), the sum, the
    quotient, the product and slack of as much; where exp overflows the value is below
    |g| e^-88 |u|."""
    g, u = g.double(), u.double()
    v = g * torch.sigmoid(g) * u
    return v, v.abs() * (8 * U) + u.abs() * 2.0 ** -119


def plain_swiglu_backward(go, g, u):
    """(grad_gate, bound, grad_up, bound). s is off by 4 U relative, so 1 - s by 5 U, and the
    bracket 1 + g (1 - s) by 7 U (1 + |g|); s and the three products before it by 7 U more."""
    go, g, u = go.double(), g.double(), u.double()
    s = torch.sigmoid(g)
    dg, du = go * u * s * (1 + g * (1 - s)), go * g * s
    tiny = 2.0 ** -119 * (1 + g.abs())
    return (dg, (go * u).abs() * (s * (1 + g.abs()) * (16 * U) + tiny), du,
            du.abs() * (8 * U) + go.abs() * tiny)


def plain_layer(ids, w, x, gate, up, down, E, pieces):
    """(out, bound before the store) in 64 bits of a layer over float64 weights [E, ...]. Products
    of n terms in binary32 are within n 2^-23 sum |terms|; silu has a slope below 1.1; `pieces`
    is what the activation loses between the products, relative."""
    T, K = ids.shape
    H, F = x.shape[-1], gate.shape[1]
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    step = 2.0 ** -23
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            if e < 0 or e >= E:
                continue
            xt = x[t].double()
            g, u = gate[e] @ xt, up[e] @ xt
            eg = H * step * (gate[e].abs() @ xt.abs())
            eu = H * step * (up[e].abs() @ xt.abs())
            s = g * torch.sigmoid(g)
            a = s * u
            ea = 1.1 * u.abs() * eg + s.abs() * eu + 1.1 * eg * eu + 10 * U * a.abs()
            wk = w[t, k].double()
            out[t] += wk * (down[e] @ a)
            bound[t] += wk.abs() * (down[e].abs() @ (ea + pieces * a.abs()))
            mag[t] += wk.abs() * (down[e].abs() @ a.abs())
    return out, bound + (F * K + K) * step * mag
