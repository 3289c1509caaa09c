"""Plain float64 forms of the hybrid-layer operators, with bounds on what a kernel's fp32
arithmetic and roundings may be off.

Units: u = 2^-24 is half a step of fp32, half(t) half a step of an output type relative to
the value (bf16 2^-8).  Each bound counts roundings of the kernel's own arithmetic; the
constants are explained where they are used.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126  # the smallest normal fp32 (and bf16) value: what underflows is off by at most this


def half(dtype):
    return torch.finfo(dtype).eps / 2


def draw(seed, shape, dtype, scale=1.0):
    """Seeded normal values on the CPU, rounded to `dtype`."""
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def assert_within(got, want, bound, what=""):
    """|got - want| <= bound elementwise (float64), NaN and infinities in the same places."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), (what, "finite places differ")
    assert torch.equal(got[~fine].nan_to_num(7.0), want[~fine].nan_to_num(7.0)), (what, "non-finite values differ")
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, (what, "over the bound by", float(over.max()),
                                                         "worst error", float((got - want)[fine].abs().max()))


# ---------------------------------------------------------------- rotary
def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0, ramp=(1.0, 32.0)):
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else base
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "ramp":
            g = min(1.0, max(0.0, (original * f / (2 * math.pi) - ramp[0]) / (ramp[1] - ramp[0])))
            f *= g + (1 - g) / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotary(x, positions, rot, layout="half", amplitude=1.0, inverse=False, **options):
    """x [B,H,N,d] (any float type), positions [B,N]; returns (float64 result, bound)."""
    y = x.double()
    ang = positions.double()[:, None, :, None] * frequencies(rot, **options)
    # fractions of a turn, as a far position's own angle loses digits even in float64
    cos, sin = amplitude * ang.cos(), amplitude * ang.sin()
    if inverse:
        sin = -sin
    if layout == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    # sine and cosine within 4 u of 1 (the fraction of a turn as a float, sincospif's 2 ulp, the
    # amplitude's product), each product and the sum one more u; float64's own angle error
    # is |angle| 2^-50
    per = (abs(amplitude) * (7 * U + ang.abs() * 2.0 ** -50)) * (a.abs() + b.abs())
    out, bound = y.clone(), torch.zeros_like(y)
    if layout == "half":
        out[..., :rot // 2], out[..., rot // 2:rot] = ra, rb
        bound[..., :rot // 2] = bound[..., rot // 2:rot] = per
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = ra, rb
        bound[..., 0:rot:2] = bound[..., 1:rot:2] = per
    return out, bound * (1 + half(x.dtype)) + half(x.dtype) * out.abs() * (torch.arange(y.shape[-1]) < rot)


# ---------------------------------------------------------------- recurrence
def recurrence(alpha, x, first):
    """(h [B,N,D], bound) in float64, token by token.  A path from x_s to h_t has t - s products and as many
    sums; the joins of runs add at most 32 more, each within u: 2 u (t - s + 32) of its weight."""
    a, x = alpha.double(), x.double()
    h = torch.zeros_like(x[:, 0]) if first is None else first.double()
    m, n = h.abs(), torch.zeros_like(h)
    hs, bs = [], []
    for t in range(x.shape[1]):
        h = a[:, t] * h + x[:, t]
        n = a[:, t].abs() * (n + m)
        m = a[:, t].abs() * m + x[:, t].abs()
        hs.append(h)
        bs.append(2 * U * (n + 32 * m))
    return torch.stack(hs, 1), torch.stack(bs, 1)


def recurrence_backward(alpha, h, dh, h0, dhN):
    """(dx, dalpha, dh0) with their fp32 bounds (before the rounding to the output's type)."""
    a = alpha.double()
    later = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1).flip(1)
    g, e = (t.flip(1) for t in recurrence(later, dh.double().flip(1), dhN))
    before = torch.cat((torch.zeros_like(a[:, :1]) if h0 is None else h0.double()[:, None], h.double()[:, :-1]), 1)
    da = g * before
    return (g, e), (da, e * before.abs() + U * da.abs()), (a[:, 0] * g[:, 0], a[:, 0].abs() * e[:, 0] + U * g[:, 0].abs())


# ---------------------------------------------------------------- window attention
def visible(Nq, Nk, window, sinks, n):
    """[Nq, Nk] truth values: what row t (position t + Nk - Nq) sees of an entry of n tokens."""
    p = torch.arange(Nq)[:, None] + (Nk - Nq)
    j = torch.arange(Nk)[None, :]
    return (j <= p) & (p < n) & ((p - j < window) | (j < sinks))


def window(q, k, v, window, sinks, lens, scale, dout=None, o=None, lse=None):
    """Forward: ((o, bound), (lse, bound)).  With dout, o and lse: ((dq, bound), (dk, bound), (dv, bound)).

    Bounds.  A score is d products and sums in fp32, its scaling and the softmax's subtraction: within
    (d + 8) u of scale sum |q k|, plus 4 u of |score| and |lse|; the exponential adds 4 u.  Weights (and
    dS) of 16-bit inputs are rounded for their products: half(bf16) each.  A weight (or dS, or a
    result) below TINY may become 0: TINY for each, times what it is multiplied by."""
    B, Hq, Nq, d = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    low = q.dtype != torch.float32
    r = half(torch.bfloat16) if low else 0.0
    out = [torch.zeros((B, Hq, Nq, d), dtype=torch.float64) for _ in range(2)]
    ls = [torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64), torch.zeros((B, Hq, Nq), dtype=torch.float64)]
    dq = [torch.zeros_like(out[0]) for _ in range(2)]
    dk = [torch.zeros((B, Hk, Nk, d), dtype=torch.float64) for _ in range(2)]
    dv = [torch.zeros((B, Hk, Nk, d), dtype=torch.float64) for _ in range(2)]
    for b in range(B):
        n = Nk if lens is None else max(0, min(int(lens[b]), Nk))
        see = visible(Nq, Nk, window, sinks, n)
        some = see.any(1)
        for h in range(Hq):
            hk = h // (Hq // Hk)
            # what no row sees may be anything: it takes no part
            used = see.any(0)[:, None]
            Q = torch.where(some[:, None], q[b, h].double(), 0.0)
            K, V = (torch.where(used, x[b, hk].double(), 0.0) for x in (k, v))
            z = torch.where(see, (Q @ K.T) * scale, -math.inf)
            dz = torch.where(see, (d + 8) * U * scale * (Q.abs() @ K.abs().T) + 4 * U * z.abs(), 0.0)
            worst = dz.amax(1, keepdim=True)
            if dout is None:
                L = torch.logsumexp(z, 1, keepdim=True)
                p = torch.where(some[:, None], torch.exp(z - L), 0.0)
                e = 2 * worst + (Nk + 8) * U
                ov = p @ V
                out[0][b, h] = ov
                out[1][b, h] = ((e + r) * p + TINY * see) @ V.abs() + TINY + (half(q.dtype)) * ov.abs()
                ls[0][b, h] = L[:, 0]
                ls[1][b, h] = torch.where(some, worst[:, 0] + (Nk + 8) * U + 4 * U * L[:, 0].abs(), 0.0)
                continue
            G, O = (torch.where(some[:, None], x[b, h].double(), 0.0) for x in (dout, o))
            L = torch.where(some, lse[b, h].double(), 0.0)[:, None]
            p = torch.where(see, torch.exp(z - L), 0.0)
            ep = dz + 4 * U * (1 + L.abs())  # relative error of a weight
            D = (G * O).sum(1, keepdim=True)
            gv = G @ V.T
            ds = p * (gv - D) * scale
            size = scale * (G.abs() @ V.abs().T + (G * O).abs().sum(1, keepdim=True))
            es = (r + ep + 4 * U) * ds.abs() + p * (d + 8) * U * size + TINY * see * (1 + size)
            dq[0][b, h] = ds @ K
            dq[1][b, h] = es @ K.abs() + (Nk + 8) * U * (ds.abs() @ K.abs())
            dk[0][b, hk] += ds.T @ Q
            dk[1][b, hk] += es.T @ Q.abs() + (Nq * Hq + 8) * U * (ds.abs().T @ Q.abs())
            dv[0][b, hk] += p.T @ G
            dv[1][b, hk] += ((r + ep + (Nq * Hq + 8) * U) * p + TINY * see).T @ G.abs()
    if dout is None:
        return (out[0], out[1]), (ls[0], ls[1])
    return tuple((x, e + half(q.dtype) * x.abs() + TINY) for x, e in (dq, dk, dv))


def slot(j, window, sinks):
    return j if j < sinks else sinks + (j - sinks) % window
