"""Plain float64 forms of the gated delta rule (token by token) and of group norm, with what a kernel
may be off.

Units: u = 2^-24 is half a step of fp32, half(t) half a step of an output type relative to the value
(bf16 2^-8; a rounding's root mean square is 2^-9 of the values' where they are spread evenly).
"""
from __future__ import annotations

import math

import torch

from hybrid_ref import TINY, U, half

F64 = torch.float64


def delta_inputs(seed, B, Hk, H, N, dk, dv, dtype, initial=True, resets=()):
    """Unit keys and queries, gates from nearly open to nearly closed, -inf at the tokens `resets`."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    s = dict(q=unit(normal(B, Hk, N, dk)), k=unit(normal(B, Hk, N, dk)), v=normal(B, H, N, dv).to(dtype),
             g=-2.0 * torch.rand((1, H, 1), generator=gen) * torch.nn.functional.softplus(normal(B, H, N) - 2.0),
             beta=torch.sigmoid(normal(B, H, N)), dout=normal(B, H, N, dv).to(dtype), S0=None, dSN=None)
    if initial:
        s["S0"], s["dSN"] = 0.3 * normal(B, H, dk, dv), 0.3 * normal(B, H, dk, dv)
    for t in resets:
        s["g"][:, :, t] = -math.inf
    return s


def delta(s, scale, backward=True):
    """dict of o, SN and, with backward, dq, dk, dv, dg, dbeta, dS0: the recurrence and its reverse as they are defined."""
    H, Hk, N = s["v"].shape[1], s["k"].shape[1], s["v"].shape[2]
    q, k = (s[i].to(F64).repeat_interleave(H // Hk, 1) for i in ("q", "k"))
    v, beta, alpha = s["v"].to(F64), s["beta"].to(F64), s["g"].to(F64).exp()
    B, dk, dv = v.shape[0], k.shape[-1], v.shape[-1]
    S = torch.zeros((B, H, dk, dv), dtype=F64) if s["S0"] is None else s["S0"].to(F64)
    states, errors, o = [S], [], torch.zeros_like(v)
    for t in range(N):
        D = alpha[:, :, t, None, None] * S
        e = v[:, :, t] - torch.einsum("bhkv,bhk->bhv", D, k[:, :, t])
        S = D + k[:, :, t, :, None] * (beta[:, :, t, None] * e)[:, :, None, :]
        o[:, :, t] = scale * torch.einsum("bhkv,bhk->bhv", S, q[:, :, t])
        states.append(S)
        errors.append(e)
    r = dict(o=o, SN=S)
    if not backward:
        return r
    do = scale * s["dout"].to(F64)
    R = torch.zeros_like(S) if s["dSN"] is None else s["dSN"].to(F64)
    dq, dk_, dv_, dg, db = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(beta), torch.zeros_like(beta)
    for t in reversed(range(N)):
        kt, qt, e, b, a = k[:, :, t], q[:, :, t], errors[t], beta[:, :, t], alpha[:, :, t]
        R = R + qt[..., :, None] * do[:, :, t, None, :]
        dq[:, :, t] = torch.einsum("bhkv,bhv->bhk", states[t + 1], do[:, :, t])
        x = torch.einsum("bhkv,bhk->bhv", R, kt)
        D = a[..., None, None] * states[t]
        dv_[:, :, t] = b[..., None] * x
        db[:, :, t] = (x * e).sum(-1)
        dk_[:, :, t] = torch.einsum("bhkv,bhv->bhk", R, b[..., None] * e) - torch.einsum("bhkv,bhv->bhk", D, dv_[:, :, t])
        R = R - kt[..., :, None] * dv_[:, :, t, None, :]
        dg[:, :, t] = (R * D).sum((-1, -2))
        R = a[..., None, None] * R
    shared = [x.reshape(B, Hk, H // Hk, N, dk).sum(2) for x in (dq, dk_)]
    r.update(dq=shared[0], dk=shared[1], dv=dv_, dg=dg, dbeta=db, dS0=R)
    return r


def delta_tolerance(dtype, out, parts):
    """Relative error allowed of a block of values, in the 2-norm.

    fp32 arithmetic: a value comes through at most 8 dot products of at most 256 terms, one after another; a sum of n
    terms is off by about u sqrt(n) in the root mean square: 8 * 16 u.  With bf16 inputs on the tensor cores (parts),
    operands of what ends in fp32 are rounded to within 2^-17 (two parts), at most 16 of them on a value's way
    and independent of one another: 4 * 2^-17, doubled for the sums' own.  What ends in bf16 may pass through four
    single roundings and its own, each 2^-9 in the root mean square at most: sqrt(5) 2^-9 < 2^-8 + 2^-10."""
    if out != torch.float32:
        return 2.0 ** -8 + 2.0 ** -10
    return 8 * 2.0 ** -17 if parts and dtype != torch.float32 else 128 * U


def assert_near(got, want, tol, what="", block=32, floor=0.02):
    """Blocks of `block` tokens of each (b, h) (or whole states) within tol of their own 2-norm; a block far below
    the others counts as `floor` of their mean."""
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), (what, "not finite")
    if want.numel() == 0:
        return
    if want.dim() == 3:
        got, want = got[..., None], want[..., None]
    n = want.shape[2]
    off, size = [], []
    for t in range(0, n, block):
        off.append((got - want)[:, :, t:t + block].square().sum((2, 3)).sqrt())
        size.append(want[:, :, t:t + block].square().sum((2, 3)).sqrt())
    off, size = torch.stack(off, 2), torch.stack(size, 2)
    bound = tol * size.clamp(min=float(size.mean()) * floor)
    worst = float((off / bound.clamp(min=TINY)).max())
    assert worst <= 1, (what, "off by", worst, "of what is allowed, in block", int((off / bound.clamp(min=TINY)).argmax()))


# ---------------------------------------------------------------- group norm
def by_group(x, groups, heads_first):
    """[B, L, G, D] in float64."""
    x = x.to(F64)
    return x.transpose(1, 2) if heads_first else x.reshape(x.shape[0], x.shape[1], groups, -1)


def silu(z, act):
    return z * torch.sigmoid(z) if act == "silu" else z


def slope(z, act):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s)) if act == "silu" else torch.ones_like(z)


def norm_forward(x, groups, w, b, gate, act, eps, per_token, heads_first, center):
    """(y, bound), (mean, bound), (rstd, bound) in float64.

    n values of size at most M about their mean (or 0): the mean is off by (log2(n) + 8) u of their mean size at
    most times the depth of the sums, taken here as (n / 32 + 8) u M, and rstd by as much relative to the
    values' spread.  h then carries both, z and act a few u more; act is at most 1.1 times as steep as z."""
    x64 = by_group(x, groups, heads_first)
    over = (3,) if per_token else (1, 3)
    n = x64.shape[3] * (1 if per_token else x64.shape[1])
    m = x64.mean(over, keepdim=True) if center else torch.zeros_like(x64.mean(over, keepdim=True))
    size = x64.abs().amax(over, keepdim=True)
    var = (x64 - m).square().mean(over, keepdim=True)
    r = 1 / (var + eps).sqrt()
    depth = (min(n, 4096) / 32 + 16) * U
    em = depth * size
    # var's own sums, and what the mean's error adds to a channel's deviations
    er = r * (depth * 4 + 2 * em * r * (size * r).clamp(max=8))
    h = (x64 - m) * r
    eh = em * r + h.abs() * (er / r + 4 * U)
    B, L, G, D = x64.shape
    wv = torch.ones(G * D, dtype=F64) if w is None else w.to(F64)
    bv = torch.zeros(G * D, dtype=F64) if b is None else b.to(F64)
    z = h.reshape(B, L, G * D) * wv + bv
    ez = eh.reshape(B, L, G * D) * wv.abs() + 4 * U * (z.abs() + bv.abs())
    if gate is None:
        y, ey = silu(z, act), 1.1 * ez + 16 * U * z.abs()
    else:
        a = silu(gate.to(F64), act)
        y, ey = z * a, a.abs() * ez + 16 * U * z.abs() * gate.to(F64).abs()
    stats = (lambda t: t.reshape(B, L, G)) if per_token else (lambda t: t.reshape(B, G))
    em, er = em.expand_as(m), er.expand_as(r)
    return (y, ey + half(x.dtype) * y.abs() + TINY), (stats(m), stats(em)), (stats(r), stats(er))


def norm_backward(x, groups, mean, rstd, dy, w, b, gate, act, per_token, heads_first, center):
    """(dx, bound), (dgate, bound), (dw, bound), (db, bound), from the statistics as given."""
    x64 = by_group(x, groups, heads_first)
    B, L, G, D = x64.shape
    over = (3,) if per_token else (1, 3)
    shape = (B, L, G, 1) if per_token else (B, 1, G, 1)
    m = mean.to(F64).reshape(shape) if center else torch.zeros(shape, dtype=F64)
    r = rstd.to(F64).reshape(shape)
    h = (x64 - m) * r
    eh = 4 * U * (h.abs() + (x64.abs() + m.abs()) * r)
    wv = (torch.ones(G * D, dtype=F64) if w is None else w.to(F64)).reshape(G, D)
    bv = (torch.zeros(G * D, dtype=F64) if b is None else b.to(F64)).reshape(G, D)
    z = h * wv + bv
    ez = eh * wv.abs() + 4 * U * (z.abs() + bv.abs())
    d = dy.to(F64).reshape(B, L, G, D)
    dgate = None
    if gate is None:
        dz = d * slope(z, act)
        edz = d.abs() * (0.5 * ez + 16 * U * (1 + z.abs()) if act == "silu" else 2 * U)  # the slope's own slope is at most 1/2
    else:
        gt = gate.to(F64).reshape(B, L, G, D)
        dz = d * silu(gt, act)
        edz = d.abs() * 16 * U * gt.abs()
        dg = d * z * slope(gt, act)
        edg = d.abs() * (1.1 * ez + 16 * U * z.abs() * (1 + gt.abs()))
        dgate = (dg.reshape(B, L, G * D), (edg + half(x.dtype) * dg.abs() + TINY).reshape(B, L, G * D))
    dh, edh = dz * wv, edz * wv.abs() + 2 * U * (dz * wv).abs()
    n = D * (1 if per_token else L)
    depth = (min(n, 4096) / 32 + 16) * U
    a2 = (dh * h).mean(over, keepdim=True)
    ea2 = (edh * h.abs() + dh.abs() * eh).mean(over, keepdim=True) + depth * (dh * h).abs().mean(over, keepdim=True)
    a1 = dh.mean(over, keepdim=True) * center
    ea1 = edh.mean(over, keepdim=True) + depth * dh.abs().mean(over, keepdim=True)
    dx = r * (dh - a1 - h * a2)
    edx = r * (edh + ea1 + h.abs() * ea2 + eh * a2.abs() + 6 * U * (dh.abs() + a1.abs() + (h * a2).abs()))
    dx, edx = dx, edx + half(x.dtype) * dx.abs() + TINY
    if heads_first:
        dx, edx = dx.transpose(1, 2), edx.transpose(1, 2)
    else:
        dx, edx = dx.reshape(B, L, G * D), edx.reshape(B, L, G * D)
    depth = (min(B * L, 4096) / 32 + 32) * U
    dw = ((dz * h).sum((0, 1)).reshape(-1), ((edz * h.abs() + dz.abs() * eh) + depth * (dz * h).abs()).sum((0, 1)).reshape(-1))
    db = (dz.sum((0, 1)).reshape(-1), (edz + depth * dz.abs()).sum((0, 1)).reshape(-1))
    return (dx, edx), dgate, dw, db
