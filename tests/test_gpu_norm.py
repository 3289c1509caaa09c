"""Group norm with an activation or a gate on the GPU against float64."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import causal_kernelized_attention_gb300 as la  # noqa: E402
from delta_ref import norm_backward, norm_forward  # noqa: E402
from hybrid_ref import U, assert_within, half  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(seed, B, L, G, D, dtype, heads_first, gate, weights, offset=0.5):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    x = 1.5 * normal(B, L, G, D) + offset
    x = (x.transpose(1, 2) if heads_first else x.reshape(B, L, G * D)).contiguous().to(dtype)
    return dict(x=x, gate=normal(B, L, G * D).to(dtype) if gate else None, w=1 + 0.3 * normal(G * D) if weights else None,
                b=0.2 * normal(G * D) if weights else None), normal(B, L, G * D).to(dtype)


def run(s, dy, G, act, per_token, heads_first, center, eps=1e-5):
    c = {i: None if x is None else x.cuda() for i, x in s.items()}
    kw = dict(w=c["w"], b=c["b"], gate=c["gate"], act=act, eps=eps, per_token=per_token, heads_first=heads_first, center=center)
    y, mean, rstd = la.la_group_norm_forward(c["x"], G, **kw)
    return (y, mean, rstd), la.la_group_norm_backward(c["x"], G, mean, rstd, dy.cuda(), **kw)


def check(s, dy, G, act, per_token, heads_first, center, eps=1e-5):
    (y, mean, rstd), (dx, dgate, dw, db) = run(s, dy, G, act, per_token, heads_first, center, eps)
    wy, wm, wr = norm_forward(s["x"], G, s["w"], s["b"], s["gate"], act, eps, per_token, heads_first, center)
    assert_within(y, *wy, "y")
    assert_within(rstd, *wr, "rstd")
    if center:
        assert_within(mean, *wm, "mean")
    else:
        assert mean is None
    wx, wg, ww, wb = norm_backward(s["x"], G, None if mean is None else mean.cpu(), rstd.cpu(), dy, s["w"], s["b"], s["gate"], act,
                                   per_token, heads_first, center)
    assert_within(dx, *wx, "dx")
    if s["gate"] is not None:
        assert_within(dgate, *wg, "dgate")
    if s["w"] is not None:
        assert_within(dw, *ww, "dw")
        assert_within(db, *wb, "db")
    else:
        assert dw is None and db is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_token,heads_first", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("center,gate,weights,act", [(c, g, w, a) for (c, g, w), a in
                                                     zip(itertools.product((True, False), repeat=3), ("silu", "silu", "none", "silu") * 2)])
def test_forms(dtype, per_token, heads_first, center, gate, weights, act):
    s, dy = inputs(1, 2, 37, 3, 16, TYPES[dtype], heads_first, gate, weights)
    check(s, dy, 3, act, per_token, heads_first, center)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,G,D", [(1, 1, 1, 1), (1, 1, 1, 8), (3, 5, 7, 33), (1, 2, 1, 512), (2, 3, 2, 509), (1, 300, 40, 8),
                                     (2, 9, 32, 64), (1, 33, 5, 100), (1, 3, 2, 600), (1, 4, 1, 1031), (1, 1, 300, 4)])
@pytest.mark.parametrize("gate", [False, True])
def test_tokens(B, L, G, D, dtype, gate):
    s, dy = inputs(2, B, L, G, D, TYPES[dtype], False, gate, True)
    check(s, dy, G, "silu", True, False, True)
    if D <= 512:
        s, dy = inputs(3, B, L, G, D, TYPES[dtype], True, gate, True)
        check(s, dy, G, "silu", True, True, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,G,D", [(1, 1, 1, 1), (1, 2, 3, 1), (2, 1, 4, 8), (3, 777, 11, 3), (1, 1000, 1, 64), (2, 256, 32, 40),
                                     (5, 33, 1, 7), (1, 19, 2, 1200), (1, 4001, 8, 10), (70, 3, 2, 8), (1, 5, 1, 2056),
                                     # too long for one cluster's shared memory; and, with a ragged edge in channels, too wide
                                     (1, 60000, 2, 16), (2, 3001, 3, 700)])
@pytest.mark.parametrize("gate", [False, True])
def test_maps(B, L, G, D, dtype, gate):
    s, dy = inputs(4, B, L, G, D, TYPES[dtype], False, gate, True)
    check(s, dy, G, "silu", False, False, True)
    check(s, dy, G, "none", False, False, False)


@pytest.mark.parametrize("per_token", [True, False])
def test_values_far_from_zero(per_token):
    """A mean of 1000 spreads: differences are taken before squares."""
    s, dy = inputs(5, 2, 400, 4, 32, torch.float32, False, False, True, offset=1500.0)
    check(s, dy, 4, "silu", per_token, False, True)


@pytest.mark.parametrize("per_token", [True, False])
def test_a_constant_group(per_token):
    """No spread: h = 0, rstd = 1 / sqrt(eps)."""
    s, dy = inputs(6, 2, 16, 2, 8, torch.float32, False, False, True)
    s["x"].fill_(3.0)
    (y, mean, rstd), _ = run(s, dy, 2, "none", per_token, False, True)
    assert torch.equal(y.cpu(), s["b"].expand(2, 16, 16)) and bool((mean == 3).all())
    assert bool(((rstd - 1e-5 ** -0.5).abs() <= 1e-4 * 1e-5 ** -0.5).all())


def test_a_token_alone_is_unaffected_by_nan_elsewhere():
    s, dy = inputs(7, 1, 40, 4, 64, torch.bfloat16, False, True, True)
    clean, _ = run(s, dy, 4, "silu", True, False, True)
    s["x"][0, 7, :64] = float("nan")
    (y, _, _), _ = run(s, dy, 4, "silu", True, False, True)
    assert bool(y[0, 7, :64].isnan().all())
    y[0, 7, :64] = clean[0][0, 7, :64]
    assert torch.equal(y, clean[0])


def test_deterministic():
    s, dy = inputs(8, 4, 1500, 8, 40, torch.bfloat16, False, True, True)
    for per_token in (True, False):
        a, b = (run(s, dy, 8, "silu", per_token, False, True)[1] for _ in range(2))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_positions_give_zero_weight_gradients():
    x = torch.zeros((2, 0, 16), device="cuda")
    w = torch.ones(16, device="cuda")
    y, mean, rstd = la.la_group_norm_forward(x, 2, w=w, b=w, per_token=True)
    dx, _, dw, db = la.la_group_norm_backward(x, 2, mean, rstd, y, w=w, b=w, per_token=True)
    assert dx.numel() == 0 and not dw.any() and not db.any()


@pytest.mark.parametrize("per_token", [True, False])
def test_graph(per_token):
    s, dy = inputs(9, 2, 300, 4, 32, torch.bfloat16, False, True, True)
    t, dy2 = inputs(10, 2, 300, 4, 32, torch.bfloat16, False, True, True)
    want = run(t, dy2, 4, "silu", per_token, False, True)
    c = {i: x.cuda() for i, x in s.items()}
    d = dy.cuda()
    kw = dict(w=c["w"], b=c["b"], gate=c["gate"], act="silu", per_token=per_token)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        la.la_group_norm_forward(c["x"], 4, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd = la.la_group_norm_forward(c["x"], 4, **kw)
        bwd = la.la_group_norm_backward(c["x"], 4, fwd[1], fwd[2], d, **kw)
    for i, x in t.items():
        c[i].copy_(x)
    d.copy_(dy2)
    graph.replay()
    for got, ref in zip(fwd + bwd, want[0] + want[1]):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,G,D,gate", [(3, 2900, 32, 40, False), (2, 4100, 32, 40, True), (1, 9000, 10, 206, False), (40, 700, 5, 52, True)])
def test_large_maps(B, L, G, D, dtype, gate):
    """Tensors beyond what one launch holds on chip, with columns that share a block and that do not."""
    s, dy = inputs(11, B, L, G, D, TYPES[dtype], False, gate, True)
    check(s, dy, G, "silu", False, False, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,G,D", [(2, 64, 4, 16), (2, 4200, 32, 40)])  # one launch, and three
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e25])
def test_infinities_and_overflow_over_positions(value, B, L, G, D, dtype):
    """An infinity or a NaN makes its group's statistics NaN or infinite and y NaN; finite values whose squares overflow fp32
    have a variance of infinity (rstd = 0).  Neither looks like a spread of 0 (rstd = 1 / sqrt(eps)).  The other groups are as without."""
    s, dy = inputs(12, B, L, G, D, TYPES[dtype], False, False, True)
    (y, mean, rstd), _ = run(s, dy, G, "none", False, False, True)
    s["x"][1, L // 3, D + 2] = value
    (y2, mean2, rstd2), _ = run(s, dy, G, "none", False, False, True)
    if value == 1e25:
        assert float(rstd2[1, 1]) == 0 and torch.equal(y2[1, :, D:2 * D].cpu(), s["b"][D:2 * D].to(TYPES[dtype]).expand(L, D))
    else:
        assert bool(rstd2[1, 1].isnan()) and not bool(mean2[1, 1].isfinite()) and bool(y2[1, :, D:2 * D].isnan().all())
    y2[1, :, D:2 * D], mean2[1, 1], rstd2[1, 1] = y[1, :, D:2 * D], mean[1, 1], rstd[1, 1]
    assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    # without centring the mean square is infinite, too
    (y3, _, rstd3), _ = run(s, dy, G, "none", False, False, False)
    assert bool(rstd3[1, 1].isnan()) if value != value else float(rstd3[1, 1]) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,G,D", [(2, 1024, 4, 16), (1, 19, 2, 1200), (1, 16384, 4, 64), (2, 8191, 8, 40), (1, 262144, 1, 7)])
@pytest.mark.parametrize("place,value,mean,spread", [("first", 300.0, 0.0, 1.0), ("first", 1e4, 0.0, 1.0), ("last", -1e4, 0.0, 1.0), ("middle", 3e3, 5.0, 1.0),
                                                     ("first", 0.0, 1000.0, 0.1), ("first", 0.0, 100.0, 0.1)])
def test_an_outlier_over_positions(place, value, mean, spread, B, L, G, D, dtype):
    """One value far from the others of its group, the first, the last or another.  The variance is a sum of squares, none
    negative, of which a thread adds at most 200 one after another here, a block at most 256, the join 64 and its trees 9: each
    addition and each square's own steps are off by at most u of what stands, 600 u of the variance together, 300 u of rstd; the
    mean by as many u of the spread, and 4 u of itself.  (Differences from any one value of the group would cost u (mean -
    value)^2 as often as there are values.)"""
    s, _ = inputs(13, B, L, G, D, TYPES[dtype], False, False, True)
    gen = torch.Generator().manual_seed(14)
    x = (mean + spread * torch.randn((B, L, G, D), generator=gen)).to(TYPES[dtype])
    at = {"first": (0, 0), "last": (L - 1, D - 1), "middle": (L // 2, D // 3)}[place]
    x[:, at[0], :, at[1]] = value
    s["x"] = x.reshape(B, L, G * D)
    c = {i: None if t is None else t.cuda() for i, t in s.items()}
    y, m, r = la.la_group_norm_forward(c["x"], G, w=c["w"], b=c["b"])
    x64 = x.double()
    want = x64.mean((1, 3), keepdim=True)
    var = (x64 - want).square().mean((1, 3), keepdim=True)
    rstd = (var + 1e-5).rsqrt()
    em = 300 * U * var.sqrt() + 4 * U * want.abs()
    assert_within(m, want.reshape(B, G), em.reshape(B, G), "mean")
    # (an error of the mean adds its square to the variance)
    er = rstd * (300 * U + 0.5 * (em * rstd).square())
    assert_within(r, rstd.reshape(B, G), er.reshape(B, G), "rstd")
    h = (x64 - want) * rstd
    z = (h * s["w"].double().reshape(G, D) + s["b"].double().reshape(G, D)).reshape(B, L, G * D)
    eh = em * rstd + h.abs() * (er / rstd + 4 * U) + 2 * U * want.abs() * rstd
    ez = (eh * s["w"].double().abs().reshape(G, D)).reshape(B, L, G * D) + 4 * U * (z.abs() + s["b"].double().abs())
    assert_within(y, z, ez + half(TYPES[dtype]) * z.abs() + 1e-30, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("B,L,G,D", [(5, 1501, 16, 64), (3, 2003, 16, 40), (3, 2003, 16, 30), (5, 3001, 3, 509), (7, 2999, 5, 8)])
def test_walks_over_many_tokens(B, L, G, D, heads_first, dtype):
    """Six and more tokens to a slot, whose lengths divide neither the step nor one another, with entries to cross."""
    s, dy = inputs(15, B, L, G, D, TYPES[dtype], heads_first, True, True)
    check(s, dy, G, "silu", True, heads_first, not heads_first)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,G,D,gate", [(1, 4096, 1, 4096, True), (2, 1300, 2, 2049, False), (3, 2500, 1, 1030, True)])
def test_wide_groups_of_many_tokens(B, L, G, D, gate, dtype):
    """Tokens wider than the lanes' registers, more of them than one launch holds on chip."""
    s, dy = inputs(16, B, L, G, D, TYPES[dtype], False, gate, True)
    check(s, dy, G, "silu", True, False, True)
    check(s, dy, G, "none", True, False, False)
