"""Gated delta rule on the GPU against the recurrence in float64."""
import math

import pytest

torch = pytest.importorskip("torch")

import causal_kernelized_attention_gb300 as la  # noqa: E402
from delta_ref import assert_near, delta, delta_inputs, delta_tolerance  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F32 = ("SN", "dg", "dbeta", "dS0")


def on_gpu(s):
    return {i: None if x is None else x.cuda() for i, x in s.items()}


def forward(s, scale=None, **kw):
    return la.la_delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], S0=s["S0"], scale=scale, **kw)


def backward(s, scale=None, **kw):
    got = la.la_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], S0=s["S0"], dSN=s["dSN"], scale=scale, **kw)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got))


def check(got, want, dtype, names):
    for i in names:
        out = torch.float32 if i in F32 else dtype
        if got[i] is not None:
            assert got[i].dtype == out
            # dg and dbeta are sums of products of either sign (dbeta_t = sum_f dX_f E_f, relative errors r of its factors
            # independent: off by r (2 sum_f (dX_f E_f)^2)^(1/2)), so that a token's sum may cancel to far less than what
            # its error goes by.  That is as large as for the other tokens, whose mean size stands for it.
            assert_near(got[i], want[i], delta_tolerance(dtype, out, True), i, floor=1.0 if i in ("dg", "dbeta") else 0.02)


CASES = [
    # B, Hk, H, N, dk, dv, initial, resets
    (1, 1, 1, 1, 64, 64, True, ()),
    (2, 1, 2, 1, 128, 128, False, ()),
    (1, 2, 2, 63, 64, 64, True, ()),
    (1, 2, 2, 64, 128, 128, True, ()),
    (1, 2, 4, 65, 128, 64, False, (64,)),
    (2, 3, 3, 130, 64, 128, True, (0, 70)),
    (1, 1, 3, 200, 128, 128, True, (129,)),
    (1, 2, 2, 333, 64, 64, True, ()),
    (2, 1, 4, 77, 32, 64, True, (5,)),
    (1, 2, 2, 97, 64, 32, True, (31, 32)),
    (1, 2, 4, 150, 32, 32, False, ()),
    (1, 1, 1, 257, 32, 128, True, ()),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, dtype):
    B, Hk, H, N, dk, dv, initial, resets = case
    s = delta_inputs(1, B, Hk, H, N, dk, dv, TYPES[dtype], initial, resets)
    want = delta(s, dk ** -0.5, backward=False)
    o, SN = forward(on_gpu(s))
    check(dict(o=o, SN=SN), want, TYPES[dtype], ("o", "SN"))
    assert la.la_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, dtype):
    B, Hk, H, N, dk, dv, initial, resets = case
    s = delta_inputs(2, B, Hk, H, N, dk, dv, TYPES[dtype], initial, resets)
    want = delta(s, 0.3)
    check(backward(on_gpu(s), 0.3), want, TYPES[dtype], ("dq", "dk", "dv", "dg", "dbeta", "dS0"))
    assert la.la_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_is_deterministic_and_independent_of_what_ran_before(dtype):
    a, b = (on_gpu(delta_inputs(i, 2, 2, 4, 190, 128, 128, TYPES[dtype])) for i in (3, 4))
    first = backward(a)
    backward(b)
    again = backward(a)
    for i, x in first.items():
        assert torch.equal(x, again[i]), i


def test_gradients_against_differences():
    """fp32: the directional derivative of sum(o dout) + sum(SN dSN) by central differences of the float64 recurrence, along
    unit directions: with a step of 2^-10 off by 2^-20 / 6 of the third derivative, 1e-4 of the gradient's norm at most as long
    as that derivative is under 600 of them; the gradient itself is within 128 u."""
    s = delta_inputs(5, 1, 2, 4, 70, 32, 32, torch.float32)
    got = backward(on_gpu(s), 0.3)
    gen = torch.Generator().manual_seed(6)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("S0", "dS0")):
        d = torch.randn(s[name].shape, generator=gen, dtype=torch.float64)
        d /= d.norm()
        h = 2.0 ** -10

        def loss(step):
            r = delta({**s, name: s[name].double() + step * d}, 0.3, backward=False)
            return float((r["o"] * s["dout"].double()).sum() + (r["SN"] * s["dSN"].double()).sum())

        slope = (loss(h) - loss(-h)) / (2 * h)  # float64: off by h^2 of the third derivative
        mine = float((got[grad].cpu().double() * d).sum())
        size = float(got[grad].double().norm())
        assert abs(mine - slope) <= 1e-4 * size, (name, mine, slope)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,H,dk,dv", [(1, 1, 1, 64, 64), (3, 2, 4, 128, 128), (5, 1, 3, 32, 64), (2, 2, 2, 128, 32), (2, 4, 4, 64, 128)])
def test_step(B, Hk, H, dk, dv, dtype):
    t = TYPES[dtype]
    s = delta_inputs(7, B, Hk, H, 3, dk, dv, t)
    s["g"][:, 0, 1] = -math.inf
    want = delta(s, dk ** -0.5, backward=False)
    d = on_gpu(s)
    S = d["S0"].clone()
    for i in range(3):
        one = [d[n][:, :, i].contiguous() for n in ("q", "k", "v", "g", "beta")]
        o = la.la_delta_step(S, *one)
        assert_near(o[:, :, None], want["o"][:, :, i:i + 1], delta_tolerance(t, t, False), "o")
    assert_near(S, want["SN"], delta_tolerance(t, torch.float32, False), "S")


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 32)])
def test_prefill_then_steps_is_the_whole_sequence(dtype, d):
    t = TYPES[dtype]
    s = delta_inputs(8, 2, 2, 4, 140, d, d, t)
    want = delta(s, d ** -0.5, backward=False)
    g = on_gpu(s)
    head = {n: g[n][:, :, :137].contiguous() for n in ("q", "k", "v", "g", "beta")}
    o, S = la.la_delta_forward(**head, S0=g["S0"])
    assert_near(o, want["o"][:, :, :137], delta_tolerance(t, t, True), "prefill")
    for i in range(137, 140):
        o = la.la_delta_step(S, *[g[n][:, :, i].contiguous() for n in ("q", "k", "v", "g", "beta")])
        assert_near(o[:, :, None], want["o"][:, :, i:i + 1], delta_tolerance(t, t, True), "step")
    assert_near(S, want["SN"], delta_tolerance(t, torch.float32, True), "S")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens_and_padding_tokens(dtype):
    t = TYPES[dtype]
    s = on_gpu(delta_inputs(9, 1, 2, 2, 90, 64, 64, t))
    none = {n: s[n][:, :, :0].contiguous() for n in ("q", "k", "v", "g", "beta", "dout")}
    o, SN = forward({**none, "S0": s["S0"]})
    assert o.numel() == 0 and torch.equal(SN, s["S0"])
    assert torch.equal(backward({**none, "S0": s["S0"], "dSN": s["dSN"]})["dS0"], s["dSN"])
    _, SN = forward({**none, "S0": None})
    assert not SN.any()
    # tokens with beta = 0 and g = 0 leave the state as it is, whatever they hold
    short = {n: s[n][:, :, :70].contiguous() for n in ("q", "k", "v", "g", "beta")}
    padded = {n: s[n].clone() for n in ("q", "k", "v", "g", "beta")}
    padded["beta"][:, :, 70:], padded["g"][:, :, 70:] = 0.0, 0.0
    padded["v"][:, :, 70:] = 1e4
    a, b = forward({**short, "S0": s["S0"]}), forward({**padded, "S0": s["S0"]})
    tol = delta_tolerance(t, torch.float32, True)
    assert_near(b[1], a[1].cpu().double(), 2 * tol)
    assert_near(b[0][:, :, :70], a[0].cpu().double(), 2 * delta_tolerance(t, t, True))


def test_a_reset_is_a_new_sequence():
    s = on_gpu(delta_inputs(10, 1, 1, 2, 150, 64, 64, torch.bfloat16, True, (83,)))
    o, SN = forward(s)
    tail = {n: s[n][:, :, 83:].contiguous() for n in ("q", "k", "v", "g", "beta")}
    o2, SN2 = forward({**tail, "S0": None})
    assert_near(o[:, :, 83:], o2.cpu().double(), 2 * delta_tolerance(torch.bfloat16, torch.bfloat16, True))
    assert_near(SN, SN2.cpu().double(), 2 * delta_tolerance(torch.bfloat16, torch.float32, True))
    got = backward(s)
    head = {n: s[n][:, :, :83].contiguous() for n in ("q", "k", "v", "g", "beta", "dout")}
    alone = backward({**head, "S0": s["S0"], "dSN": None})  # nothing comes back across the reset
    assert not got["dg"][:, :, 83].any()
    assert_near(got["dS0"], alone["dS0"].cpu().double(), 2 * delta_tolerance(torch.bfloat16, torch.float32, True))


@pytest.mark.parametrize("dk, dv", [(64, 64), (128, 128), (32, 64), (128, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_heads_than_the_machine_takes_at_once(dtype, dk, dv):
    """Heads enough for other launches than a few take (96 and, in the backward, twice that)."""
    t = TYPES[dtype]
    s = delta_inputs(16, 2, 24, 48, 150, dk, dv, t, True, (77,))
    g, scale = on_gpu(s), dk ** -0.5
    o, SN = forward(g)
    check(dict(o=o, SN=SN, **backward(g)), delta(s, scale), t, ("o", "SN", "dq", "dk", "dv", "dg", "dbeta", "dS0"))
    assert la.la_get_device_status() == 0


@pytest.mark.parametrize("dk, dv", [(64, 64), (128, 128), (64, 128), (128, 64), (32, 64)])
def test_long_calls_of_some_heads(dk, dv):
    """Heads and chunks enough for preparation and scan side by side (48 heads of 16 chunks, the last one odd), in
    two graphs at once on inputs of their own, and with a head poisoned."""
    s = [on_gpu(delta_inputs(30 + i, 1, 24, 48, 1009, dk, dv, torch.bfloat16, True, (500,))) for i in range(2)]
    want = [forward(x) for x in s]
    exact = delta(s[0], dk ** -0.5, backward=False)
    check(dict(zip(("o", "SN"), want[0])), {n: x.cpu() for n, x in exact.items()}, torch.bfloat16, ("o", "SN"))
    streams = [torch.cuda.Stream() for _ in s]
    graphs, outs = [], []
    for x, st in zip(s, streams):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            outs.append(forward(x, stream=st))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, w))
    bad = {n: x.clone() for n, x in s[0].items()}
    bad["v"][0, 7, 900] = math.nan
    o, SN = forward(bad)
    others = [h for h in range(48) if h != 7]
    assert torch.equal(o[:, others], want[0][0][:, others]) and torch.equal(SN[:, others], want[0][1][:, others])
    assert torch.equal(o[:, 7, :896], want[0][0][:, 7, :896]) and not torch.isfinite(SN[:, 7]).all()
    assert la.la_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_poisoned_head_stays_alone(dtype):
    """NaN, infinities and wide open gates in one head: the others, and its own earlier tokens, are as without them."""
    t = TYPES[dtype]
    s = on_gpu(delta_inputs(17, 1, 2, 4, 200, 64, 64, t))
    o, SN = forward(s)
    grads = backward(s)
    for where, value in (("v", math.nan), ("v", math.inf), ("g", math.nan), ("g", 1e4), ("beta", math.nan), ("beta", math.inf)):
        bad = {n: x.clone() for n, x in s.items()}
        bad[where][0, 1, 130] = value
        o2, SN2 = forward(bad)
        got = backward(bad)
        others = [0, 2, 3]
        assert torch.equal(o2[:, others], o[:, others]) and torch.equal(SN2[:, others], SN[:, others])
        assert torch.equal(o2[:, 1, :128], o[:, 1, :128])
        assert not torch.isfinite(SN2[:, 1]).all() and not torch.isfinite(o2[:, 1, 130:]).all()
        for n in ("dv", "dg", "dbeta", "dS0"):
            assert torch.equal(got[n][:, others], grads[n][:, others]), (where, n)
        for n in ("dq", "dk"):
            assert torch.equal(got[n][:, 1], grads[n][:, 1]), (where, n)
    assert la.la_get_device_status() == 0


def test_two_graphs_and_an_eager_call_at_once():
    """Captured calls keep workspaces of their own: two graphs and eager calls of the same shapes on three streams."""
    t = torch.bfloat16
    data = [delta_inputs(20 + i, 2, 4, 8, 700, 64, 64, t) for i in range(3)]
    s = [on_gpu(x) for x in data]
    want = [(forward(x), backward(x)) for x in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, st in zip(s[:2], streams):
        with torch.cuda.stream(st):
            forward(x, stream=st), backward(x, stream=st)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            outs.append((forward(x, stream=st), backward(x, stream=st)))
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = forward(s[2], stream=streams[2]), backward(s[2], stream=streams[2])
    torch.cuda.synchronize()
    for (f, b), (wf, wb) in zip(outs + [eager], want):
        assert all(torch.equal(x, y) for x, y in zip(f, wf))
        assert all(torch.equal(b[n], wb[n]) for n in wb)
    assert la.la_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graphs_streams_and_given_outputs(dtype):
    """A captured forward, backward and step, replayed with other inputs in place, beside an eager call on another stream."""
    t = TYPES[dtype]
    a, b = (delta_inputs(i, 1, 2, 4, 100, 64, 64, t) for i in (11, 12))
    want = delta(b, 0.25)
    s = on_gpu(a)
    S = s["S0"].clone()
    one = [s[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward(s, 0.25), backward(s, 0.25)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, SN = forward(s, 0.25)
        grads = backward(s, 0.25)
        la.la_delta_step(S, *one, scale=0.25)
    for n, x in on_gpu(b).items():
        s[n].copy_(x)
    S.copy_(s["S0"])
    for x, n in zip(one, ("q", "k", "v", "g", "beta")):
        x.copy_(s[n][:, :, 0])
    other = on_gpu(delta_inputs(13, 1, 2, 4, 300, 64, 64, t))
    side.wait_stream(torch.cuda.current_stream())
    graph.replay()
    with torch.cuda.stream(side):
        forward(other, stream=side), backward(other, stream=side)
    torch.cuda.synchronize()
    check(dict(o=o, SN=SN, **grads), want, t, ("o", "SN", "dq", "dk", "dv", "dg", "dbeta", "dS0"))
    first = {n: b[n][:, :, :1] if n not in ("S0", "dSN") else b[n] for n in b}
    assert_near(S, delta(first, 0.25, backward=False)["SN"], delta_tolerance(t, torch.float32, True))
    # outputs given by the caller
    out = dict(o=torch.empty_like(o), SN=torch.empty_like(SN))
    r = forward(s, 0.25, **out)
    assert r[0] is out["o"] and r[1] is out["SN"] and torch.equal(r[0], o) and torch.equal(r[1], SN)


def test_a_layer_of_delta_rule_and_head_norm():
    """The two operators as a layer uses them: heads normalised per token, gated, channels last; forward and gradients
    against float64 autograd of the plain formulas."""
    B, H, N, d = 2, 3, 130, 64
    s = delta_inputs(14, B, H, H, N, d, d, torch.bfloat16, False)
    gen = torch.Generator().manual_seed(15)
    gate, dy = (torch.randn((B, N, H * d), generator=gen).bfloat16() for _ in range(2))
    w = 1 + 0.1 * torch.randn(H * d, generator=gen)
    g = on_gpu(s)
    o, _ = forward(g)
    y, mean, rstd = la.la_group_norm_forward(o, H, w=w.cuda(), gate=gate.cuda(), act="silu", per_token=True, heads_first=True,
                                             center=False)
    do, dgate, dw, _ = la.la_group_norm_backward(o, H, mean, rstd, dy.cuda(), w=w.cuda(), gate=gate.cuda(), act="silu",
                                                 per_token=True, heads_first=True, center=False)
    got = la.la_delta_backward(g["q"], g["k"], g["v"], g["g"], g["beta"], do)
    # the plain layer; the norm's gradient is handed on as float64
    want = delta(s, d ** -0.5, backward=False)["o"].clone().requires_grad_()
    h = want * (want.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    z = h.transpose(1, 2).reshape(B, N, H * d) * w.double()
    gd = gate.double().requires_grad_()
    out = z * gd * torch.sigmoid(gd)
    out.backward(dy.double())
    tol = delta_tolerance(torch.bfloat16, torch.bfloat16, True)
    assert_near(y.reshape(B, N, H, d).transpose(1, 2), out.detach().reshape(B, N, H, d).transpose(1, 2), 3 * tol, "y")
    assert_near(do, want.grad, 4 * tol, "do")
    s["dout"] = want.grad
    ref = delta(s, d ** -0.5)
    for i, x in zip(("dq", "dk", "dv"), got):
        assert_near(x, ref[i], 5 * tol, i)
    assert_near(dgate.reshape(B, N, H, d).transpose(1, 2), gd.grad.reshape(B, N, H, d).transpose(1, 2), 4 * tol, "dgate")


def correlated(seed, kind, B, Hk, H, N, d, dtype):
    """Keys that overwrite one another: 8 keys in turn, read back; a token repeated 16 times; keys near one direction; positive
    ones.  Writes are nearly whole (beta 0.7 to 1), gates nearly open."""
    s = delta_inputs(seed, B, Hk, H, N, d, d, torch.float32)
    gen = torch.Generator().manual_seed(seed + 1)
    if kind == "overwritten":
        few = torch.randn((B, Hk, 8, d), generator=gen)
        k = few[:, :, torch.arange(N) % 8]
        q = few[:, :, (torch.arange(N) * 5 + 3) % 8]
    elif kind == "repeated":
        k = s["k"][:, :, ::16].repeat_interleave(16, 2)[:, :, :N]
        q = k.roll(-3, 2)
    elif kind == "parallel":
        base = torch.randn((B, Hk, 1, d), generator=gen)
        k, q = (base + 0.1 * torch.randn((B, Hk, N, d), generator=gen) for _ in range(2))
    else:
        k, q = s["k"].abs(), s["q"].abs()
    s["k"], s["q"] = ((x / x.norm(dim=-1, keepdim=True)).to(dtype) for x in (k, q))
    s["v"], s["dout"] = s["v"].to(dtype), s["dout"].to(dtype)
    s["beta"] = 1 - 0.3 * torch.rand((B, H, N), generator=gen)
    s["g"] = -0.02 * torch.rand((B, H, N), generator=gen)
    return s


KINDS = ["overwritten", "repeated", "parallel", "positive"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_keys_that_overwrite_one_another(kind, d, dtype):
    """What is read back is the difference of what the state and the chunk's own writes answer, each as large as the old
    value.  Every operand is held to 2^-17 (fp32: u), so that terms some times as large as o leave o's own rounding what
    counts; the states, whose old content goes in the keys' directions, may be off by four times as much of their own size."""
    t = TYPES[dtype]
    s = correlated(40, kind, 2, 1, 2, 190, d, t)
    want = delta(s, d ** -0.5, backward=False)
    o, SN = forward(on_gpu(s))
    assert_near(o, want["o"], delta_tolerance(t, t, True), "o")
    assert_near(SN, want["SN"], 4 * delta_tolerance(t, torch.float32, True), "SN")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gate", [-0.9, -1.1, -4.0, -90.0])
def test_gates_that_close_within_a_chunk(gate, d, dtype):
    """A chunk's first writes are closed to exp(-57), exp(-70), less than fp32 holds by its end, and are read before that."""
    t = TYPES[dtype]
    s = delta_inputs(42, 1, 2, 2, 150, d, d, t)
    s["g"] = gate * (0.9 + 0.2 * torch.rand(s["g"].shape, generator=torch.Generator().manual_seed(1)))
    want = delta(s, 0.5)
    g = on_gpu(s)
    o, SN = forward(g, 0.5)
    check(dict(o=o, SN=SN, **backward(g, 0.5)), want, t, ("o", "SN", "dq", "dk", "dv", "dg", "dbeta", "dS0") if gate > -90 else ("o", "SN", "dq", "dk", "dv", "dbeta"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_gradients_of_keys_that_overwrite_one_another(kind, d, dtype):
    """dq is read from the same two terms as o, and dk from those of the gradients; what ends in fp32 as the states above."""
    t = TYPES[dtype]
    s = correlated(44, kind, 2, 1, 2, 190, d, t)
    want = delta(s, d ** -0.5)
    got = backward(on_gpu(s), d ** -0.5)
    for i in ("dq", "dk", "dv"):
        assert_near(got[i], want[i], delta_tolerance(t, t, True), i)
    for i in ("dg", "dbeta", "dS0"):
        assert_near(got[i], want[i], 4 * delta_tolerance(t, torch.float32, True), i, floor=0.02 if i == "dS0" else 1.0)


@pytest.mark.parametrize("H,dk,dv", [(0, 64, 64), (2, 0, 64), (2, 64, 0)])
def test_sizes_of_nothing_give_zeros(H, dk, dv):
    """No heads that read the keys, no key features, no value features: what is left of the outputs sums over nothing."""
    def full(*shape, dtype=torch.bfloat16):
        return torch.full(shape, 3.0, dtype=dtype, device="cuda")

    q, v, g = full(2, 2, 5, dk), full(2, H, 5, dv), full(2, H, 5, dtype=torch.float32)
    out = dict(dq=full(2, 2, 5, dk), dk=full(2, 2, 5, dk), dv=full(2, H, 5, dv), dg=full(2, H, 5, dtype=torch.float32),
               dbeta=full(2, H, 5, dtype=torch.float32))
    o, SN = la.la_delta_forward(q, q, v, g, g, scale=1.0, o=full(2, H, 5, dv))
    assert not o.any() and SN.numel() == 0
    la.la_delta_backward(q, q, v, g, g, v, scale=1.0, **out)
    assert not any(x.any() for x in out.values())
    o = la.la_delta_step(SN, q[:, :, 0].contiguous(), q[:, :, 0].contiguous(), v[:, :, 0].contiguous(), g[:, :, 0].contiguous(),
                         g[:, :, 0].contiguous(), scale=1.0, o=full(2, H, dv))
    assert not o.any()


def test_workspaces_of_growing_calls():
    """A stream keeps one buffer for its calls, at most a quarter larger than the largest of them needs (0.297 MB a head and
    chunk in the backward at d 128), and the buffers that it has outgrown are freed."""
    import gc
    def calls(chunks, stream):
        s = on_gpu(delta_inputs(50, 1, 4, 8, 2, 128, 128, torch.bfloat16, False))
        g = {n: None if x is None else x[:, :, :1].repeat(*((1, 1, 64 * chunks) + (1,) * (x.dim() - 3))).contiguous() for n, x in s.items()}
        torch.cuda.synchronize()
        first, again = backward(g, stream=stream), backward(g, stream=stream)
        torch.cuda.synchronize()
        assert all(x is None or torch.equal(x, again[n]) for n, x in first.items())

    stream = torch.cuda.Stream()
    calls(4, torch.cuda.default_stream())  # code that the steps below load, 100 MB of it PyTorch's, is not counted
    gc.collect(), torch.cuda.synchronize(), torch.cuda.empty_cache()
    before = torch.cuda.mem_get_info()[0]
    for chunks in (40, 85, 175, 360, 365, 370):
        calls(chunks, stream)
    gc.collect(), torch.cuda.synchronize(), torch.cuda.empty_cache()
    held = before - torch.cuda.mem_get_info()[0]
    assert held <= 1.25 * 8 * 370 * 0.297e6 + 64e6, held


@pytest.mark.parametrize("ticket", [0, 100, 767])
def test_a_lost_chunk_times_out_and_the_next_call_is_clean(ticket):
    """48 heads of 16 chunks, prepared and scanned in one launch: a chunk (ticket / 48 of head ticket % 48) that is prepared but
    never published makes its scan's wait run out, which the status word tells."""
    lib = la.load_library()
    s = on_gpu(delta_inputs(60, 1, 24, 48, 1009, 64, 64, torch.bfloat16))
    want = forward(s)
    torch.cuda.synchronize()
    assert la.la_get_device_status() == 0
    try:
        lib.la_test_set_wait_limit_ns(50_000_000)
        got = forward(s)  # a short limit alone does not fire
        torch.cuda.synchronize()
        assert la.la_get_device_status() == 0 and all(torch.equal(x, y) for x, y in zip(got, want))
        lib.la_test_set_wait_limit_ns(2_000_000)
        lib.la_test_drop_publication(ticket)
        forward(s)
        torch.cuda.synchronize()
        assert la.la_get_device_status() == 5 and la.la_get_device_status() == 0
    finally:
        lib.la_test_drop_publication(-1)
        lib.la_test_set_wait_limit_ns(0)
    got = forward(s)
    torch.cuda.synchronize()
    assert la.la_get_device_status() == 0 and all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_that_overwrite_one_key(dtype):
    """beta = 1 and one unit key, again and again: what was stored is replaced, and read back with the key itself."""
    t = TYPES[dtype]
    s = delta_inputs(61, 2, 1, 2, 6, 64, 64, t)
    s["k"] = s["k"][:, :, :1].expand(-1, -1, 6, -1).contiguous()
    s["q"], s["beta"], s["g"] = s["k"].clone(), torch.ones_like(s["beta"]), torch.zeros_like(s["g"])
    want = delta(s, 1.0, backward=False)
    g = on_gpu(s)
    S = g["S0"].clone()
    for i in range(6):
        o = la.la_delta_step(S, *[g[n][:, :, i].contiguous() for n in ("q", "k", "v", "g", "beta")], scale=1.0)
        assert_near(o[:, :, None], want["o"][:, :, i:i + 1], delta_tolerance(t, t, False), "o")
    assert_near(S, want["SN"], delta_tolerance(t, torch.float32, False), "S")
    o, SN = forward(g, 1.0)
    assert_near(o, want["o"], delta_tolerance(t, t, True), "o")
    assert_near(SN, want["SN"], 4 * delta_tolerance(t, torch.float32, True), "SN")
