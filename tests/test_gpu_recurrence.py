"""The gated recurrence on the GPU against its float64 form (tests/hybrid_ref.py)."""
import pytest

import hybrid_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
T = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_kernelized_attention_gb300 import build
    build.build()


def la():
    import causal_kernelized_attention_gb300 as m
    return m


def gates(seed, shape, closed=0.02):
    gen = torch.Generator().manual_seed(seed)
    a = torch.sigmoid(2 + 2 * torch.randn(shape, generator=gen))
    return a * (torch.rand(shape, generator=gen) > closed)


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


SHAPES = [(1, 1, 1), (2, 1, 4), (1, 7, 33), (3, 255, 32), (2, 256, 36), (2, 257, 40), (1, 513, 5), (1, 1000, 128),
          (2, 4099, 12), (1, 9000, 3), (5, 64, 1000), (1, 3, 4096)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("B,N,D", SHAPES)
def test_forward_backward(dtype, initial, B, N, D):
    """One token to many tiles and cluster steps, whole vectors and odd widths, with and without a
    first state (and its gradient)."""
    t = T[dtype]
    x, a, dh = ref.draw(1, (B, N, D), t), gates(2, (B, N, D)), ref.draw(3, (B, N, D), t)
    h0, dhN = (ref.draw(4, (B, D), torch.float32), ref.draw(5, (B, D), torch.float32)) if initial else (None, None)
    want, bound = ref.recurrence(a, x, h0)
    h, hN = la().la_recurrence_forward(*cu(x, a), h0=cu(h0)[0])
    ref.assert_within(h, want, bound * (1 + ref.half(t)) + ref.half(t) * want.abs(), "h")
    ref.assert_within(hN, want[:, -1], bound[:, -1], "hN")
    saved = want.to(t)
    got = la().la_recurrence_backward(*cu(a, saved, dh), h0=cu(h0)[0], dhN=cu(dhN)[0])
    parts = ref.recurrence_backward(a, saved, dh, h0, dhN)
    (g, e), (da, eda), (d0, e0) = parts
    ref.assert_within(got[0], g, e * (1 + ref.half(t)) + ref.half(t) * g.abs(), "dx")
    ref.assert_within(got[1], da, eda, "dalpha")
    if initial:
        ref.assert_within(got[2], d0, e0, "dh0")
    else:
        assert got[2] is None


def test_gradient_against_differences():
    """The backward pass against central differences of the float64 recurrence."""
    B, N, D = 2, 9, 6
    a, x, h0 = gates(1, (B, N, D), 0.0).double(), ref.draw(2, (B, N, D), torch.float64), ref.draw(3, (B, D), torch.float64)
    w, wN = ref.draw(4, (B, N, D), torch.float64), ref.draw(5, (B, D), torch.float64)

    def loss(a, x, h0):
        h = ref.recurrence(a, x, h0)[0]
        return float((h * w).sum() + (h[:, -1] * wN).sum())

    h = ref.recurrence(a, x, h0)[0].float()
    dx, da, d0 = la().la_recurrence_backward(*cu(a.float(), h, w.float()), h0=h0.float().cuda(), dhN=wN.float().cuda())
    step = 1e-5
    for i, (arr, grad) in enumerate(((a, da), (x, dx), (h0, d0))):
        for at in (0, 7, arr.numel() - 1):
            vals = []
            for s in (step, -step):
                moved = [t.clone() for t in (a, x, h0)]
                moved[i].view(-1)[at] += s
                vals.append(loss(*moved))
            # fp32 inputs: relative 1e-5 of sums of about N terms of size 3
            assert abs((vals[0] - vals[1]) / (2 * step) - float(grad.view(-1)[at])) < 1e-4


def test_long_few_channels():
    """A long sequence of few channels goes over many cluster steps; decays that forget nothing keep
    every token."""
    B, N, D = 1, 70000, 8
    x, a = ref.draw(1, (B, N, D), torch.float32), torch.ones((B, N, D))
    a[:, 35001] = 0.0
    h, hN = la().la_recurrence_forward(*cu(x, a))
    want = x.double().cumsum(1)
    want[:, 35001:] = x.double()[:, 35001:].cumsum(1)
    m = x.double().abs().cumsum(1)
    n = torch.arange(1, N + 1, dtype=torch.float64)[None, :, None]
    ref.assert_within(h, want, 2 * ref.U * (n + 32) * m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 333), (128, 4096)])
def test_steps_continue_the_forward(dtype, B, D):
    """Steps from the forward's last state give the forward's outputs within its bounds; so does a
    forward continued from hN."""
    t = T[dtype]
    N = 20
    x, a = ref.draw(1, (B, N, D), t).cuda(), gates(2, (B, N, D)).cuda()
    h, hN = la().la_recurrence_forward(x, a)
    P = 12
    h1, state = la().la_recurrence_forward(x[:, :P].contiguous(), a[:, :P].contiguous())
    h2, end = la().la_recurrence_forward(x[:, P:].clone(memory_format=torch.contiguous_format),
                                             a[:, P:].clone(memory_format=torch.contiguous_format), h0=state)
    assert torch.equal(h[:, :P], h1)
    want, bound = ref.recurrence(a.cpu(), x.cpu(), None)
    ref.assert_within(h2, want[:, P:], (bound * (1 + ref.half(t)) + ref.half(t) * want.abs())[:, P:])
    ref.assert_within(end, want[:, -1], bound[:, -1])
    for i in range(P, N):
        o = la().la_recurrence_step(state, x[:, i].clone(), a[:, i].clone())
        assert torch.equal(o, state.to(t))
        ref.assert_within(o, want[:, i], (bound * (1 + ref.half(t)) + ref.half(t) * want.abs())[:, i])


def test_empty_and_edges():
    """N = 0 hands the state through; nothing is written around the outputs."""
    h0 = ref.draw(1, (2, 8), torch.float32).cuda()
    e = torch.empty((2, 0, 8), device="cuda")
    assert torch.equal(la().la_recurrence_forward(e, e, h0=h0)[1], h0)
    assert torch.equal(la().la_recurrence_backward(e, e, e, h0=h0, dhN=h0)[2], h0)
    assert not la().la_recurrence_forward(e, e)[1].any()
    assert la().la_recurrence_forward(torch.empty((0, 3, 8), device="cuda"), torch.empty((0, 3, 8), device="cuda"))[0].numel() == 0
    B, N, D = 2, 300, 36
    n = B * N * D
    buf = torch.full((n + 512,), 99.0, dtype=torch.bfloat16, device="cuda")
    dal = torch.full((n + 512,), 99.0, device="cuda")
    x, a = ref.draw(2, (B, N, D), torch.bfloat16).cuda(), gates(3, (B, N, D)).cuda()
    la().la_recurrence_forward(x, a, h=buf[256:256 + n].view(B, N, D))
    assert bool((buf[:256] == 99).all()) and bool((buf[-256:] == 99).all())
    la().la_recurrence_backward(a, x, x, dx=buf[256:256 + n].view(B, N, D), dalpha=dal[256:256 + n].view(B, N, D))
    for b in (buf, dal):
        assert bool((b[:256] == 99).all()) and bool((b[-256:] == 99).all())


def test_nonfinite_stays_in_its_channel():
    B, N, D = 1, 700, 64
    x, a = ref.draw(1, (B, N, D), torch.float32), gates(2, (B, N, D), 0.0)
    x[0, 100, 5] = float("nan")
    h, _ = la().la_recurrence_forward(*cu(x, a))
    bad = torch.isnan(h.cpu())
    assert bool(bad[0, 100:, 5].all()) and int(bad.sum()) == N - 100


def test_streams_and_graphs():
    """Captured and replayed on new data, and on a side stream."""
    B, N, D = 2, 1500, 64
    x, a = ref.draw(1, (B, N, D), torch.bfloat16).cuda(), gates(2, (B, N, D)).cuda()
    h, hN = torch.empty_like(x), torch.empty((B, D), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        la().la_recurrence_forward(x, a, h=h, hN=hN)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la().la_recurrence_forward(x, a, h=h, hN=hN)
    x.copy_(ref.draw(9, (B, N, D), torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    want, _ = la().la_recurrence_forward(x, a)
    assert torch.equal(h, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D", [(1, 4096, 64), (1, 4097, 17), (3, 5001, 66), (2, 6000, 130), (9, 4480, 8)])
def test_segments(dtype, B, N, D):
    """Long sequences of few channels, split over the machine in segments: whole tiles and not, with first
    and last states."""
    test_forward_backward(dtype, True, B, N, D)


def test_segments_in_graphs_on_two_streams():
    """Two captured graphs replayed at once on new data, and eager calls on one stream between them."""
    B, N, D = 1, 20000, 64
    make = lambda s: [ref.draw(s, (B, N, D), torch.bfloat16).cuda(), gates(s + 1, (B, N, D)).cuda(),  # noqa: E731
                      ref.draw(s + 2, (B, N, D), torch.bfloat16).cuda()]
    call = lambda x, a, dh: (*la().la_recurrence_forward(x, a),  # noqa: E731
                             *la().la_recurrence_backward(a, x, dh, dhN=None)[:2])
    sets, graphs, outs = [make(10), make(20)], [], []
    for s in sets:
        call(*s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(*s))
        graphs.append(g)
    for s, n in zip(sets, (make(30), make(40))):
        for a, b in zip(s, n):
            a.copy_(b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = [call(*s) for s in sets]
    torch.cuda.synchronize()
    for got, want in zip(outs, eager):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert la().la_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("B,N,D", [
    (2, 3900, 64), (2, 3899, 65), (1, 3001, 2048), (1, 9003, 1280), (1, 2900, 1281), (1, 1500, 3848)])
def test_whole_sequences_over_cluster_steps(dtype, initial, B, N, D):
    """Clusters of CTAs that take a sequence in three steps and more, by TMA and by plain loads: fewer tiles
    than segments want (64, 65 channels), or channels enough to fill half of the machine (the others;
    9003 tokens pass 9 steps)."""
    test_forward_backward(dtype, initial, B, N, D)


@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("B,N,D", [(1, 2000, 2560), (1, 2001, 2600), (1, 1100, 4096), (2, 1001, 2568), (3, 777, 4096)])
def test_many_channels_turn_the_ring(initial, B, N, D):
    """Full-width training in bf16: the backward's three-stage ring of tiles goes round several times, in
    clusters of two CTAs (one entry) and of one."""
    test_forward_backward("bf16", initial, B, N, D)
