"""Rotary positions on the GPU against their float64 form (tests/hybrid_ref.py)."""
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


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="ramp", factor=16.0, original=4096, amplitude=1.2772588722239782)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot", [
    (1, 1, 1, 1, 32, 32), (3, 5, 1, 7, 64, 48), (2, 8, 2, 33, 128, 128), (1, 3, 3, 257, 64, 2), (2, 12, 4, 65, 128, 32),
    (1, 17, 17, 19, 8, 6), (2, 2, 1, 40, 256, 256), (1, 2, 2, 5, 64, 0), (1, 4, 1, 30, 96, 24)])
def test_forward_and_backward(dtype, layout, B, Hq, Hk, N, d, rot):
    """Widths and parts of the head that take every vector size, positions of packed
    sequences and far ones, each scaling, and the gradient."""
    q, k = ref.draw(1, (B, Hq, N, d), T[dtype]), ref.draw(2, (B, Hk, N, d), T[dtype])
    gen = torch.Generator().manual_seed(N)
    pos = torch.randint(-3, 200000, (B, N), generator=gen, dtype=torch.int32)
    for options in SCALINGS:
        got = la().la_rotary_forward(q.cuda(), k.cuda(), positions=pos.cuda(), rot=rot, layout=layout, **options)
        back = la().la_rotary_backward(q.cuda(), k.cuda(), positions=pos.cuda(), rot=rot, layout=layout, **options)
        for x, y, z in zip((q, k), got, back):
            ref.assert_within(y, *ref.rotary(x, pos, rot, layout, **options), (options, "forward"))
            ref.assert_within(z, *ref.rotary(x, pos, rot, layout, inverse=True, **options), (options, "backward"))


def test_offset_one_tensor_and_in_place():
    """Positions offset + n with a large offset, q alone, q and k in place, one token as [B, H, d]."""
    q, k = ref.draw(3, (2, 4, 50, 64), torch.bfloat16), ref.draw(4, (2, 2, 50, 64), torch.bfloat16)
    off = 3_000_000_000
    pos = (torch.arange(50, dtype=torch.float64) + off).expand(2, 50)
    want, bound = ref.rotary(q, pos, 64)
    only = la().la_rotary_forward(q.cuda(), offset=off)
    assert isinstance(only, torch.Tensor)
    ref.assert_within(only, want, bound)
    qc, kc = q.cuda(), k.cuda()
    oq, ok = la().la_rotary_forward(qc, kc, oq=qc, ok=kc, offset=off)
    assert oq is qc and ok is kc
    assert torch.equal(qc, only)
    ref.assert_within(kc, *ref.rotary(k, pos, 64))
    p1 = torch.tensor([5, 70000], dtype=torch.int32)
    one = la().la_rotary_forward(q[:, :, 0].contiguous().cuda(), positions=p1.cuda())
    ref.assert_within(one, *(t[:, :, 0] for t in ref.rotary(q[:, :, :1], p1[:, None], 64)))


def test_far_positions_turn_exactly():
    """The angle of position p + P is that of p plus P's: reduced exactly at the far end of the range."""
    x = torch.zeros((1, 1, 4, 8))
    x[..., :4] = 1.0
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 0]], dtype=torch.int32)
    got = la().la_rotary_forward(x.cuda(), positions=pos.cuda(), base=10000.0)
    ref.assert_within(got, *ref.rotary(x, pos, 8))


def test_neighbours_stay_untouched():
    """Outputs inside a larger buffer leave what is around them, and non-finite features stay with their pair."""
    q = ref.draw(5, (1, 2, 9, 64), torch.bfloat16)
    q[0, 0, 3, 7] = float("inf")
    q[0, 1, 4, 60] = float("nan")
    buf = torch.full((q.numel() + 512,), 99.0, dtype=torch.bfloat16, device="cuda")
    o = buf[256:256 + q.numel()].view(q.shape)
    la().la_rotary_forward(q.cuda(), oq=o, rot=32)
    assert bool((buf[:256] == 99).all()) and bool((buf[-256:] == 99).all())
    bad = ~torch.isfinite(o.cpu())
    assert {tuple(i) for i in bad.nonzero().tolist()} == {(0, 0, 3, 7), (0, 0, 3, 23), (0, 1, 4, 60)}


def test_empty():
    for shape in ((0, 2, 3, 8), (2, 0, 3, 8), (2, 2, 0, 8)):
        assert la().la_rotary_forward(torch.empty(shape, device="cuda")).shape == shape


def test_many_rows():
    """More entries, and more heads, than a grid's second dimension holds."""
    q = ref.draw(7, (1, 70000, 1, 8), torch.bfloat16)
    ref.assert_within(la().la_rotary_forward(q.cuda(), offset=77), *ref.rotary(q, torch.full((1, 1), 77.0), 8))
    q = ref.draw(6, (70000, 2, 1, 8), torch.bfloat16)
    pos = torch.arange(70000, dtype=torch.int32)[:, None]
    ref.assert_within(la().la_rotary_forward(q.cuda(), positions=pos.cuda()), *ref.rotary(q, pos, 8))


@pytest.mark.parametrize("base", [34, 10000])
@pytest.mark.parametrize("offset", [0, 2 ** 31 - 4, 2 ** 40])
def test_frequencies_of_wide_heads(base, offset):
    """128 pairs at far positions against 60-digit angles.  A frequency is a product of at most 7 powers of the
    base: 7 (2^-52 + 2^-53), the exponents' rounding ln(base) 2^-53 and 3 2^-53 on the way to turns are below
    2^-48 of the angle; the fraction of a turn ends at 2^-64, 2 pi 2^-64 for each position."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    N, rot = 3, 256
    ang = torch.empty((N, rot // 2), dtype=torch.float64)
    full = torch.empty_like(ang)
    for i in range(rot // 2):
        f = (-Decimal(base).ln() * 2 * i / rot).exp()
        for n in range(N):
            full[n, i], ang[n, i] = float((offset + n) * f), float((offset + n) * f % (2 * pi))
    x = torch.zeros((1, 1, N, rot))
    x[..., :rot // 2] = 1.0
    got = la().la_rotary_forward(x.cuda(), offset=offset, base=float(base))[0, 0]
    off = 7 * ref.U + full * 2.0 ** -48 + (torch.arange(N)[:, None] + offset) * 6.3 * 2.0 ** -64
    ref.assert_within(got[:, :rot // 2], ang.cos(), off, "cosines")
    ref.assert_within(got[:, rot // 2:], ang.sin(), off, "sines")
