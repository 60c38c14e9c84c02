"""ds4sp_rope against the float64 oracle.

Tolerance of a turned value m (a c - b s): the angle is exact but for the frequency's own
rounding, |position| * 2^-55 turns; sincospif is within 2 ulp (2^-23 for values up to 1);
m, m c, and the product and sum in fp32 are four roundings of at most 2^-24 each on
m (|a| + |b|). Together at most 6 * 2^-24 < 2^-21 of m (|a| + |b|), plus the position's
2 pi 2^-55; then half a step of the output's type (or of its smallest values' spacing).
"""
import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


def assert_turned(got, x, positions, dims, offset=0, layout=0, transpose=False, mscale=0.0, **freq):
    x64 = x.double().cpu().numpy()
    want = O.rope(x64, positions, dims, offset, layout, transpose, mscale, **freq)
    _, m = O.rope_frequencies(dims, **freq)
    m = mscale if mscale > 0 else m
    size = np.zeros_like(want)
    part = np.abs(x64[..., offset:offset + dims])
    if layout == 0:
        pair = part[..., 0::2] + part[..., 1::2]
        size[..., offset:offset + dims] = np.repeat(pair, 2, axis=-1)
    else:
        pair = part[..., :dims // 2] + part[..., dims // 2:]
        size[..., offset:offset + dims] = np.concatenate([pair, pair], -1)
    far = np.abs(np.asarray(positions, np.float64))[:, None, None] * 2 * np.pi * 2.0 ** -55
    info = torch.finfo(x.dtype)
    tol = m * size * (2.0 ** -21 + far) + np.abs(want) * info.eps / 2 + info.smallest_normal * info.eps / 2
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"{(err - tol).max()} over, {err.max()} off"
    rest = np.ones(x.shape[-1], bool)
    rest[offset:offset + dims] = False
    assert torch.equal(got[..., torch.from_numpy(rest)], x[..., torch.from_numpy(rest)])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("n,heads,head,dims,offset", [
    (1, 1, 64, 64, 0), (5, 16, 64, 64, 0), (3, 3, 7, 2, 5), (130, 16, 576, 64, 512), (33, 5, 100, 34, 9),
    (17, 64, 128, 64, 64), (2, 1, 256, 256, 0), (700, 64, 128, 64, 0), (1031, 7, 24, 20, 2)])
def test_rope_matches_oracle(dtype, layout, n, heads, head, dims, offset):
    g = torch.Generator().manual_seed(n + dims)
    x = torch.randn(n, heads, head, generator=g).to(dtype).cuda()
    y = D.ds4sp_rope(x, D.make_rope(dims, offset, layout), pos0=11, pos_step=4)
    assert_turned(y, x, 11 + 4 * np.arange(n), dims, offset, layout)


SCALINGS = [dict(), dict(scaling=1, factor=4.0), dict(scaling=1, factor=0.01), dict(scaling=2, factor=8.0),
            dict(scaling=3, factor=32.0, orig_len=4096), dict(scaling=3, factor=0.5, orig_len=131072),
            dict(scaling=3, factor=16.0, orig_len=1, base=500000.0)]


@pytest.mark.parametrize("freq", SCALINGS)
@pytest.mark.parametrize("transpose", [False, True])
def test_rope_scalings_far_positions_and_transpose(freq, transpose):
    pos = np.array([0, 1, 122879, (1 << 20) + 7, (1 << 31) - 1, -5, -(1 << 31)], np.int64)
    x = torch.randn(len(pos), 4, 64, generator=torch.Generator().manual_seed(2)).cuda()
    y = D.ds4sp_rope(x, D.make_rope(64, **freq), positions=torch.from_numpy(pos).int().cuda(), transpose=transpose)
    # numpy's own argument t = position * f is rounded to 2^-53 of up to 2^31 radians (2^38 at
    # a factor of 0.01): leave the far positions to the pairs that stay below 2^24 turns
    f, _ = O.rope_frequencies(64, **freq)
    for row, p in enumerate(pos):
        slow = np.abs(p) * f < 2.0 ** 24
        keep = np.repeat(slow, 2)
        want = O.rope(x[row:row + 1].double().cpu().numpy(), [p], 64, transpose=transpose, **freq)[..., keep]
        tol = (x[row].abs().max().item() * 2 * 4 * 2.0 ** -21 + abs(p) * 2.0 ** -50) + np.abs(want) * 2.0 ** -24
        assert (np.abs(y[row:row + 1].double().cpu().numpy()[..., keep] - want) <= tol).all(), (p, freq)


def test_rope_mscale():
    x = torch.randn(9, 2, 32, generator=torch.Generator().manual_seed(3)).cuda()
    y = D.ds4sp_rope(x, D.make_rope(32, scaling=3, factor=8.0, orig_len=100, mscale=0.75))
    assert_turned(y, x, np.arange(9), 32, mscale=0.75, scaling=3, factor=8.0, orig_len=100)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_rope_strides_into_a_wider_head_and_in_place(dtype, shift):
    """Queries read from a projection of 192 values a head and written beside the absorbed
    part; shift 1 and 2 leave the rows unaligned. Neighbours keep their values."""
    g = torch.Generator().manual_seed(4)
    proj = torch.randn(37, 16, 192 + shift, generator=g).to(dtype).cuda()
    q = torch.randn(37, 16, 576 + shift, generator=g).to(dtype).cuda()
    before = q.clone()
    x, out = proj[..., 128 + shift:], q[..., 512 + shift:]
    for layout in (0, 1):
        assert D.ds4sp_rope(x, D.make_rope(64, layout=layout), out=out, pos0=100) is out
        assert_turned(out, x, 100 + np.arange(37), 64, layout=layout)
        assert torch.equal(q[..., :512 + shift], before[..., :512 + shift])
        alone = D.ds4sp_rope(x, D.make_rope(64, layout=layout), pos0=100)
        inp = proj.clone()
        D.ds4sp_rope(inp[..., 128 + shift:], D.make_rope(64, layout=layout), out=inp[..., 128 + shift:], pos0=100)
        assert torch.equal(inp[..., 128 + shift:], alone) and torch.equal(inp[..., :128 + shift], proj[..., :128 + shift])


def test_rope_heads_outside_tokens_and_broadcast_source():
    """[heads, tokens] storage (token stride below the head stride), and one row turned for
    every head (head stride 0)."""
    x = torch.randn(5, 40, 64, generator=torch.Generator().manual_seed(5)).cuda().transpose(0, 1)
    out = torch.empty(5, 40, 64, device="cuda").transpose(0, 1)
    D.ds4sp_rope(x, D.make_rope(64), out=out)
    assert_turned(out, x, np.arange(40), 64)
    row = torch.randn(40, 1, 64, generator=torch.Generator().manual_seed(6)).cuda().expand(40, 5, 64)
    y = D.ds4sp_rope(row, D.make_rope(64))
    assert y.is_contiguous() and torch.equal(y[:, 0], y[:, 4])
    assert_turned(y, row, np.arange(40), 64)


def test_rope_gradient_is_the_transposed_rotation():
    """d(w . rope(x))/dx = ropeT(w): against central differences of the kernel in fp32.
    The map is linear, so the difference quotient is exact but for the outputs' rounding:
    each of 16 terms is off by at most 2^-21 of |x| + h, over 2 h."""
    rope = D.make_rope(16, offset=3, layout=1, scaling=3, factor=4.0, orig_len=64)
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(6, 2, 24, generator=g).cuda(), torch.randn(6, 2, 24, generator=g).cuda()
    grad = D.ds4sp_rope(w, rope, pos0=9, transpose=True)
    h = 0.5
    for d in range(24):
        e = torch.zeros_like(x)
        e[..., d] = h
        up, down = (D.ds4sp_rope(x + s * e, rope, pos0=9) for s in (1, -1))
        num = ((up - down).double() * w.double()).sum(-1) / (2 * h)
        tol = 24 * 2 * 2.0 ** -21 * 1.2 * (x.abs().max() + h) * w.abs().max() / h
        assert (num - grad[..., d].double()).abs().max() <= tol


def test_rope_special_values_stay_in_their_pair():
    x = torch.zeros(1, 1, 8, device="cuda")
    x[..., 0], x[..., 5] = float("inf"), float("nan")
    y = D.ds4sp_rope(x, D.make_rope(8), pos0=3)
    assert not torch.isfinite(y[0, 0, 0:2]).any() and torch.isnan(y[0, 0, 4:6]).all()
    assert torch.equal(y[0, 0, 2:4], x[0, 0, 2:4]) and torch.equal(y[0, 0, 6:], x[0, 0, 6:])


def test_rope_captured_on_another_stream():
    x = torch.randn(20, 16, 64, generator=torch.Generator().manual_seed(8)).half().cuda()
    rope, out = D.make_rope(64), torch.empty_like(x)
    want = D.ds4sp_rope(x, rope, pos0=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    D.ds4sp_rope(x, rope, out=out, pos0=5, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.ds4sp_rope(x, rope, out=out, pos0=5)
    x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).half())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, D.ds4sp_rope(x, rope, pos0=5))
