"""ds4sp_cache_write and ds4sp_cache_read against the float64 oracle.

Without a rotation everything is decided exactly: the scale of a kv_format 5 block is a
power of two, so its codes are one rounding of an exact quotient; the block formats of 32
values are ds4sp_quantize_kv's bytes; a value read back is code * scale, exact in fp32,
rounded once. Those tests compare bits. With a rotation, a stored value is off by the
rotation's fp32 error (2^-21 of the pair's |a| + |b|, see test_gpu_rope) and half a step of
its format, or a whole step where that error crosses a rounding border.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache_ops as O
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


def rows_of(n, dims, seed, dtype=torch.float16, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, dims, generator=g) * torch.exp(spread * torch.randn(n, 1, generator=g))).to(dtype).cuda()


def new_cache(fmt, rows, dims=576):
    return torch.full((D.ds4sp_cache_bytes(fmt, dims, rows),), 0xA5, dtype=torch.uint8, device="cuda")


def read(cache, dims=576, fmt=5, dtype=torch.float32, **kw):
    return D.ds4sp_cache_read(cache, fmt, dims, dtype=dtype, **kw)


# ------------------------------------------------------------------ e4m3 with a scale per block

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", [16, 80, 576, 592, 1024])
@pytest.mark.parametrize("n", [1, 63, 64, 65, 200])
def test_e4m3_bytes(dtype, dims, n):
    x = rows_of(n, dims, n + dims, dtype)
    cache = new_cache(5, n, dims)
    D.ds4sp_cache_write(cache, 5, x, 0)
    ref = O.BlockCache(n, dims)
    ref.write(0, x.double().cpu().numpy())
    want = O.stored_bytes(ref.codes, ref.exp).reshape(-1, 65, dims)
    got = cache.cpu().numpy().reshape(-1, 65, dims)
    for b in range(len(want)):
        k = min(64, n - 64 * b)
        assert np.array_equal(got[b, :k], want[b, :k]) and np.array_equal(got[b, 64], want[b, 64])
        assert (got[b, k:64] == 0xA5).all()              # rows behind the last are left as they were
    assert np.array_equal(read(cache, dims, row0=0, n=n).double().cpu().numpy(), ref.read(np.arange(n)))


def test_e4m3_special_values():
    """Ties, the smallest values, a block of zeros, infinities and NaN, values past the
    largest scale, and fp16's largest."""
    x = torch.zeros(64 * 5, 32)
    x[0, :8] = torch.tensor([448, -448, 17.0, 19.0, 21.0, -2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10])
    x[1, :4] = torch.tensor([1.0625, 1.1875, 1.3125, 465.0 / 1.1])
    x[128, 0], x[128, 1], x[129, 2], x[130, 3] = float("inf"), 3.0, float("nan"), -float("inf")
    x[192, 0], x[192, 1] = 1e30, -5.0
    x[256, 0], x[256, 1] = 65504.0, 2.0 ** -24
    cache = new_cache(5, 320, 32)
    D.ds4sp_cache_write(cache, 5, x.cuda(), 0)
    ref = O.BlockCache(320, 32)
    ref.write(0, x.double().numpy())
    got = read(cache, 32).double().cpu().numpy()
    assert np.array_equal(got, ref.read(np.arange(320)), equal_nan=True)
    assert got[128, 0] == 3.5 and got[130, 3] == -3.5 and np.isnan(got[129, 2])    # 448 * 2^-7
    assert got[192, 0] == 448 * 2.0 ** 40 and ref.exp[1] == -40 and ref.exp[3] == 40


@pytest.mark.parametrize("pieces", [[1] * 70, [5, 59, 1, 64, 3], [40, 100, 7], [64, 64, 1], [63, 2, 130]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_e4m3_appends(pieces, dtype):
    """Rows written in pieces, scales growing and shrinking between them, against the oracle
    doing the same; then a piece of it written again (a rejected draft's rows)."""
    n = sum(pieces)
    x = rows_of(n, 576, n, dtype, spread=2.0)
    cache, ref, at = new_cache(5, n), O.BlockCache(n, 576), 0
    for k in pieces:
        D.ds4sp_cache_write(cache, 5, x[at:at + k], at)
        ref.write(at, x[at:at + k].double().cpu().numpy())
        at += k
        assert np.array_equal(read(cache, row0=0, n=at).double().cpu().numpy(), ref.read(np.arange(at))), at
    again = rows_of(3, 576, 9, dtype, spread=2.0)
    D.ds4sp_cache_write(cache, 5, again, n - 3)
    ref.write(n - 3, again.double().cpu().numpy())
    assert np.array_equal(read(cache, row0=0, n=n).double().cpu().numpy(), ref.read(np.arange(n)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dims,offset", [(64, 512), (34, 9), (2, 575 - 1), (256, 0)])
def test_e4m3_with_rotation(dtype, layout, dims, offset):
    """Blocks whose largest value is not rotated, so that their scales are exact."""
    n, row0 = 131, 70
    x = rows_of(n, 576, 3, dtype, spread=0.3)
    x[:, 300] = 100.0 if not offset <= 300 < offset + dims else x[:, 300]
    cache = new_cache(5, 256)
    D.ds4sp_cache_write(cache, 5, rows_of(70, 576, 4), 0)
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(5)).int().cuda()
    D.ds4sp_cache_write(cache, 5, x, row0, rope=D.make_rope(dims, offset, layout, scaling=1, factor=3.0), positions=pos)
    x64 = x.double().cpu().numpy()
    y = O.rope(x64[:, None], pos.cpu().numpy(), dims, offset, layout, scaling=1, factor=3.0)[:, 0]
    got = read(cache, row0=row0, n=n).double().cpu().numpy()
    top = np.abs(x64).max()
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 1e-30))) - 3)       # e4m3's spacing at y
    least = 2.0 ** (O.scale_exponent(np.array([2 * top])) - 9)
    tol = np.maximum(step, least) * 0.5 + 2 * top * 2.0 ** -21
    crossed = np.maximum(step, least) * 1.0 + 2 * top * 2.0 ** -21
    err = np.abs(got - y)
    assert (err <= crossed).all() and (err > tol).mean() < 1e-3


def test_e4m3_strided_and_unaligned_rows():
    wide = rows_of(100, 601, 6)
    for first in (0, 1, 8, 25):
        x = wide[:, first:first + 576]
        cache, plain = new_cache(5, 100), new_cache(5, 100)
        rope = D.make_rope(64, offset=512)
        D.ds4sp_cache_write(cache, 5, x, 0, rope=rope, pos0=7, pos_step=4)
        D.ds4sp_cache_write(plain, 5, x.contiguous(), 0, rope=rope, pos0=7, pos_step=4)
        assert torch.equal(cache, plain)
    one = rows_of(1, 576, 7).expand(70, 576)                  # a broadcast row
    cache = new_cache(5, 70)
    D.ds4sp_cache_write(cache, 5, one, 0)
    assert torch.equal(read(cache, row0=0, n=1).expand(70, 576), read(cache, row0=0, n=70))


# ------------------------------------------------------------------ the other formats

@pytest.mark.parametrize("fmt", [1, 2, 3])
@pytest.mark.parametrize("dims", [512, 576])
def test_block_formats_write_the_quantizer_bytes(fmt, dims):
    x = rows_of(301, dims, fmt)
    x[5] = 0
    x[6, :32] = torch.tensor([4.0, -4.0] * 16)                # equal extremes
    want = D.ds4sp_quantize_kv(x, fmt)
    cache = new_cache(fmt, 310, dims)
    D.ds4sp_cache_write(cache, fmt, x[:200], 3)
    D.ds4sp_cache_write(cache, fmt, x[200:], 203)
    got = cache.view(310, -1)
    assert torch.equal(got[3:304], want)
    assert (got[:3] == 0xA5).all() and (got[304:] == 0xA5).all()


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
@pytest.mark.parametrize("src", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_block_formats_read_back(fmt, src, dtype):
    x = rows_of(77, 576, 11, src, spread=0.5)
    cache = new_cache(fmt, 77)
    D.ds4sp_cache_write(cache, fmt, x, 0)
    if fmt == 0:
        key = val = x.half().double().cpu().numpy()
    else:
        key, val = oracle.kv_values(x.float().cpu().numpy(), fmt)
        key, val = np.asarray(key, np.float64), np.asarray(val, np.float64)
    for part, want in ((0, key), (1, val[:, :512])):
        got = read(cache, fmt=fmt, dtype=dtype, part=part)
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(dtype)), part


def test_fp16_rows_are_the_attention_cache():
    x = rows_of(33, 576, 12, torch.bfloat16)
    kv = torch.zeros(40, 576, dtype=torch.float16, device="cuda")
    rope = D.make_rope(64, offset=512)
    D.ds4sp_cache_write(kv, 0, x, 5, rope=rope, pos0=5)
    x32 = x.float()
    turned = D.ds4sp_rope(x32[:, None, 512:], D.make_rope(64), pos0=5)[:, 0]
    assert torch.equal(kv[5:38], torch.cat((x32[:, :512], turned), 1).half())
    assert (kv[:5] == 0).all() and (kv[38:] == 0).all()


# ------------------------------------------------------------------ reading by index

@pytest.mark.parametrize("fmt", [0, 1, 2, 3, 5])
def test_read_by_index(fmt):
    x = rows_of(200, 576, 13)
    cache = new_cache(fmt, 200)
    D.ds4sp_cache_write(cache, fmt, x, 0)
    held = 256 if fmt == 5 else 200
    rows = torch.tensor([199, 0, 0, 64, 63, -1, 128, 199, held, 1 << 30, -(1 << 31), 65]).int().cuda()
    all_rows = read(cache, fmt=fmt, row0=0, n=200)
    for part in (0, 1):
        got = read(cache, fmt=fmt, rows=rows, part=part)
        ok = (rows >= 0) & (rows < 200)
        want = read(cache, fmt=fmt, row0=0, n=200, part=part)[rows.clamp(0, 199).long()]
        want[~ok] = 0
        assert torch.equal(got, want)
    assert all_rows.shape == (200, 576)


@pytest.mark.parametrize("dtype", DTYPES)
def test_read_into_strided_rows(dtype):
    x = rows_of(90, 576, 14)
    cache = new_cache(5, 90)
    D.ds4sp_cache_write(cache, 5, x, 0)
    want = read(cache, dtype=dtype, row0=3, n=80)
    for first, width in ((0, 576), (1, 577), (8, 600), (3, 601)):
        out = torch.full((80, width), -1.0, dtype=dtype, device="cuda")
        view = out[:, first:first + 576]
        assert D.ds4sp_cache_read(cache, 5, 576, row0=3, n=80, out=view) is view
        assert torch.equal(view, want)
        assert (out[:, :first] == -1).all() and (out[:, first + 576:] == -1).all()


def test_long_cache_offsets():
    """Rows whose bytes lie past 2^31: a 4 GB cache of 7.4 million rows."""
    rows = 7_400_000
    cache = torch.empty(D.ds4sp_cache_bytes(5, 576, rows), dtype=torch.uint8, device="cuda")
    x = rows_of(100, 576, 15)
    D.ds4sp_cache_write(cache, 5, x, 7_399_872)                # a block's start
    idx = torch.arange(7_399_872, 7_399_972).int().cuda()
    got = read(cache, rows=idx)
    small = new_cache(5, 100)
    D.ds4sp_cache_write(small, 5, x, 0)
    assert torch.equal(got, read(small, row0=0, n=100))


def test_captured_append_on_another_stream():
    x = rows_of(5, 576, 16)
    cache = new_cache(5, 128)
    D.ds4sp_cache_write(cache, 5, rows_of(60, 576, 17), 0)
    start = cache.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    D.ds4sp_cache_write(cache, 5, x, 60, stream=s)
    out = torch.empty(65, 576, device="cuda")
    D.ds4sp_cache_read(cache, 5, 576, row0=0, n=65, out=out, stream=s)
    s.synchronize()
    want = out.clone()
    cache.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.ds4sp_cache_write(cache, 5, x, 60)
        D.ds4sp_cache_read(cache, 5, 576, row0=0, n=65, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x.mul_(100.0)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want) and torch.equal(out, read(cache, row0=0, n=65))


@pytest.mark.parametrize("rows,dims", [(0, 576), (1, 576), (63, 64), (64, 576), (200, 576), (129, 2048)])
def test_quantizer_writes_the_scaled_cache(rows, dims):
    """ds4sp_quantize_kv in kv_format 5 is a write of fp16 rows from row 0 on: the same bytes."""
    x = rows_of(rows, dims, 21)
    want = torch.zeros(D.ds4sp_cache_bytes(5, dims, rows), dtype=torch.uint8, device="cuda")
    if rows:
        D.ds4sp_cache_write(want, 5, x, 0)
    out = torch.zeros(max(want.numel(), 16), dtype=torch.uint8, device="cuda")
    assert D.ds4sp_quantize_kv(x, 5, out=out) is out
    assert torch.equal(out[: want.numel()], want)
    fresh = D.ds4sp_quantize_kv(x, 5)
    assert fresh.dim() == 1 and fresh.numel() >= want.numel()
    if rows:
        assert torch.equal(read(fresh, dims, n=rows), read(want, dims, n=rows))
