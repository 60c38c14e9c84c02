"""How exact the rotation is: cos and sin come from 64 bits and are rounded once, in ds4sp_rope
and in the rows that ds4sp_cache_write turns.

Bounds. The kernel's angle is off by at most 2^-35 of a turn (a 64-bit fraction of a turn cut to
34 bits), 2^-32 radians, and by the frequency's own rounding, |position| * (f * 2^-50 + 2^-61); the
oracle's product position * f is rounded to 2^-53 of itself. The Taylor sums add 2^-37. So m cos and m
sin are off by half a step, 2^-24 of the value, and m * ANGLE = m * (2^-31 + |position| f * 2^-49).
A turned value a c - b s then has the two factors' roundings, one product's and the sum's: at most
3 * 2^-24 of m (|a| + |b|); a stored kv_format 5 value is turned in 64 bits and rounded once, so it
is the code of a value within m ANGLE (|a| + |b|) of the exact one.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D

pytestmark = pytest.mark.gpu

SCALINGS = [dict(), dict(scaling=1, factor=3.7), dict(scaling=2, factor=8.0),
            dict(scaling=3, factor=32.0, orig_len=4096), dict(scaling=1, factor=0.013)]


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


def angle_error(positions, f):
    return 2.0 ** -31 + np.abs(np.asarray(positions, np.float64))[:, None] * f * 2.0 ** -49


@pytest.mark.parametrize("freq", SCALINGS)
@pytest.mark.parametrize("layout", [0, 1])
def test_cos_and_sin_are_rounded_once(freq, layout):
    """The unit vectors (1, 0) turned: m cos and m sin themselves."""
    n, dims = 40000, 64
    pos = torch.randint(-(1 << 17), 1 << 20, (n,), generator=torch.Generator().manual_seed(1)).int()
    x = torch.zeros(n, 1, dims, device="cuda")
    first = slice(0, dims, 2) if layout == 0 else slice(0, dims // 2)
    second = slice(1, dims, 2) if layout == 0 else slice(dims // 2, dims)
    x[..., first] = 1.0
    y = D.ds4sp_rope(x, D.make_rope(dims, layout=layout, **freq), positions=pos.cuda())[:, 0].double().cpu().numpy()
    f, m = O.rope_frequencies(dims, **freq)
    t = pos.double().numpy()[:, None] * f
    for got, want in ((y[:, first], m * np.cos(t)), (y[:, second], m * np.sin(t))):
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -24 + m * angle_error(pos.numpy(), f)).all()


@pytest.mark.parametrize("below", [2.0 ** -25, 2.0 ** -27, 2.0 ** -30, 2.0 ** -31, 0.0, -2.0 ** -28])
@pytest.mark.parametrize("turn", [0.25, 0.5, 0.75, 1.0, 0.125, 0.375, 0.625])
def test_angles_at_the_quadrants_borders(turn, below):
    """One position whose angle lies a little below a border (or on it, or above)."""
    f = 2 * math.pi * turn * (1 - below)
    x = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]]], device="cuda").flip(0)       # position 0, then 1
    y = D.ds4sp_rope(x, D.make_rope(2, scaling=1, factor=1.0 / f)).double().cpu().numpy()
    assert np.array_equal(y[0, 0], [0.0, 1.0])
    want = np.array([math.cos(f), math.sin(f)])
    assert (np.abs(y[1, 0] - want) <= np.abs(want) * 2.0 ** -24 + 2.0 ** -31 + f * 2.0 ** -49).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dims,offset,layout", [(64, 512, 0), (64, 512, 1), (128, 448, 0), (256, 64, 1), (34, 9, 0), (8, 568, 0)])
def test_stored_codes_are_the_exact_values_codes(dtype, dims, offset, layout):
    """kv_format 5: a code is the exact turned value's, rounded once, in each form of the kernel
    (a part held and turned once, turned twice, unaligned)."""
    n = 6000
    freq = dict(scaling=3, factor=32.0, orig_len=4096)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(n, 576, generator=g).to(dtype)
    x[:, 0] = 16.0                                     # every block's largest: scale 2^-4
    cache = torch.zeros(D.ds4sp_cache_bytes(5, 576, n), dtype=torch.uint8, device="cuda")
    D.ds4sp_cache_write(cache, 5, x.cuda(), 0, rope=D.make_rope(dims, offset, layout, **freq), pos0=50000, pos_step=4)
    got = D.ds4sp_cache_read(cache, 5, 576, row0=0, n=n, dtype=torch.float32).double().cpu().numpy()
    pos = 50000 + 4 * np.arange(n)
    x64 = x.double().numpy()
    y = O.rope(x64[:, None], pos, dims, offset, layout, **freq)[:, 0]
    f, m = O.rope_frequencies(dims, **freq)
    part, pair_off = np.abs(x64[:, offset:offset + dims]), angle_error(pos, f)
    off = np.zeros_like(y)
    if layout == 0:
        off[:, offset:offset + dims] = np.repeat(m * (part[:, 0::2] + part[:, 1::2]) * pair_off, 2, axis=1)
    else:
        off[:, offset:offset + dims] = np.tile(m * (part[:, :dims // 2] + part[:, dims // 2:]) * pair_off, 2)
    scale = 2.0 ** O.scale_exponent(np.array([16.0]))
    low, high = (O.e4m3_round((y + s * off) / scale) * scale for s in (-1, 1))
    assert ((got >= low) & (got <= high)).all()
    assert (got != O.e4m3_round(y / scale) * scale).sum() <= 1


@pytest.mark.parametrize("dims,offset", [(64, 512), (128, 448), (34, 9)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_values_in_a_rotated_part(dtype, dims, offset):
    """Infinities saturate at 448 scales, NaNs stay, neither moves the block's scale nor another
    pair; values whose turned form passes fp32's largest saturate at the largest scale."""
    x = torch.zeros(130, 576)
    x[:, 0] = 16.0
    x[3, offset], x[5, offset + 2], x[6, offset + 4] = float("inf"), float("nan"), -float("inf")
    x[128, offset] = x[128, offset + 1] = 3.3e38
    cache = torch.zeros(D.ds4sp_cache_bytes(5, 576, 130), dtype=torch.uint8, device="cuda")
    D.ds4sp_cache_write(cache, 5, x.to(dtype).cuda(), 0, rope=D.make_rope(dims, offset), pos0=1)
    got = D.ds4sp_cache_read(cache, 5, 576, row0=0, n=130, dtype=torch.float32).double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        y = O.rope(x.to(dtype).double().numpy()[:, None], 1 + np.arange(130), dims, offset)[:, 0]
    first = y[:128]
    assert np.array_equal(np.isnan(got[:128]), np.isnan(first))
    at = np.isinf(first)
    assert at.sum() >= 3 and np.array_equal(got[:128][at], np.sign(first[at]) * 448 * 2.0 ** -4)
    rest = np.isfinite(first)
    assert np.array_equal(got[:128][rest], O.e4m3_round(first[rest] * 2.0 ** 4) * 2.0 ** -4)
    assert np.array_equal(got[128, offset:offset + 2], np.sign(y[128, offset:offset + 2]) * 448 * 2.0 ** 40)
