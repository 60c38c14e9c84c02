"""Rotary positions and cache rows, on the CPU: the oracle's pins, and the refusals of
ds4sp_rope, ds4sp_cache_write and ds4sp_cache_read, which all come before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D


@pytest.fixture(scope="module")
def lib():
    B.build()
    return D.load_library()


# ------------------------------------------------------------------ oracle pins

def test_e4m3_round_is_torch_rounding():
    x = np.concatenate([np.linspace(-460, 460, 4001), O.e4m3_table()[:127], np.ldexp(1.0, np.arange(-14, 9)),
                        (O.e4m3_table()[:126] + O.e4m3_table()[1:127]) / 2])       # every tie
    want = torch.from_numpy(x.clip(-448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_round(x), want)


def test_e4m3_table_is_torch_decoding():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_table(), v, equal_nan=True)


@pytest.mark.parametrize("top,e", [(0.0, -40), (448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.76, -7),
                                   (65504.0, 8), (2.0 ** -24, -32), (1e30, 40), (1e-30, -40), (np.inf, -40)])
def test_scale_exponent(top, e):
    assert O.scale_exponent(np.array([0.0, -top])) == e


def test_append_keeps_the_larger_scale_and_rounds_again():
    c = O.BlockCache(128, 16)
    c.write(0, np.full((3, 16), 0.3))
    assert c.exp[0] == O.scale_exponent(np.array([0.3]))
    small = c.read([0])[0, 0]
    c.write(3, np.full((1, 16), 400.0))
    assert c.exp[0] == 0 and c.read([0])[0, 0] == O.e4m3_round(np.array(small))
    c.write(4, np.full((2, 16), 1e-3))
    assert c.exp[0] == 0 and c.read([3])[0, 0] == O.e4m3_round(np.array(400.0))


def test_rope_against_complex_turns_and_transpose_undoes_it():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((5, 2, 12)), np.array([0, 1, 7, 100000, 3])
    y = O.rope(x, pos, 8, offset=3, layout=1, scaling=1, factor=2.0)
    f = np.array([10000.0 ** (-2 * i / 8) / 2 for i in range(4)])
    z = (x[..., 3:7] + 1j * x[..., 7:11]) * np.exp(1j * pos[:, None, None] * f)
    assert np.allclose(y[..., 3:7], z.real, atol=1e-12) and np.allclose(y[..., 7:11], z.imag, atol=1e-12)
    assert np.array_equal(y[..., :3], x[..., :3]) and np.array_equal(y[..., 11:], x[..., 11:])
    back = O.rope(y, pos, 8, offset=3, layout=1, scaling=1, factor=2.0, transpose=True)
    assert np.allclose(back, x, atol=1e-12)


def test_yarn_keeps_fast_pairs_and_divides_slow_ones():
    f, m = O.rope_frequencies(64, scaling=3, factor=32.0, orig_len=4096)
    plain, _ = O.rope_frequencies(64)
    assert f[0] == plain[0] and math.isclose(f[-1], plain[-1] / 32) and math.isclose(m, 0.1 * math.log(32) + 1)
    assert np.all(np.diff(f) < 0)


# ------------------------------------------------------------------ sizes and refusals

def test_cache_bytes(lib):
    assert D.ds4sp_cache_bytes(0, 576, 10) == 11520
    assert D.ds4sp_cache_bytes(3, 576, 10) == 9120
    assert D.ds4sp_cache_bytes(5, 576, 1) == D.ds4sp_cache_bytes(5, 576, 64) == 65 * 576
    assert D.ds4sp_cache_bytes(5, 576, 65) == 130 * 576
    assert D.ds4sp_cache_bytes(5, 576, (1 << 31) - 1) == (1 << 25) * 65 * 576
    for fmt, dims, rows in ((4, 576, 1), (6, 576, 1), (5, 24, 1), (1, 48, 1), (0, 12, 1), (5, 8192, 1),
                            (5, 576, -1), (0, 576, 1 << 31)):
        assert D.ds4sp_cache_bytes(fmt, dims, rows) == 0, (fmt, dims, rows)


P = 0x10000      # a 16-byte aligned address that is never read: every call below is refused


def _rope(lib, cfg, x=P, dtype=0, n=4, heads=2, head=64, xs=(128, 64), out=2 * P, os_=(128, 64), pos=None):
    ref = ctypes.byref(cfg) if cfg is not None else None
    return lib.ds4sp_rope(ref, x, dtype, n, heads, head, xs[0], xs[1], out, os_[0], os_[1], pos, 0, 1, 0, None)


@pytest.mark.parametrize("kw", [dict(dims=0), dict(dims=3), dict(dims=258), dict(dims=64, offset=-2), dict(dims=64, offset=2),
                                dict(dims=64, layout=2), dict(dims=64, scaling=4), dict(dims=64, base=1.0),
                                dict(dims=64, base=float("nan")), dict(dims=64, scaling=1, factor=0.0),
                                dict(dims=64, scaling=2, factor=float("inf")), dict(dims=2, scaling=2, factor=2.0),
                                dict(dims=64, scaling=3, factor=2.0), dict(dims=64, mscale=float("nan"))])
def test_rope_refuses_configurations(lib, kw):
    assert _rope(lib, D.make_rope(**kw)) == D.ERR_INVALID_ARG
    assert lib.ds4sp_last_error()


@pytest.mark.parametrize("kw", [dict(scaling=1, factor=1e-309), dict(scaling=2, factor=1e-318),
                                dict(scaling=3, factor=1e-309, orig_len=4096), dict(mscale=1e300)])
def test_rope_refuses_frequencies_and_magnitudes_out_of_range(lib, kw):
    assert _rope(lib, D.make_rope(64, **kw)) == D.ERR_INVALID_ARG
    assert lib.ds4sp_last_error()


@pytest.mark.parametrize("kw", [dict(heads=(1 << 30) + 1), dict(head=(1 << 20) + 1, os_=(1 << 22, 1 << 21))])
def test_rope_refuses_sizes(lib, kw):
    assert _rope(lib, D.make_rope(64), **kw) == D.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(x=None), dict(out=None), dict(x=P + 1), dict(dtype=2, out=P + 2), dict(dtype=3),
                                dict(n=-1), dict(heads=0), dict(head=0), dict(xs=(-1, 64)), dict(os_=(63, 64)),
                                dict(os_=(128, 63)), dict(pos=P + 2)])
def test_rope_refuses_arguments(lib, kw):
    assert _rope(lib, D.make_rope(64), **kw) == D.ERR_INVALID_ARG
    assert lib.ds4sp_last_error()


def test_rope_of_nothing_is_no_launch(lib):
    assert _rope(lib, D.make_rope(64), n=0, x=None, out=None) == D.OK
    assert _rope(lib, None) == D.ERR_INVALID_ARG


def _write(lib, cache=P, fmt=5, dims=576, rows=128, row0=0, n=4, x=2 * P, dtype=0, ld=576, rope=None, pos=None):
    return lib.ds4sp_cache_write(cache, fmt, dims, rows, row0, n, x, dtype, ld,
                                 ctypes.byref(rope) if rope else None, pos, 0, 1, None)


def _read(lib, cache=P, fmt=5, dims=576, rows=128, idx=None, row0=0, n=4, part=0, out=2 * P, dtype=0, ld=576):
    return lib.ds4sp_cache_read(cache, fmt, dims, rows, idx, row0, n, part, out, dtype, ld, None)


@pytest.mark.parametrize("kw", [dict(cache=None), dict(cache=P + 8), dict(fmt=4), dict(fmt=-1), dict(dims=568),
                                dict(fmt=3, dims=256), dict(rows=3), dict(row0=-1), dict(row0=125), dict(n=-1),
                                dict(row0=(1 << 31) - 1), dict(x=None), dict(x=P + 1), dict(dtype=2, x=P + 2),
                                dict(dtype=9), dict(ld=-1), dict(pos=P + 1), dict(rope=D.make_rope(64, offset=520)),
                                dict(rope=D.make_rope(63))])
def test_cache_write_refuses(lib, kw):
    assert _write(lib, **kw) == D.ERR_INVALID_ARG
    assert lib.ds4sp_last_error()


@pytest.mark.parametrize("kw", [dict(cache=None), dict(cache=P + 4), dict(fmt=4), dict(dims=560 + 8), dict(rows=3),
                                dict(rows=-1), dict(row0=-1), dict(row0=125), dict(n=-1), dict(part=2), dict(part=-1),
                                dict(fmt=1, dims=256, part=1), dict(out=None), dict(out=P + 1), dict(dtype=3),
                                dict(ld=575), dict(idx=P + 2)])
def test_cache_read_refuses(lib, kw):
    assert _read(lib, **kw) == D.ERR_INVALID_ARG
    assert lib.ds4sp_last_error()


def test_cache_calls_of_no_rows_are_no_launch(lib):
    assert _write(lib, n=0, x=None, cache=None) == D.OK
    assert _read(lib, n=0, out=None, cache=None) == D.OK
    assert _write(lib, n=0, rope=D.make_rope(64, offset=520)) == D.ERR_INVALID_ARG


def test_binding_refuses_host_tensors(lib):
    with pytest.raises(D.Ds4spError):
        D.ds4sp_rope(torch.zeros(1, 1, 64), D.make_rope(64))
    with pytest.raises(D.Ds4spError):
        D.ds4sp_cache_write(torch.zeros(65 * 576, dtype=torch.uint8), 5, torch.zeros(1, 576), 0)
    with pytest.raises(D.Ds4spError):
        D.ds4sp_cache_read(torch.zeros(65 * 576, dtype=torch.uint8), 5, 576)


@pytest.mark.parametrize("kw", [dict(exp_mode=1), dict(exp_mode=1, pv_mode=1), dict(attn_kernel=1),
                                dict(attn_kernel=1, pv_mode=1)])
def test_create_refuses_what_a_scaled_cache_has_not(lib, kw):
    cfg = D.make_config(16, 64, 64, 32, 1024, kv_format=5, **kw)
    out = ctypes.c_void_p(123)
    assert lib.ds4sp_create(ctypes.byref(cfg), ctypes.byref(out)) == D.ERR_UNSUPPORTED
    assert out.value is None and lib.ds4sp_last_error()


@pytest.mark.parametrize("rows,ok", [(0, False), (1, True), (64, True), (65, True)])
def test_binding_asks_for_whole_blocks(rows, ok):
    """70 tokens (two blocks) and their 17 compressed rows (one), against a cache of `rows` rows."""
    h = D.Handle(0, D.make_config(16, 64, 64, 32, 1024, kv_format=5))
    two = torch.zeros(D.ds4sp_cache_bytes(5, 576, 70), dtype=torch.uint8)
    some = torch.zeros(D.ds4sp_cache_bytes(5, 576, rows), dtype=torch.uint8)
    plain = torch.zeros(70, 576, dtype=torch.uint8)
    D._check_blocks(h, two, some if ok else None, 70)
    refused = [(plain, two), (plain.half(), two)] + ([] if ok else [(two, some)]) + ([] if rows > 64 else [(some, two)])
    for raw, cmp in refused:
        with pytest.raises(D.Ds4spError):
            D._check_blocks(h, raw, cmp, 70)
