"""What the Python binding refuses before it calls the library: every call here has host tensors
or none that is read, and must be refused with the message of its own check."""
import pytest
import torch

from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    D.load_library()


def refused(match):
    return pytest.raises(D.Ds4spError, match=match)


@pytest.mark.parametrize("fmt,rows,dims", [(1, 3, 576), (2, 1, 64), (3, 5, 576), (5, 1, 576), (5, 65, 64)])
def test_quantizer_refuses_an_output_that_is_too_small(fmt, rows, dims):
    need = D.ds4sp_cache_bytes(fmt, dims, rows)
    x = torch.zeros(rows, dims, dtype=torch.float16)
    for size in (0, 16, need - 1):
        with refused(f"need {need}"):
            D.ds4sp_quantize_kv(x, fmt, out=torch.zeros(size, dtype=torch.uint8))
    with refused("CUDA device"):                      # large enough: the next check's refusal
        D.ds4sp_quantize_kv(x, fmt, out=torch.zeros(need, dtype=torch.uint8))


BIG = 1 << 32


def test_sizes_and_rows_beyond_32_bits_are_refused():
    """The library counts rows in 32 bits; a larger count would reach it cut to its low bits."""
    cache, x = torch.zeros(65 * 576, dtype=torch.uint8), torch.zeros(1, 576)
    for row0 in (BIG, BIG + 3, 1 << 31, -1, -BIG):
        with refused("^row0:"):
            D.ds4sp_cache_write(cache, 5, x, row0)
        with refused("^row0:"):
            D.ds4sp_cache_read(cache, 5, 576, row0=row0, n=1)
    for n in (BIG + 1, -1):
        with refused("^n:"):
            D.ds4sp_cache_read(cache, 5, 576, n=n)
    with refused(f"^x: {BIG + 1}"):
        D.ds4sp_cache_write(cache, 5, x.expand(BIG + 1, 576), 0)
    for shape in ((BIG + 1, 1, 64), (1, BIG + 1, 64), (1 << 31, 1, 64)):
        with refused(f"^x: {max(shape)}"):
            D.ds4sp_rope(torch.zeros(1, 1, 64).expand(shape), D.make_rope(64))


def test_rope_refuses_a_tensor_it_would_cut_off_from_its_gradient():
    x, plain, rope = torch.zeros(1, 1, 64, requires_grad=True), torch.zeros(1, 1, 64), D.make_rope(64)
    with refused("^x: requires a gradient"):
        D.ds4sp_rope(x, rope)
    with refused("^x: requires a gradient"):
        D.ds4sp_rope(2 * x, rope, out=plain)
    with refused("^out: requires a gradient"):
        D.ds4sp_rope(plain, rope, out=x)
    for call in (lambda: D.ds4sp_rope(x.detach(), rope), lambda: torch.no_grad()(D.ds4sp_rope)(x, rope)):
        with refused("CUDA device"):                  # the next check's refusal
            call()
