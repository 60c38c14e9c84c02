"""The fp32-staged attention over a kv_format 5 cache (pv_mode 1) is as near to 64 bits as an
elementary fp32 form on the same stored rows: scores, softmax and product in torch, fp32
throughout. Rows of uneven size, whose logits spread wide; norms over 256 tokens' outputs, so that
the comparison is of the two forms' errors and not of single roundings.
"""
import math

import pytest
import torch

from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D
from test_gpu_attn_scaled import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


def elementary(q, rows, seen):
    z = torch.matmul(q, rows.transpose(1, 2)) / math.sqrt(576)
    z = torch.where(seen[:, None], z, torch.full((), -math.inf, device="cuda", dtype=z.dtype))
    p = torch.exp(z - z.amax(-1, keepdim=True))
    return torch.matmul(p / p.sum(-1, keepdim=True), rows[..., :512])


@pytest.mark.parametrize("k,n_swa", [(128, 128), (512, 128), (300, 20), (0, 250)])
def test_no_further_from_64_bits_than_an_elementary_fp32_form(k, n_swa):
    n, t0 = 256, 3000
    c = Case(n, t0, k, n_swa, seed=30 + k)
    for x, cache in ((c.raw_x, c.raw), (c.cmp_x, c.cmp)):
        x[:, 512:] *= 4                                  # rotary keys of larger spread
        D.ds4sp_cache_write(cache, 5, x, 0)
    out = c.run().double()
    at = t0 + torch.arange(n, device="cuda")[:, None] - torch.arange(n_swa - 1, -1, -1, device="cuda")
    rows = D.ds4sp_cache_read(c.raw, 5, 576, row0=0, n=c.T, dtype=torch.float32)[at.clamp(min=0)]
    seen = at >= 0
    if k:
        cmp_ = D.ds4sp_cache_read(c.cmp, 5, 576, row0=0, n=c.T // 4, dtype=torch.float32)
        rows, seen = torch.cat((cmp_[c.topk.clamp(min=0).long()], rows), 1), torch.cat((c.topk >= 0, seen), 1)
    want = elementary(c.q.double(), rows.double(), seen)
    plain = elementary(c.q.float(), rows, seen).double()
    assert (out - want).norm() <= (plain - want).norm()


@pytest.mark.parametrize("pv_mode", [0, 1])
@pytest.mark.parametrize("n", [60, 4])
def test_a_token_with_one_row_returns_it(n, pv_mode):
    """One attended row (a window of one, nothing selected): the stored values themselves, where the
    logit leaves the weight's logarithm negative (scales of 2^-7 to 2^-5, logits below 2)."""
    c = Case(n, 0 if n == 4 else 1000, 0, 1, seed=40 + n, spread=0.0, pv_mode=pv_mode)
    c.q.mul_(0.25)
    rows = D.ds4sp_cache_read(c.raw, 5, 576, row0=c.t0, n=n, dtype=torch.float32)[:, :512]
    assert torch.equal(c.run(), rows[:, None].expand(n, 16, 512))
