"""Attention over a kv_format 5 cache whose blocks' scales differ widely: one attended row (a
sink) in a block whose scale is 2^r times the others'.

A row's weight is p s, p its probability and s its block's scale, and the terms hold it to
TOL of itself (test_gpu_attn_scaled's module text derives it) but to no less than FLOOR of the
token's largest weight: half of the last term's smallest spacing, 2^-19 (three terms) or 2^-28
(five), where the largest weight is 1/8 at least. So where the sink is 0, an element's error relative to sum p |v| is at
most TOL + FLOOR * R, R the largest p s over the smallest: the probabilities' bits that an uneven
cache costs. This is the bound that the header states; the tests hold it, and that error is
as small as the format's own where R is near 1.
"""
import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D
from test_gpu_attn_scaled import TOL, Case, scales_of

pytestmark = pytest.mark.gpu
FLOOR = {0: 2.0 ** -16, 1: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


@pytest.mark.parametrize("pv_mode", [0, 1])
@pytest.mark.parametrize("n", [40, 3])
@pytest.mark.parametrize("r", [0, 4, 8, 10, 12, 14])
def test_one_row_of_large_scale_beside_small_ones(r, n, pv_mode):
    c = Case(n, 2000, 256, 128, seed=20 + r, spread=0.0, pv_mode=pv_mode)
    c.q[..., :256] = 0                                  # the sink's logit is 0
    c.cmp_x[:64] = 0
    c.cmp_x[0, :256] = 3.5 * 2.0 ** r                   # the others reach 3.5 to 5: scale 2^-7 or 2^-6
    c.topk[:, 1:] = torch.from_numpy(64 + np.sort(np.stack([np.random.default_rng(i).choice(400, 255, replace=False)
                                                            for i in range(n)]), 1)).int().cuda()
    c.topk[:, 0] = 0
    D.ds4sp_cache_write(c.cmp, 5, c.cmp_x, 0)
    out = c.run()
    c.check(out)                                        # with the bound's two parts, row by row
    raw, cmp_ = c.stored()
    sizes = [scales_of(x, len(y)) for x, y in ((c.raw, c.raw_x), (c.cmp, c.cmp_x))]
    top, got = c.topk.cpu().numpy(), out.double().cpu().numpy()
    for i in range(n):
        q = c.q[i].double().cpu().numpy()
        rows, size = (O.attended(a, b, top, c.t0, i, c.n_swa) for a, b in ((raw, cmp_), sizes))
        z = q @ rows.T / 24.0
        p = np.exp(z - z.max(1, keepdims=True))
        ratio = (p * size).max(1) / (p * size).min(1)
        err = np.abs(got[i] - O.attention_rows(q, rows))[:, 256:]
        mass = O.attention_rows(q, rows, absolute=True)[:, 256:]
        bound = TOL[pv_mode] + FLOOR[pv_mode] * ratio[:, None]
        assert (err <= bound * mass).all()
