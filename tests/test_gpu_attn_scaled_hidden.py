"""Attention over a kv_format 5 cache where a token's first rows are all hidden: by a top-k
list of -1 (what the explicit-mask form writes for a token whose mask leaves nothing), by the
mask itself, or by entries outside the cache.

The softmax's reference must come from the first rows that are attended: a fixed one would
lose the weights of rows whose logits or scales are small, and keep their sums. So the rows
here are small (0.05: scales of 2^-11) and their logits lie around -15. Tolerances are those
of test_gpu_attn_scaled, whose conditions hold: the queries are multiples of 2^-6 (and one
value of at most 7,200), which their three terms hold exactly, and |q| |k| < 2,200 (logits of
-90: below fp32's smallest weights against a reference of 0, which the few-token form's merge
would take from a unit that has no row).
"""
import numpy as np
import pytest
import torch

from gpu_common import run_prefill
from oracle import cache_ops as O
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D
from test_gpu_attn_scaled import FLOOR, TOL, Case, assert_rows, scales_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


def small_case(n, k, pv_mode, size=0.05, shift=-15.0, n_swa=128, t0=3000):
    c = Case(n, t0, k, n_swa, seed=n + k, spread=0.0, pv_mode=pv_mode)
    c.q.copy_(torch.round(c.q.float() * 64) / 64)
    c.q[..., 575] = shift * 24 / size                 # key 575 (no value) is `size` in every row
    for x, cache in ((c.raw_x, c.raw), (c.cmp_x, c.cmp)):
        x.mul_(size)
        x[:, 575] = size
        D.ds4sp_cache_write(cache, 5, x, 0)
    return c


def all_visible(c):
    """The mask of what is visible anyway."""
    t, j = torch.arange(c.T, device="cuda")[:, None], torch.arange(c.T // 4, device="cuda")
    return (4 * j + 3 <= t).to(torch.uint8).contiguous()


@pytest.mark.parametrize("pv_mode", [0, 1])
@pytest.mark.parametrize("n", [40, 3, 1])
@pytest.mark.parametrize("size,shift", [(0.05, -15.0), (1.0, -20.0), (1.0, -90.0), (0.05, 6.0)])
def test_tokens_whose_selected_rows_are_all_hidden(n, pv_mode, size, shift):
    """By a list of -1, then by the mask: four units of 128 rows before the window's."""
    c = small_case(n, 512, pv_mode, size, shift)
    mask = all_visible(c)
    hidden = list(range(0, n, 2))
    listed = c.topk.clone()
    for i in hidden:
        mask[c.t0 + i] = 0
    D.ds4sp_debug_set_mask(c.h, mask)
    by_mask = c.run()
    c.topk[hidden] = -1
    out = c.run()
    assert torch.equal(out, by_mask)
    c.check(out)
    assert (out.abs().amax((1, 2)) > 0).all()
    D.ds4sp_debug_set_mask(c.h, None)
    c.topk.copy_(listed)


@pytest.mark.parametrize("pv_mode", [0, 1])
@pytest.mark.parametrize("n", [40, 3])
@pytest.mark.parametrize("first", [32, 128, 130, 300, 511])
def test_first_selected_rows_outside_the_cache(n, pv_mode, first):
    """The first `first` of 512 entries are skipped and reported; the others are attended."""
    c = small_case(n, 512, pv_mode)
    c.topk[:, :first] = 1 << 29
    out = c.run(status=D.ERR_DEVICE_BOUNDS)
    c.topk[:, :first] = -1
    c.check(out)


@pytest.mark.parametrize("pv_mode", [0, 1])
def test_units_without_rows_between_units_with_some(pv_mode):
    """Units 0, 2 and 3 of five hidden; the last ones' logits are far above the others'."""
    c = small_case(40, 512, pv_mode)
    c.raw_x[:, 575] = -0.05                           # +15, 30 above the compressed rows
    D.ds4sp_cache_write(c.raw, 5, c.raw_x, 0)
    c.topk[:, :128] = 1 << 29
    c.topk[:, 256:] = -5
    out = c.run(status=D.ERR_DEVICE_BOUNDS)
    c.topk[:, :128] = -1
    c.topk[:, 256:] = -1
    c.check(out)


@pytest.mark.parametrize("n", [40, 3])
def test_heads_that_are_not_numbers_beside_hidden_rows(n):
    """Heads 0-2 and 8 of NaN queries: the others' reference still comes from the first unit
    with rows, and is raised, not set again, by the later ones."""
    c = small_case(n, 512, 1)
    c.topk[:, :128] = 1 << 29
    want = c.run(status=D.ERR_DEVICE_BOUNDS)
    bad = torch.zeros(16, dtype=torch.bool)
    bad[[0, 1, 2, 8]] = True
    c.q[:, bad, 7] = float("nan")
    out = c.run(status=D.ERR_DEVICE_BOUNDS)
    assert torch.isnan(out[:, bad]).all() and torch.equal(out[:, ~bad], want[:, ~bad])


def test_a_masked_prefill_and_its_few_token_calls():
    """Through the whole path: the masked top-k lists -1, the prefill and calls of one to three
    tokens agree with the oracle for tokens whose mask leaves nothing."""
    T, k, n_swa, pv = 1200, 160, 96, 0
    c = small_case(8, k, pv, t0=T - 8, n_swa=n_swa)
    g = torch.Generator().manual_seed(3)
    q = torch.cat((torch.randn(T - 8, 16, 576, generator=g).half().cuda(), c.q))
    q.copy_(torch.round(q.float() * 64) / 64)
    q[..., 575] = c.q[0, 0, 575]
    dev = {"q": q, "kv_raw": c.raw, "kv_cmp": c.cmp,
           "q_idx": torch.randint(-3, 4, (T, 64, 128), generator=g).half().cuda(),
           "k_idx": torch.randint(-3, 4, (T // 4, 128), generator=g).half().cuda(),
           "w": torch.randint(0, 4, (T, 64), generator=g).float().cuda()}
    mask = all_visible(c)
    hidden = [700, 1000, 1194, 1196, 1199]
    mask[hidden] = 0
    D.ds4sp_debug_set_mask(c.h, mask)
    topk, out = run_prefill(c.h, dev, T, k)
    assert (topk[hidden] == -1).all()
    raw, cmp_ = c.stored()
    sizes = [scales_of(x, n) for x, n in ((c.raw, T), (c.cmp, T // 4))]
    top = topk.cpu().numpy()

    def check(got, t):
        assert_rows(got.double().cpu().numpy(), q[t].double().cpu().numpy(), O.attended(raw, cmp_, top, 0, t, n_swa),
                    O.attended(*sizes, top, 0, t, n_swa), None, TOL[pv], FLOOR[pv], t)

    for t in hidden + [1193, 1195, 1198]:
        check(out[t], t)
    for lo, n in ((1194, 1), (1195, 2), (1196, 3), (1199, 1)):
        few = torch.empty(n, 16, 512, device="cuda")
        D.ds4sp_sparse_attn(c.h, q[lo:lo + n], c.raw, c.cmp, topk[lo:lo + n], lo, n, few)
        assert D.ds4sp_device_status(c.h)[0] == D.OK
        for i in range(n):
            check(few[i], lo + i)
    D.ds4sp_debug_set_mask(c.h, None)
