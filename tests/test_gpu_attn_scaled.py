"""Attention over a kv_format 5 cache (e4m3 rows, a scale per block of 64) against the
float64 oracle on the stored values.

Tolerances, as relative error in the 2-norm over a token's head (and its largest element
against the head's largest): the stored values and the queries enter exactly, so what is
left is fp32 sums and the terms of the probabilities. S sums 576 products in fp32: each of
18 instructions rounds the running sum, and the whole is off by about 2^-22 of
sum|q k| <= |q| |k|; times scale that is a logit error of 2^-22 * |q| |k| / 24, below 2e-5
for |q| |k| up to 2,000 (the inputs here: |q| ~ 24, |k| < 80). The exponential adds 2^-22.
A weight is first hi + lo, hi its fp16 rounding: pv_mode 0 keeps hi alone, off by at most
2^-11 of the weight (its three terms hold hi's eleven bits: a term is off by 2^-4 of itself at
most, so three leave 2^-12); pv_mode 1 has five, which leave 2^-20. The 640 rows' errors do not
add up in phase, but the bound takes them as if they did: pv_mode 1 3e-5 (2e-5 + 2^-22 + 2^-20 +
sums of 640 in fp32, 2^-24 * 4 instructions a unit), pv_mode 0 3e-5 + 2^-11 = 5.2e-4, each of
sum p |v|, which for cancelling values is larger than |out|: both bounds are applied to
sum p |v| per element. The last term's smallest spacing is 2^-9 of its unit, 2^-9 (three terms)
or 2^-18 (five), so a row also adds up to 2^-19 or 2^-28 of |code|, where the largest weight of
the first rows is set to 1/8 (three terms) or 1/32 (five), so that w is at least p s / (p s)_max
of that: over the sum of w / s this is the bound's second part (``floor``), which for a row of
small weight and large values is the larger one.
"""
import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D

pytestmark = pytest.mark.gpu
TOL = {0: 5.2e-4, 1: 3e-5}
FLOOR = {0: 2.0 ** -16, 1: 2.0 ** -23}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


def rows_of(n, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, 576, generator=g) * torch.exp(spread * torch.randn(n, 1, generator=g))).half().cuda()


def cache_of(x):
    c = torch.full((D.ds4sp_cache_bytes(5, 576, max(len(x), 1)),), 0x7F, dtype=torch.uint8, device="cuda")   # NaN codes
    D.ds4sp_cache_write(c, 5, x, 0)
    return c


def choose(n, t0, k, n_c, seed):
    """min(k, n_vis(t)) visible rows per token, ascending, then -1."""
    rng = np.random.default_rng(seed)
    top = np.full((n, k), -1, np.int32)
    for i in range(n):
        nv = min((t0 + i + 1) // 4, n_c)
        m = min(k, nv)
        top[i, :m] = np.sort(rng.choice(nv, m, replace=False))
    return torch.from_numpy(top).cuda()


def scales_of(cache, rows):
    rec = cache.view(-1, 576)[64::65, :4].contiguous().view(torch.float32).view(-1)
    return rec[torch.arange(rows, device="cuda") // 64].double().cpu().numpy()


def assert_rows(got, q, rows, size, scale, tol, floor, what):
    want, mass = O.attention_rows(q, rows, scale), O.attention_rows(q, rows, scale, absolute=True)
    z = q @ rows.T * (1 / 24.0 if scale is None else scale)
    w = np.exp(z - (z + np.log(size)).max(1, keepdims=True)) * size        # 1 for the largest
    least = floor * (np.abs(rows[:, :512]) / size[:, None]).sum(0) / (w / size).sum(1, keepdims=True)
    err = np.abs(got - want)
    assert (err <= tol * mass + least).all(), (what, (err / (tol * mass + least)).max())


class Case:
    def __init__(self, n, t0, k, n_swa, seed=0, spread=0.5, pv_mode=1, T=None, **cfg):
        g = torch.Generator().manual_seed(seed)
        self.n, self.t0, self.n_swa = n, t0, n_swa
        T = T or t0 + n
        self.T = T
        self.raw_x, self.cmp_x = rows_of(T, seed + 1, spread), rows_of(max(T // 4, 1), seed + 2, spread)
        self.q = torch.randn(n, 16, 576, generator=g).half().cuda()
        self.raw, self.cmp = cache_of(self.raw_x), cache_of(self.cmp_x)
        self.topk = choose(n, t0, k, T // 4, seed) if k else None
        self.h = D.ds4sp_create(D.make_config(n_idx_heads=64, d_idx=128, top_k=k, n_swa=n_swa, max_tokens=T,
                                              kv_format=5, pv_mode=pv_mode, **cfg))
        self.tol, self.floor = TOL[pv_mode], FLOOR[pv_mode]
        self.scale = cfg.get("softmax_scale") or None

    def run(self, lo=0, hi=None, stream=None, status=D.OK):
        hi = self.n if hi is None else hi
        out = torch.full((hi - lo, 16, 512), float("nan"), device="cuda")
        D.ds4sp_sparse_attn(self.h, self.q[lo:hi], self.raw, self.cmp,
                            self.topk[lo:hi] if self.topk is not None else None, self.t0 + lo, hi - lo, out, stream)
        if stream is None:
            st, _ = D.ds4sp_device_status(self.h)
            assert st == status
        return out

    def stored(self):
        return [D.ds4sp_cache_read(c, 5, 576, row0=0, n=len(x), dtype=torch.float32).double().cpu().numpy()
                for c, x in ((self.raw, self.raw_x), (self.cmp, self.cmp_x))]

    def check(self, out, tokens=None, lo=0):
        raw, cmp_ = self.stored()
        q = self.q.double().cpu().numpy()
        top = self.topk.cpu().numpy() if self.topk is not None else None
        got = out.double().cpu().numpy()
        for i in range(len(got)) if tokens is None else tokens:
            rows = O.attended(raw, cmp_, top, self.t0, lo + i, self.n_swa)
            size = O.attended(*(scales_of(c, len(x)) for c, x in ((self.raw, self.raw_x), (self.cmp, self.cmp_x))),
                              top, self.t0, lo + i, self.n_swa)
            assert_rows(got[i], q[lo + i], rows, size, self.scale, self.tol, self.floor, i)
        return got


@pytest.mark.parametrize("pv_mode", [0, 1])
@pytest.mark.parametrize("n,t0,k,n_swa", [
    (1, 0, 16, 8), (3, 0, 16, 8), (64, 0, 16, 32), (40, 0, 0, 1), (200, 0, 64, 300), (37, 800, 129, 1),
    (45, 700, 128, 128), (50, 5000, 512, 128), (170, 300, 33, 95), (37, 8000, 2000, 77)])
def test_prefill_matches_oracle(n, t0, k, n_swa, pv_mode):
    c = Case(n, t0, k, n_swa, seed=n + k, pv_mode=pv_mode)
    c.check(c.run())


@pytest.mark.parametrize("pv_mode", [0, 1])
@pytest.mark.parametrize("n,t0,k,n_swa", [
    (1, 0, 0, 1), (1, 0, 16, 128), (1, 3, 16, 1), (1, 20000, 512, 128), (2, 20001, 512, 128), (5, 122875, 512, 128),
    (36, 4000, 100, 7), (1, 8192, 1900, 140), (3, 9000, 1920, 200)])
def test_few_tokens_match_oracle(n, t0, k, n_swa, pv_mode):
    c = Case(n, t0, k, n_swa, seed=n + k, pv_mode=pv_mode)
    c.check(c.run())


def test_a_tokens_result_does_not_depend_on_the_call():
    """Few-token calls of widths 1 .. 5 give a token the same bits; so do long calls of
    different lengths and starts."""
    c = Case(80, 3000, 200, 100)
    whole = c.run()
    assert torch.equal(c.run(40, 80), whole[40:])
    assert torch.equal(c.run(0, 37), whole[:37])
    five = c.run(70, 75)
    for lo in range(70, 75):
        assert torch.equal(c.run(lo, 75), five[lo - 70:])
        assert torch.equal(c.run(lo, lo + 1)[0], five[lo - 70])
    assert torch.equal(c.run(), whole)


def test_uneven_block_scales_and_zero_blocks():
    """Blocks of scale 2^-32 .. 2^8 beside blocks of zeros: a row's scale joins its weight."""
    c = Case(60, 2000, 300, 200, seed=5, spread=0.0)
    for x, cache in ((c.raw_x, c.raw), (c.cmp_x, c.cmp)):
        for b in range(0, len(x), 64):
            x[b:b + 64] *= [1.0, 2.0 ** -20, 0.0, 0.125, 3.0, 2.0 ** -8][b // 64 % 6]
        D.ds4sp_cache_write(cache, 5, x, 0)
    c.check(c.run())
    c.check(c.run(10, 13), lo=10)


def test_all_rows_zero():
    c = Case(45, 500, 30, 40, seed=6)
    for x, cache in ((c.raw_x, c.raw), (c.cmp_x, c.cmp)):
        x.zero_()
        D.ds4sp_cache_write(cache, 5, x, 0)
    assert torch.equal(c.run(), torch.zeros(45, 16, 512, device="cuda"))
    assert torch.equal(c.run(4, 6), torch.zeros(2, 16, 512, device="cuda"))


def test_reference_raised_by_later_units():
    """Logits that grow along the rows by far more than 2^8 a unit, and one that falls: each
    unit of 128 rows raises the reference. Keys are one direction, values another."""
    n, T = 40, 2048
    c = Case(n, T - n, 500, 120, seed=7, spread=0.0)
    c.raw_x.mul_(0.5)
    c.cmp_x.mul_(0.5)
    ramp = torch.linspace(-40.0, 40.0, T // 4, device="cuda")
    c.cmp_x[:, 575] = ramp.half()
    c.raw_x[:, 575] = 45.0
    c.q[..., 575] = 20.0
    c.q[:, 3, 575] = -20.0                  # head 3 falls
    c.q[:, 5, 575] = 0.0                    # head 5 stays
    D.ds4sp_cache_write(c.raw, 5, c.raw_x, 0)
    D.ds4sp_cache_write(c.cmp, 5, c.cmp_x, 0)
    # |q| |k| here: |q575 k575| alone reaches 900, and sum|q k| / 24 about 70: the bound of
    # the module text (logit error 2^-22 * 2000 / 24) covers it
    c.check(c.run())
    c.check(c.run(20, 23), lo=20)


def test_query_range():
    """Heads of zeros, of fp16's smallest and largest values, and of uneven values."""
    c = Case(40, 600, 60, 40, seed=8, softmax_scale=1e-4)
    c.q[:, 0] = 0
    c.q[:, 1] *= 2.0 ** -14
    c.q[:, 2] = (c.q[:, 2].float() * 16000).clamp(-65504, 65504).half()
    c.q[:, 4, ::2] *= 2.0 ** -10
    # logit error: 2^-22 * 1e-4 * |q| |k| with |q| ~ 16000 * 24 and |k| ~ 30: 2.7e-4 for head 2
    c.tol = 4e-4
    c.check(c.run())


def test_not_a_number_stays_with_its_head_or_row():
    c = Case(40, 600, 60, 40, seed=9)
    want = c.run()
    c.q[7, 3, 100] = float("nan")
    c.q[8, 2, 5] = float("inf")
    out = c.run()
    bad = torch.isnan(out).all(-1)
    assert bad[7, 3] and bad[8, 2] and bad.sum() == 2
    keep = ~torch.isnan(out)
    assert torch.equal(out[keep], want[keep])
    c.q.copy_(torch.nan_to_num(c.q, 0.0, 0.0, 0.0))
    row = c.t0 + 39                          # attended by the last token alone
    c.raw_x[row, 17] = float("nan")
    D.ds4sp_cache_write(c.raw, 5, c.raw_x, 0)
    out = c.run()
    assert torch.isnan(out[39]).all() and torch.isfinite(out[:39]).all()


def test_selected_rows_outside_the_cache_are_skipped_and_reported():
    c = Case(50, 900, 40, 30, seed=10)
    want = c.run()
    good = c.topk.clone()
    c.topk[3, 5], c.topk[20, 0], c.topk[21, 39] = 1 << 30, -7, 950 // 4 + 5
    out = c.run(status=D.ERR_DEVICE_BOUNDS)
    touched = torch.tensor([3, 20, 21])
    same = torch.ones(50, dtype=torch.bool)
    same[touched] = False
    assert torch.equal(out[same], want[same])
    c.topk[c.topk == 1 << 30] = -1
    c.topk[c.topk == -7] = -1
    c.topk[21, 39] = -1
    c.check(out, tokens=[3, 20, 21])
    c.topk.copy_(good)
    assert torch.equal(c.run(), want)


def test_explicit_mask_form():
    c = Case(60, 1000, 50, 30, seed=11)
    want = c.run()
    mask = torch.zeros(1060, 265, dtype=torch.uint8, device="cuda")
    t = torch.arange(1060, device="cuda")
    mask[4 * torch.arange(265, device="cuda")[None] + 3 <= t[:, None]] = 1
    D.ds4sp_debug_set_mask(c.h, mask)
    assert torch.equal(c.run(), want)
    top = c.topk.cpu().numpy()
    for i in (0, 33):                        # hide half of a token's rows, and all of another's
        mask[1000 + i, torch.from_numpy(top[i][: 25 if i == 0 else 50].astype(np.int64))] = 0
    out = c.run()
    c.topk[0, :25] = -1
    c.topk[33] = -1
    c.check(out, tokens=[0, 33])
    assert torch.equal(out[1:33], want[1:33])
    D.ds4sp_debug_set_mask(c.h, None)


def test_prefill_of_a_written_cache_by_bands_and_from_the_host():
    """Rotate, write, prefill: the run of the operators as they are used, by bands on the
    device, then from host buffers (whose copies bring whole blocks): the same bits."""
    from gpu_common import run_prefill
    T, k, n_swa, band = 1500, 96, 100, 512
    g = torch.Generator().manual_seed(12)
    rope = D.make_rope(64, scaling=3, factor=32.0, orig_len=4096)
    row_rope = D.make_rope(64, offset=512, scaling=3, factor=32.0, orig_len=4096)
    q = torch.randn(T, 16, 576, generator=g).half().cuda()
    D.ds4sp_rope(q[..., 512:], rope, out=q[..., 512:])
    raw, cmp_ = (torch.zeros(D.ds4sp_cache_bytes(5, 576, r), dtype=torch.uint8, device="cuda") for r in (T, T // 4))
    D.ds4sp_cache_write(raw, 5, torch.randn(T, 576, generator=g).cuda(), 0, rope=row_rope)
    D.ds4sp_cache_write(cmp_, 5, torch.randn(T // 4, 576, generator=g).cuda(), 0, rope=row_rope, pos_step=4)
    dev = {"q": q, "kv_raw": raw, "kv_cmp": cmp_,
           "q_idx": torch.randint(-3, 4, (T, 8, 64), generator=g).half().cuda(),
           "k_idx": torch.randint(-3, 4, (T // 4, 64), generator=g).half().cuda(),
           "w": torch.randint(0, 4, (T, 8), generator=g).float().cuda()}
    for dependent in (1, 0):
        cfg = D.make_config(n_idx_heads=8, d_idx=64, top_k=k, n_swa=n_swa, max_tokens=T, band=band, kv_format=5,
                            pv_mode=1, dependent_launch=dependent)
        with D.ds4sp_create(cfg) as h:
            topk, out = run_prefill(h, dev, T, k)
            if dependent:
                first = out
                stored = [D.ds4sp_cache_read(c, 5, 576, row0=0, n=n, dtype=torch.float32).double().cpu().numpy()
                          for c, n in ((raw, T), (cmp_, T // 4))]
                toks = [0, 1, 2, 3, 64, 511, 512, 700, 1023, 1024, 1499]
                sizes = [scales_of(c, n) for c, n in ((raw, T), (cmp_, T // 4))]
                top, got = topk.cpu().numpy(), out.double().cpu().numpy()
                for t in toks:
                    assert_rows(got[t], q[t].double().cpu().numpy(), O.attended(*stored, top, 0, t, n_swa),
                                O.attended(*sizes, top, 0, t, n_swa), None, TOL[1], FLOOR[1], t)
                host = {n: v.cpu().pin_memory() for n, v in dev.items()}
                dev2 = {n: torch.empty_like(v) for n, v in dev.items()}
                topk2, out2 = torch.empty_like(topk), torch.empty_like(out)
                out_h = torch.empty(out.shape).pin_memory()
                D.prefill_host(h, host, dev2, T, topk2, out2, D.band_workspace(h, T, "cuda"), out_h)
                torch.cuda.synchronize()
                assert torch.equal(out_h, out.cpu()) and torch.equal(topk2, topk)
            else:
                assert torch.equal(out, first)


@pytest.mark.parametrize("n", [3, 60])
def test_captured_and_on_another_stream(n):
    c = Case(n, 2000, 100, 64, seed=13)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.run(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(c.run(), want)
    graph = torch.cuda.CUDAGraph()
    static = torch.empty(n, 16, 512, device="cuda")
    with torch.cuda.graph(graph):
        D.ds4sp_sparse_attn(c.h, c.q, c.raw, c.cmp, c.topk, c.t0, n, static)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(static, want)
    c.q.copy_(torch.randn(c.q.shape, generator=torch.Generator().manual_seed(14)).half())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(static, c.run()) and not torch.equal(static, want)


@pytest.mark.parametrize("n", [3, 200])
def test_give_up_returns_and_the_next_call_is_whole(n):
    """With the wait limit at 0 every wait that is not already complete gives up: the launch
    ends with the status bit set, and at the default limit the next call gives the same bits
    as before."""
    c = Case(n, 3000, 300, 128, seed=15)
    want = c.run()
    D.ds4sp_debug_set_wait_limit_ns(c.h, 0)
    c.run(status=D.ERR_DEVICE_BOUNDS)
    D.ds4sp_debug_set_wait_limit_ns(c.h, -1)
    assert torch.equal(c.run(), want)


def test_long_cache_offsets():
    """Rows whose bytes lie past 2^32 of the raw cache: 7.5 million tokens (4.4 GB)."""
    T, n_swa = 7_500_000, 200
    raw = torch.zeros(D.ds4sp_cache_bytes(5, 576, T), dtype=torch.uint8, device="cuda")
    tail = 7_499_776                         # a block's start
    x = rows_of(T - tail, 16)
    D.ds4sp_cache_write(raw, 5, x, tail)
    q = torch.randn(2, 16, 576, generator=torch.Generator().manual_seed(17)).half().cuda()
    out = torch.empty(2, 16, 512, device="cuda")
    with D.ds4sp_create(D.make_config(n_idx_heads=64, d_idx=128, top_k=0, n_swa=n_swa, max_tokens=T, kv_format=5,
                                      pv_mode=1)) as h:
        D.ds4sp_sparse_attn(h, q, raw, None, None, T - 2, 2, out)
        assert D.ds4sp_device_status(h)[0] == D.OK
    stored = D.ds4sp_cache_read(raw, 5, 576, row0=tail, n=T - tail, dtype=torch.float32).double().cpu().numpy()
    for i in range(2):
        end = T - 2 + i + 1 - tail
        rows = stored[end - n_swa:end]
        size = scales_of(raw[tail // 64 * 65 * 576:], T - tail)[end - n_swa:end]
        assert_rows(out[i].double().cpu().numpy(), q[i].double().cpu().numpy(), rows, size, None, TOL[1], FLOOR[1], i)
