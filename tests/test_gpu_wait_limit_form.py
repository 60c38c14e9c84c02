"""Which kernels a lowered wait limit runs: the fused indexer + top-k kernel's give-up is not
provoked, so below the default limit a handle of topk_mode 1 runs the two kernels, and at the
default limit the fused one again. The launches are counted, not inferred, and the limit is half
a second here, so that no wait gives up.
"""
import pytest
import torch

from gpu_common import handle_for, run_prefill, to_device
from sparse_mla_prefill_b200 import build as B
from sparse_mla_prefill_b200 import ds4sp as D
from sparse_mla_prefill_b200.inputs import Workload, generate_small

pytestmark = pytest.mark.gpu

WL = Workload("form", T=600, H_i=8, D_i=64, top_k=32, n_swa=16, seed=0, band=600)


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    B.build()
    D.load_library()


def test_a_lowered_limit_runs_two_kernels_and_the_default_the_fused_one():
    dev = to_device(generate_small(WL.T, WL.H_i, WL.D_i, seed=5))
    results = []
    with handle_for(WL, topk_mode=1) as h:
        D.ds4sp_profile_enable(h, True)
        for limit, launches in ((None, [1, 0, 1]), (500_000_000, [1, 1, 1]), (-1, [1, 0, 1])):
            if limit is not None:
                D.ds4sp_debug_set_wait_limit_ns(h, limit)
            results.append(run_prefill(h, dev, WL.T, WL.top_k))        # asserts status 0
            counts = D.ds4sp_profile_read(h)
            assert [counts[k][1] for k in ("indexer", "topk", "attention")] == launches, limit
    for topk, out in results[1:]:
        assert torch.equal(topk, results[0][0]) and torch.equal(out, results[0][1])
