"""GPU tests of waits that run out in a CTA's later jobs: the call ends, the status says so, and the next call is right.
Nothing is withheld and nothing faults: the limits are shorter than what a CTA's second job waits for."""
import math

import pytest
import torch

from _paged_util import D, Paged, check, cu_of, run_paged, scalar, status_clear, values
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,keys", [(64, 384), (300, 300)])
def test_waits_that_run_out_between_the_jobs_of_a_cta(dtype, n, keys):
    """About five jobs a CTA. The K loader has started its next job's first tile when it waits for the products of the
    job before, so a limit of some microseconds can run out right there."""
    sq, kv, h_q = [n] * 96, [keys] * 96, 32
    c = Paged(dtype, kv, 8, 64, seed=n)
    q, dq = values(torch.Generator().manual_seed(n), (sum(sq), h_q, D), dtype)
    cu = cu_of(sq)
    total = sum(sq)
    plan = b.sdpa_paged_plan(len(kv), h_q, 8, D, dtype, n, total, keys, force_splits=1)
    out = torch.empty((total, h_q, D), device="cuda")
    args = [q.cuda(), b.kv_pages(c.k.cuda(), c.v.cuda()), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), scalar(dq, dtype),
            scalar(c.dk, dtype), scalar(c.dv, dtype), 1 / math.sqrt(D), "f32", 1.0, out]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    seen = 0
    try:
        for limit in (300, 600, 1000, 1500, 2000, 2500, 3000, 3500, 4000, 5000, 6000, 8000, 12000):
            b.mla_set_wait_limit_ns(limit)
            flush.fill_(1)          # the keys are not in the cache
            b.sdpa_paged(plan, total, *args)
            torch.cuda.synchronize()
            st, site = b.mla_get_status()
            assert st in (0, b.MLA_STATUS_TIMEOUT) and (site != 0) == (st != 0), (limit, st, site)
            assert site in (0, 201, 202, 203, 204), "a copy or a product was still in flight at the end"
            seen += st
    finally:
        b.mla_set_wait_limit_ns(0)
    assert seen, "no wait ran out"
    got, lse, _ = run_paged(c, q, dq, cu, h_q, force_splits=1, amax=False)
    ref = c.reference(q[:n * 2], dq, cu_of(sq[:2] + [0] * 94), 1 / math.sqrt(D))
    check(got[:n * 2], lse[:n * 2], None, ref, dtype)
