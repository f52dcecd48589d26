"""GPU tests of waits that run out in the kernels over 4-bit pages: each of their roles' sites, nothing left in flight, and a right next
call. Nothing is withheld and nothing faults: the limits are shorter than what loads and blocks take.

Sites: 201 to 204 the roles of the 256-row kernel, 301 a computing warp of the kernels of 8 and of 16 rows that waits for a block, 303 a
loading warp that waits for a free place; 205 and 302 would be copies still in flight at a CTA's end."""
import math

import pytest
import torch

from _four_bit_util import Paged4, f32, run4
from _paged_util import D, check, cu_of, status_clear
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


@pytest.mark.parametrize("sq,kv,h_q,h_kv,row_kernel", [
    ([1] * 64, 6000, 8, 2, 2),      # long sequences: a loading warp's ring is full
    ([1] * 600, 200, 8, 2, 2),      # many short ones a CTA: loads and computation meet at the pieces' ends
    ([3] * 64, 6000, 8, 2, 1),
    ([1] * 300, 200, 16, 1, 1),
    ([16] * 40, 3000, 8, 2, 0),
    ([200] * 12, 900, 8, 2, 0),
])
def test_waits_that_run_out(sq, kv, h_q, h_kv, row_kernel):
    kv = [kv] * len(sq)
    c, cu, total = Paged4(kv, h_kv, 64, seed=13), cu_of(sq), sum(sq)
    q = torch.randn((total, h_q, D), generator=torch.Generator().manual_seed(14)).to(torch.bfloat16)
    plan = b.sdpa_paged_plan(len(kv), h_q, h_kv, D, "e2m1", max(sq), total, max(kv))
    assert plan.row_kernel == row_kernel
    ws = torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    out = torch.empty((total, h_q, D), device="cuda")
    args = [q.cuda(), c.pages(), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), None, f32(c.dk), f32(c.dv), 1 / math.sqrt(D), "f32", 1.0, out,
            None, None, ws]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    sites = []
    try:
        for limit in (100, 200, 300, 500, 700, 1000, 1500, 2000, 3000, 4000, 6000, 8000):
            b.mla_set_wait_limit_ns(limit)
            flush.fill_(1)          # the keys are not in the cache
            b.sdpa_paged(plan, total, *args)
            torch.cuda.synchronize()
            st, site = b.mla_get_status()
            assert st in (0, b.MLA_STATUS_TIMEOUT) and (site != 0) == (st != 0), (limit, st, site)
            sites.append(site)
    finally:
        b.mla_set_wait_limit_ns(0)
    assert any(sites), "no wait ran out"
    assert set(sites) <= ({0, 301, 303} if row_kernel else {0, 201, 202, 203, 204}), sites
    n = min(len(sq), 20)
    got, lse, _ = run4(c, q, cu, h_q, amax=False)
    ref = c.reference(q[:int(cu[n])], cu_of(sq[:n] + [0] * (len(sq) - n)), 1 / math.sqrt(D))
    check(got[:int(cu[n])], lse[:int(cu[n])], None, ref, "e4m3")
