"""sdpa_paged writes where its plan says: a plan whose workspace is not the planner's is refused before any device work."""
import ctypes
import os

import pytest

from split_kv_sparse_gb300 import binding as b
from split_kv_sparse_gb300 import build as bld

FAKE = 1 << 20     # never dereferenced: every call below fails its host checks first


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(b.LIB_PATH):
        bld.build()
    return b.lib()


def call(plan, ws=FAKE):
    p = b.KvPages(FAKE, FAKE, 1, 8, 16, 2, 128, 0, 4096, 256, 128)
    return b.lib().sdpa_paged(ctypes.byref(plan), 2, FAKE, 1024, 128, ctypes.byref(p), FAKE, 4, FAKE, FAKE, None, None, None,
                              0.1, 0, 1.0, FAKE, None, None, ws, None)


@pytest.mark.parametrize("max_q,force", [(1, 0), (1, 4), (100, 0), (100, 4)])
@pytest.mark.parametrize("change", [dict(workspace_bytes=0), dict(workspace_bytes=0, o_acc_bytes=0), dict(o_acc_bytes=1 << 40),
                                    dict(lse_acc_offset=0), dict(lse_acc_bytes=0), dict(map_offset=0), dict(num_sms=1 << 20),
                                    dict(num_sms=1 << 30), dict(total_q_max=1 << 20), "row_kernel", "adaptive_splits"])
def test_plans_that_do_not_fit_their_workspace_are_refused(max_q, force, change):
    plan = b.sdpa_paged_plan(2, 8, 2, 128, "bf16", max_q, 2 * max_q, 5000, num_sms=152, force_splits=force)
    assert plan.num_splits > 1
    if isinstance(change, str):
        change = {change: 1 - getattr(plan, change)}
    if force and "num_sms" in change and change["num_sms"] < 1 << 24:
        pytest.skip("a forced split count does not depend on the SMs")
    for k, v in change.items():
        setattr(plan, k, v)
    assert call(plan) == 3
    assert call(plan, None) == 3


def test_a_count_of_sms_past_an_int_is_refused():
    for max_q in (1, 100):
        with pytest.raises(b.SplitKVError) as e:
            b.sdpa_paged_plan(2, 8, 2, 128, "bf16", max_q, 2 * max_q, 5000, num_sms=(1 << 31) - 1)
        assert e.value.status == 2


@pytest.mark.parametrize("tokens,h_kv", [(96, 8), (262144, 8), (4096, 128)])
@pytest.mark.parametrize("max_q", [1, 500])
def test_the_workspace_is_what_the_header_says(tokens, h_kv, max_q):
    """Partials bounded by the SMs, whatever the tokens, and 8 bytes of map a token and KV head."""
    p = b.sdpa_paged_plan(96, 4 * h_kv, h_kv, 128, "bf16", max_q, tokens, 16384, num_sms=152)
    assert p.row_kernel == (max_q == 1)
    partials = 512 * (2 * 304 * 16 if p.row_kernel else 3 * 152 * 256)
    assert p.o_acc_bytes <= partials and partials < (5.1e6 if p.row_kernel else 60.0e6)
    assert 0 <= p.workspace_bytes - p.o_acc_bytes - p.lse_acc_bytes - 8 * tokens * h_kv <= 768
