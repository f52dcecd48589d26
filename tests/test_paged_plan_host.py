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
