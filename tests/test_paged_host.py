"""Host-side tests of the paged-cache and prompt entry points (no GPU needed): plans, refusals before any device work,
and the binding's checks of tensors."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.paged as op
from split_kv_sparse_gb300 import binding as b
from split_kv_sparse_gb300 import build as bld

FAKE = 1 << 20     # never dereferenced: every call below fails its host checks first


@pytest.fixture(scope="module", autouse=True)
def built_library():
    import os
    if not os.path.exists(b.LIB_PATH):
        bld.build()
    return b.lib()


def pages(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=1, num_pages=8, page_size=16, h_kv=2, d=128, reserved=0, page_stride=4096,
             row_stride=256, head_stride=128) | kw
    return b.KvPages(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(d=64), 2), (dict(dtype=0), 2), (dict(h_q=7), 1), (dict(batch=0), 1), (dict(h_kv=0), 1), (dict(max_q_per_seq=0), 1),
    (dict(total_q_max=0), 1), (dict(max_kv=0), 1), (dict(force_splits=65), 1), (dict(force_splits=-1), 1),
    (dict(max_splits=65), 1), (dict(num_sms=-1), 1), (dict(h_q=129, h_kv=1), 2), (dict(total_q_max=1 << 30), 1),
])
def test_plan_refusals(kw, code):
    a = dict(batch=2, h_q=8, h_kv=2, d=128, dtype=1, max_q_per_seq=1, total_q_max=2, max_kv=100, num_sms=152) | kw
    pos = [a.pop(k) for k in ("batch", "h_q", "h_kv", "d", "dtype", "max_q_per_seq", "total_q_max", "max_kv")]
    with pytest.raises(b.SplitKVError) as e:
        b.sdpa_paged_plan(*pos, **a)
    assert e.value.status == code


def test_plan_is_deterministic_and_sizes_its_workspace():
    for batch in (1, 8, 96):
        for max_q in (1, 4, 16, 500):
            a = b.sdpa_paged_plan(batch, 32, 8, 128, "e4m3", max_q, batch * max_q, 16384, num_sms=152)
            z = b.sdpa_paged_plan(batch, 32, 8, 128, "e4m3", max_q, batch * max_q, 16384, num_sms=152)
            assert bytes(a) == bytes(z) and 1 <= a.num_splits <= b.MLA_MAX_SPLITS
            for S in (1, 5):
                p = b.sdpa_paged_plan(batch, 32, 8, 128, "e4m3", max_q, batch * max_q, 16384, num_sms=152, force_splits=S)
                assert p.num_splits == S and p.adaptive_splits == 0 and (p.workspace_bytes == 0) == (S == 1)
            assert a.row_kernel == (max_q * 4 <= 16)
            # two pieces of split jobs for each of two CTAs an SM, or three waves of split jobs, whatever the tokens
            rows = 2 * 304 * 16 if a.row_kernel else 3 * 152 * 256
            assert a.num_splits == 64 and a.adaptive_splits == 1
            assert a.o_acc_bytes == rows * 128 * 4 and a.lse_acc_bytes == rows * 4 and a.lse_acc_offset % 256 == 0
            assert a.map_offset >= a.lse_acc_offset + a.lse_acc_bytes
            assert a.workspace_bytes >= a.map_offset + batch * max_q * 8 * 8


def status_of(fn, *args):
    return getattr(b.lib(), fn)(*args)


def test_map_refusals():
    ok = dict(batch=2, page=16, held=FAKE, new=FAKE, cu=FAKE, total=3, table=FAKE, width=4, free=FAKE, cap=8, fin=FAKE,
              fout=FAKE, slots=FAKE, pos=FAKE, stream=None)
    for kw, code in [(dict(batch=0), 1), (dict(batch=16385), 2), (dict(page=0), 1), (dict(width=0), 1), (dict(cap=0), 1),
                     (dict(total=-1), 1), (dict(slots=None), 1), (dict(slots=FAKE + 4), 1), (dict(held=None), 1),
                     (dict(cu=FAKE + 2), 1), (dict(table=None), 1), (dict(fin=None), 1), (dict(fout=None), 1),
                     (dict(free=None), 1), (dict(new=None), 1), (dict(pos=FAKE + 1), 1),
                     (dict(batch=16384, width=1 << 20), 2)]:
        assert status_of("kv_pages_map", *(ok | kw).values()) == code, kw


def test_map_refuses_ordinals_past_32_bits():
    """A list's count and every page of a table freed at once have to add up to an int32."""
    for batch, width, cap, code in [(16384, 1 << 17, 8, 2), (1, 1 << 30, 8, 2), (2, 4, 1 << 30, 2), (2, 4, (1 << 31) - 1, 2)]:
        assert status_of("kv_pages_map", batch, 16, FAKE, FAKE, FAKE, 3, FAKE, width, FAKE, cap, FAKE, FAKE, FAKE, FAKE,
                         None) == code, (batch, width, cap)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(dtype=0), 2), (dict(dtype=3), 2), (dict(num_pages=0), 1),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=131072), 2), (dict(h_kv=0), 1), (dict(d=64), 2),
    (dict(page_stride=0), 1), (dict(row_stride=-256), 1), (dict(row_stride=250), 1), (dict(head_stride=4), 1),
    (dict(page_stride=1 << 40), 1),
])
def test_page_descriptor_refusals(kw, code):
    p = pages(**kw)
    assert status_of("kv_pages_write", ctypes.byref(p), 1, FAKE, FAKE, 256, 128, FAKE, None, None, None) == code
    plan = b.sdpa_paged_plan(2, 8, 2, 128, 1, 1, 2, 100, num_sms=152, force_splits=1)
    assert status_of("sdpa_paged", ctypes.byref(plan), 2, FAKE, 1024, 128, ctypes.byref(p), FAKE, 4, FAKE, FAKE, None,
                     None, None, 0.1, 0, 1.0, FAKE, None, None, None, None) == code


def test_write_refusals():
    p = pages()
    ok = dict(p=ctypes.byref(p), rows=1, k=FAKE, v=FAKE, ts=256, hs=128, slots=FAKE, dk=None, dv=None, stream=None)
    for kw in [dict(rows=-1), dict(k=None), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(slots=None), dict(slots=FAKE + 4),
               dict(ts=0), dict(ts=-256), dict(hs=4), dict(ts=252), dict(dk=FAKE + 1), dict(rows=1 << 31)]:
        assert status_of("kv_pages_write", *(ok | kw).values()) == 1, kw
    assert status_of("kv_pages_write", *(ok | dict(rows=0, k=None, v=None, slots=None)).values()) == 0


def test_paged_attention_refusals():
    plan = b.sdpa_paged_plan(2, 8, 2, 128, 1, 1, 2, 5000, num_sms=152, force_splits=4)
    p = pages()
    ok = dict(plan=ctypes.byref(plan), total_q=2, q=FAKE, ts=1024, hs=128, pages=ctypes.byref(p), table=FAKE, width=4,
              lens=FAKE, cu=FAKE, dq=None, dk=None, dv=None, scale=0.1, od=0, inv=1.0, out=FAKE, lse=None, amax=None,
              ws=FAKE, stream=None)
    other = pages(dtype=2), pages(h_kv=4)
    for kw in [dict(total_q=0), dict(total_q=3), dict(q=None), dict(q=FAKE + 8), dict(ts=1020), dict(hs=-128), dict(hs=0),
               dict(table=None), dict(table=FAKE + 2), dict(width=0), dict(lens=None), dict(cu=None), dict(dq=FAKE + 2),
               dict(scale=float("inf")), dict(od=3), dict(od=2, inv=float("nan")), dict(out=None), dict(out=FAKE + 4),
               dict(lse=FAKE + 1), dict(amax=FAKE + 3), dict(pages=ctypes.byref(other[0])),
               dict(pages=ctypes.byref(other[1])), dict(plan=None), dict(pages=None)]:
        assert status_of("sdpa_paged", *(ok | kw).values()) == 1, kw
    if plan.workspace_bytes:
        for ws in (None, FAKE + 16):
            assert status_of("sdpa_paged", *(ok | dict(ws=ws)).values()) == 3
    bad = b.SdpaPagedPlan()      # zeroed: not made by the planner
    assert status_of("sdpa_paged", *(ok | dict(plan=ctypes.byref(bad))).values()) in (1, 2)


def test_prompt_refusals():
    ok = dict(batch=2, h_q=8, h_kv=2, d=128, dtype=1, total_q=5, total_kv=5, q=FAKE, qts=1024, qhs=128, k=FAKE, v=FAKE,
              kts=256, khs=128, cuq=FAKE, cuk=FAKE, dq=None, dk=None, dv=None, scale=0.1, od=1, inv=1.0, out=FAKE, lse=None,
              amax=None, stream=None)
    for kw, code in [(dict(batch=0), 1), (dict(h_q=9), 1), (dict(d=64), 2), (dict(dtype=3), 2), (dict(h_q=258), 2),
                     (dict(total_q=0), 1), (dict(total_kv=0), 1), (dict(total_kv=1 << 31), 1), (dict(q=None), 1),
                     (dict(k=FAKE + 8), 1), (dict(v=None), 1), (dict(qts=1), 1), (dict(kts=0), 1), (dict(khs=-128), 1),
                     (dict(cuq=None), 1), (dict(cuk=FAKE + 2), 1), (dict(scale=float("nan")), 1), (dict(od=5), 1),
                     (dict(out=None), 1), (dict(lse=FAKE + 2), 1), (dict(total_q=1 << 29), 1)]:
        assert status_of("sdpa_prompt", *(ok | kw).values()) == code, kw


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(b.SplitKVError, match="CUDA"):
        b.kv_pages(x, x)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(b.SplitKVError, match="held_lens"):
        b.kv_pages_map(16, i, i, i, 1, i.view(1, 4), i, i, i, i.long())
    plan = b.sdpa_paged_plan(2, 8, 2, 128, "bf16", 1, 2, 100, num_sms=152)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(b.SplitKVError, match="q must be"):
        b.sdpa_paged(plan, 2, q, pages(), i.view(1, 4), i, i, None, None, None, 0.1, "f32", 1.0, q.float())
    with pytest.raises(b.SplitKVError, match="q must be"):
        b.sdpa_prompt(1, q, q, q, i, i, None, None, None, 0.1, "f32", 1.0, q.float())
    with pytest.raises(b.SplitKVError, match="missing"):
        b.kv_pages_write(pages(), None, None, None)


def test_strides_of_views():
    s = b._strided
    x = torch.zeros((5, 6, 128))
    assert s("t", "x", x[:, 2:4], 3)[:2] == (768, 128)
    assert s("t", "x", x[:, 2:3], 3)[:2] == (768, 128)        # one head: its stride says nothing
    assert tuple(s("t", "x", x[:1, :1], 3)) == (128, 128, 1)
    with pytest.raises(b.SplitKVError):
        s("t", "x", x.transpose(1, 2), 3)
    with pytest.raises(b.SplitKVError):
        s("t", "x", x[0], 3)


def test_oracle_map_and_attention():
    """Closed forms: pages popped from the top in request order, freed ones first; equal scores give the mean of V."""
    table, F, left, slots, pos = op.map_pages(16, [32, 0, 5], [0, 20, 6], [0, 0, 20, 21], 23,
                                              [[3, 4], [-1, -1], [7, -1]], [9, 8, 0, 0, 0], 2)
    assert F.tolist() == [9, 8, 3, 4, 0] and table.tolist() == [[3, 4], [4, 3], [7, -1]] and left == (2, 0)
    assert slots[:16].tolist() == list(range(64, 80)) and slots[16:20].tolist() == [48, 49, 50, 51]
    assert slots[20] == 7 * 16 + 5 and pos[20] == 5 and slots[21:].tolist() == [-1, -1]
    v = np.random.default_rng(0).standard_normal((4, 1, 8))
    O, L, A = op.attend(np.zeros((2, 2, 8)), np.zeros((4, 1, 8)), v, np.array([[1, 1, 0, 0], [0, 0, 0, 0]], bool), 1.0)
    assert np.allclose(O[0], v[:2, 0].mean(0)) and np.all(O[1] == 0) and np.all(np.isneginf(L[1])) and np.allclose(L[0], 1)
    assert np.allclose(A[0, 0], np.abs(v[:2, 0]).mean(0))
