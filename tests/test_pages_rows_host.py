"""Host-side tests of the 4-bit cache, the append that rotates and the read-back (no GPU needed): refusals before any device work,
the binding's checks of tensors, plans, and the oracle's own pins."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle.paged as op
from oracle import codecs
from split_kv_sparse_gb300 import binding as b
from split_kv_sparse_gb300 import build as bld
from test_paged_binding_host import On

FAKE = 1 << 20     # never dereferenced: every call below fails its host checks first


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(b.LIB_PATH):
        bld.build()
    return b.lib()


def pages(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=4, num_pages=8, page_size=16, h_kv=2, d=128, reserved=0, page_stride=2048, row_stride=128,
             head_stride=64, k_scales=FAKE, v_scales=FAKE, scale_page_stride=256, scale_head_stride=128) | kw
    return b.KvPages(*a.values())


def status_of(fn, *args):
    return getattr(b.lib(), fn)(*args)


# ------------------------------------------------------------------ refusals --

@pytest.mark.parametrize("kw,code", [
    (dict(k_scales=None), 1), (dict(v_scales=None), 1), (dict(k_scales=FAKE + 8), 1), (dict(v_scales=FAKE + 4), 1),
    (dict(scale_page_stride=0), 1), (dict(scale_page_stride=24), 1), (dict(scale_head_stride=-128), 1), (dict(scale_head_stride=8), 1),
    (dict(scale_page_stride=1 << 40), 1), (dict(row_stride=72), 1), (dict(head_stride=0), 1), (dict(k=FAKE + 8), 1), (dict(d=64), 2),
    (dict(page_size=24), 2), (dict(dtype=3), 2), (dict(dtype=5), 2), (dict(num_pages=0), 1),
])
def test_descriptor_refusals(kw, code):
    p = pages(**kw)
    assert status_of("kv_pages_write", ctypes.byref(p), 1, FAKE, FAKE, 256, 128, FAKE, None, None, None) == code
    assert status_of("kv_pages_read", ctypes.byref(p), 1, FAKE, None, None, FAKE, FAKE, 256, 128, None) == code
    plan = b.sdpa_paged_plan(2, 8, 2, 128, "e2m1", 1, 2, 100, num_sms=152, force_splits=1)
    assert status_of("sdpa_paged", ctypes.byref(plan), 2, FAKE, 1024, 128, ctypes.byref(p), FAKE, 4, FAKE, FAKE, None,
                     None, None, 0.1, 0, 1.0, FAKE, None, None, None, None) in (code, 1)


ROTARY = dict(p=None, rows=1, h_q=4, q=FAKE, qts=512, qhs=128, k=FAKE, v=FAKE, ts=256, hs=128, pos=FAKE, cs=FAKE, n=100, rot=128, inter=0,
              slots=FAKE, dq=None, dk=None, dv=None, qd=1, qo=FAKE, qots=512, qohs=128, ko=None, kots=0, kohs=0, stream=None)


@pytest.mark.parametrize("dtype", [1, 2, 4])
def test_rotary_refusals(dtype):
    p = pages(dtype=dtype) if dtype == 4 else pages(dtype=dtype, page_stride=4096, row_stride=256, head_stride=128)
    ok = ROTARY | dict(p=ctypes.byref(p))
    for kw, code in [(dict(p=None), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(h_q=-1), 1), (dict(q=None), 1), (dict(q=FAKE + 8), 1),
                     (dict(qts=0), 1), (dict(qhs=4), 1), (dict(k=None), 1), (dict(v=FAKE + 2), 1), (dict(ts=250), 1), (dict(hs=-128), 1),
                     (dict(pos=None), 1), (dict(pos=FAKE + 2), 1), (dict(cs=None), 1), (dict(cs=FAKE + 4), 1), (dict(n=0), 1), (dict(n=1 << 32), 1),
                     (dict(rot=0), 2), (dict(rot=48), 2), (dict(rot=160), 2), (dict(rot=-32), 2), (dict(inter=2), 1), (dict(slots=None), 1),
                     (dict(slots=FAKE + 4), 1), (dict(dq=FAKE + 1), 1), (dict(dk=FAKE + 2), 1), (dict(dv=FAKE + 3), 1), (dict(qd=0), 1),
                     (dict(qd=4), 1), (dict(qo=None), 1), (dict(qo=FAKE + 8), 1), (dict(qots=4), 1), (dict(qohs=0), 1),
                     (dict(qd=2, qots=520), 1), (dict(ko=FAKE + 8, kots=256, kohs=128), 1), (dict(ko=FAKE, kots=0, kohs=128), 1),
                     (dict(ko=FAKE, kots=256, kohs=12), 1), (dict(rows=(1 << 31) - 1, h_q=1 << 10), 1)]:
        assert status_of("kv_pages_write_rotary", *(ok | kw).values()) == code, kw
    assert status_of("kv_pages_write_rotary", *(ok | dict(rows=0, q=None, k=None, v=None, pos=None, slots=None, qo=None)).values()) == 0


def test_read_refusals():
    p = pages()
    ok = dict(p=ctypes.byref(p), rows=1, slots=FAKE, dk=None, dv=None, k=FAKE, v=FAKE, ts=256, hs=128, stream=None)
    for kw in [dict(p=None), dict(rows=-1), dict(rows=1 << 31), dict(k=None), dict(k=FAKE + 2), dict(v=None), dict(v=FAKE + 8), dict(slots=None),
               dict(slots=FAKE + 4), dict(ts=0), dict(hs=4), dict(dk=FAKE + 1), dict(dv=FAKE + 2)]:
        assert status_of("kv_pages_read", *(ok | kw).values()) == 1, kw
    assert status_of("kv_pages_read", *(ok | dict(rows=0, k=None, v=None, slots=None)).values()) == 0


def test_plans_and_types():
    """Few query rows take the kernels of 8 and 16 rows; the bytes of a plan do not depend on the type; prompts have no 4-bit form."""
    for max_q, group, kernel in [(1, 4, 2), (2, 4, 2), (1, 8, 2), (3, 4, 1), (4, 4, 1), (1, 16, 1)]:
        p = b.sdpa_paged_plan(8, 2 * group, 2, 128, "e2m1", max_q, 8 * max_q, 16384, num_sms=152)
        e = b.sdpa_paged_plan(8, 2 * group, 2, 128, "e4m3", max_q, 8 * max_q, 16384, num_sms=152)
        assert p.row_kernel == kernel and e.row_kernel == 1
        assert (p.workspace_bytes, p.o_acc_bytes, p.num_splits) == (e.workspace_bytes, e.o_acc_bytes, e.num_splits)
    # forced splits of the kernel of 8 rows: every job of 8 rows has its slots
    p = b.sdpa_paged_plan(8, 8, 2, 128, "e2m1", 2, 16, 16384, num_sms=152, force_splits=4)
    assert p.row_kernel == 2 and p.o_acc_bytes == (16 // 2 + 8) * 2 * 4 * 16 * 128 * 4
    assert status_of("sdpa_prompt", 1, 8, 2, 128, 4, 4, 4, FAKE, 1024, 128, FAKE, FAKE, 256, 128, FAKE, FAKE, None, None, None, 0.1, 0, 1.0, FAKE,
                     None, None, None) == 2
    plan = b.sdpa_paged_plan(2, 8, 2, 128, "e2m1", 1, 2, 100, num_sms=152, force_splits=1)
    args = [2, FAKE, 1024, 128, None, FAKE, 4, FAKE, FAKE, None, None, None, 0.1, 0, 1.0, FAKE, None, None, None, None]
    other = pages(dtype=2, row_stride=256, head_stride=128)
    args[4] = ctypes.byref(other)
    assert status_of("sdpa_paged", ctypes.byref(plan), *args) == 1          # pages of another type than the plan's
    args[4] = ctypes.byref(pages())
    for row_kernel in (-1, 3):
        plan.row_kernel = row_kernel
        assert status_of("sdpa_paged", ctypes.byref(plan), *args) == 1
    wide = b.sdpa_paged_plan(2, 32, 2, 128, "e2m1", 1, 2, 100, num_sms=152, force_splits=1)
    wide.row_kernel = 2                                                    # 16 heads a group do not fit 8 rows
    assert status_of("sdpa_paged", ctypes.byref(wide), *args) == 1


# ------------------------------------------------------------------- binding --

@pytest.fixture
def current(monkeypatch):
    dev = [0]
    monkeypatch.setattr(b, "_device", lambda where: dev[0])
    monkeypatch.setattr(b, "_on", lambda stream, d: None)
    return dev


def four(page=16, h=2, n=8, dev=0):
    codes = [On(dev, (n, page, h, 64), torch.uint8) for _ in range(2)]
    scales = [On(dev, (n, h, page, 8), torch.uint8) for _ in range(2)]
    for s in scales:
        s.x = s.x.permute(0, 2, 1, 3)
        s.shape = s.x.shape
    return codes + scales


def test_descriptor_of_a_four_bit_cache(current):
    p = b.kv_pages(*four())
    assert (p.dtype, p.d, p.h_kv, p.page_size) == (b.SDPA_E2M1, 128, 2, 16)
    assert (p.page_stride, p.row_stride, p.head_stride) == (2048, 128, 64) and (p.scale_page_stride, p.scale_head_stride) == (256, 128)
    p = b.kv_pages(*four(h=1, n=1))
    assert p.scale_page_stride % 16 == 0 and p.scale_head_stride % 16 == 0 and p.scale_page_stride > 0
    bad = four()
    bad[2] = bad[3] = On(0, (8, 16, 2, 8), torch.uint8)          # rows of a head apart
    with pytest.raises(b.SplitKVError, match="side by side"):
        b.kv_pages(*bad)
    for i, x in [(0, On(0, (8, 16, 2, 64), torch.bfloat16)), (1, On(0, (8, 16, 2, 32), torch.uint8)), (2, None), (3, On(0, (8, 16, 2, 4), torch.uint8)),
                 (2, On(0, (8, 16, 2, 8), torch.bfloat16)), (0, On(1, (8, 16, 2, 64), torch.uint8)), (3, On(1, (8, 16, 2, 8), torch.uint8))]:
        bad = four()
        bad[i] = x
        with pytest.raises(b.SplitKVError) as e:
            b.kv_pages(*bad)
        assert e.value.status == b.MLA_ERR_INVALID_ARG


def test_rotary_and_read_checks(current):
    p = b.kv_pages(*four())
    t = lambda *shape, dtype=torch.bfloat16, dev=0: On(dev, shape, dtype)
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    ok = dict(q=t(3, 8, 128), k_new=t(3, 2, 128), v_new=t(3, 2, 128), positions=t(3, dtype=i32), cos_sin=t(64, 128, dtype=f32),
              slot_map=t(3, dtype=i64))
    for kw in [dict(q=t(2, 8, 128)), dict(q=t(3, 8, 64)), dict(q=t(3, 8, 128, dtype=f32)), dict(k_new=t(3, 4, 128)), dict(v_new=t(2, 2, 128)),
               dict(positions=t(2, dtype=i32)), dict(positions=t(3, dtype=i64)), dict(cos_sin=t(64, 128)), dict(cos_sin=t(64 * 128, dtype=f32)),
               dict(slot_map=t(3, dtype=i32)), dict(q_out=t(3, 8, 64)), dict(q_out=t(3, 8, 128, dtype=f32)), dict(q=None, q_out=t(3, 8, 128)),
               dict(k_out=t(3, 8, 128)), dict(k_out=t(3, 2, 128, dtype=torch.uint8)), dict(descale_q=t(1)), dict(k_new=t(3, 2, 128, dev=1))]:
        with pytest.raises(b.SplitKVError) as e:
            b.kv_pages_write_rotary(p, **(ok | kw))
        assert e.value.status == b.MLA_ERR_INVALID_ARG, kw
    read = dict(slot_map=t(3, dtype=i64), k_out=t(3, 2, 128), v_out=t(3, 2, 128))
    for kw in [dict(slot_map=t(2, dtype=i64)), dict(k_out=t(3, 3, 128)), dict(v_out=t(3, 2, 64)), dict(k_out=t(3, 2, 128, dtype=f32)),
               dict(descale_v=t(1)), dict(v_out=t(3, 2, 128, dev=1))]:
        with pytest.raises(b.SplitKVError) as e:
            b.kv_pages_read(p, **(read | kw))
        assert e.value.status == b.MLA_ERR_INVALID_ARG, kw
    current[0] = 1
    with pytest.raises(b.SplitKVError, match="pages lie on CUDA device 0"):
        b.kv_pages_read(p, t(3, dtype=i64, dev=1), t(3, 2, 128, dev=1), t(3, 2, 128, dev=1))


# -------------------------------------------------------------------- oracle --

def test_e2m1_codes():
    """Every code decodes and encodes to itself; every middle goes to the even code, its neighbours to the nearer one."""
    c = np.arange(16)
    v = codecs.e2m1_decode(c)
    assert v.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert np.array_equal(codecs.e2m1_encode(v)[1:8], c[1:8]) and np.array_equal(codecs.e2m1_encode(v)[9:], c[9:])
    for k in range(7):
        m = (v[k] + v[k + 1]) / 2
        assert codecs.e2m1_encode(m) == k + (k & 1) and codecs.e2m1_encode(-m) == 8 + k + (k & 1)
        assert codecs.e2m1_encode(np.nextafter(m, 0)) == k and codecs.e2m1_encode(np.nextafter(m, 9)) == k + 1
    assert codecs.e2m1_encode(1e9) == 7 and codecs.e2m1_encode(-np.inf) == 15


def test_four_bit_groups():
    """Round trip of values on the grid; a group's error is at most half a step at its largest; groups do not touch each other."""
    rng = np.random.default_rng(1)
    scales = codecs.e4m3_encode(2.0 ** rng.integers(-3, 6, (5, 8)))
    codes = rng.integers(0, 256, (5, 64)).astype(np.uint8)
    codes[:, ::8] |= 0x07                                        # a 6 in every group
    y = op.four_bit_decode(codes, scales)
    assert np.array_equal(op.four_bit_decode(*op.four_bit_encode(y)), y)
    x = rng.standard_normal((50, 128)) * np.exp(rng.uniform(-3, 3, (50, 1)))
    top = np.repeat(np.abs(x).reshape(50, 8, 16).max(-1), 16, -1)
    assert np.all(np.abs(op.four_bit_decode(*op.four_bit_encode(x)) - x) <= top / 6 * (1 + 2.0 ** -4))
    z = x.copy()
    z[:, 16:32] *= 100
    a, c = op.four_bit_encode(x), op.four_bit_encode(z)
    assert np.array_equal(np.delete(a[0], slice(8, 16), 1), np.delete(c[0], slice(8, 16), 1))
    assert np.array_equal(np.delete(a[1], 1, 1), np.delete(c[1], 1, 1))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R", [32, 96, 128])
def test_rotation_is_a_complex_product(inter, R):
    """Turning by p then by q is turning by p + q; lengths stay; scores depend on the difference of positions only."""
    n = 40
    f = 10000.0 ** (-np.arange(0, R, 2) / R)
    a = np.arange(2 * n)[:, None] * f
    cs = np.concatenate([np.cos(a), np.sin(a)], 1)
    x = np.random.default_rng(R).standard_normal((3, 2, 128))
    y = op.rotate(x, cs, [7, 12, 0], inter)
    assert np.array_equal(y[..., R:], x[..., R:]) and np.allclose(y[2], x[2])
    pair = (lambda v: v[..., 0:R:2] + 1j * v[..., 1:R:2]) if inter else (lambda v: v[..., :R // 2] + 1j * v[..., R // 2:R])
    assert np.allclose(pair(y), pair(x) * np.exp(1j * a[[7, 12, 0]])[:, None])
    assert np.allclose(op.rotate(y, cs, [n, n, n], inter), op.rotate(x, cs, [7 + n, 12 + n, n], inter))
    assert np.array_equal(op.rotate(x, cs, [-1, 2 * n, 1 << 30], inter), x)


def test_head_counts_beyond_int32_arithmetic():
    most, p = 1 << 24, pages(h_kv=(1 << 24) + 1)
    assert status_of("kv_pages_write", ctypes.byref(p), 1, FAKE, FAKE, 256, 128, FAKE, None, None, None) == 1
    assert status_of("kv_pages_read", ctypes.byref(p), 1, FAKE, None, None, FAKE, FAKE, 256, 128, None) == 1
    for h_q, h_kv in ((most + 1, 2), ((1 << 31) - 1, 2), (4, most + 1), (4, (1 << 31) - 1)):
        p = pages(dtype=1, page_stride=4096, row_stride=256, head_stride=128, h_kv=h_kv)
        assert status_of("kv_pages_write_rotary", *(ROTARY | dict(p=ctypes.byref(p), h_q=h_q)).values()) == 1
        if h_kv > most:
            assert status_of("kv_pages_read", ctypes.byref(p), 1, FAKE, None, None, FAKE, FAKE, 256, 128, None) == 1
