"""GPU tests of the paged KV cache (kv_pages_map, kv_pages_write), of attention over its pages (sdpa_paged) and over
packed prompts (sdpa_prompt), against the integer / fp64 oracle in oracle/paged.py. Tolerances: _paged_util."""
import math
import types

import numpy as np
import pytest
import torch

import oracle.paged as op
from _paged_util import (D, TORCH_OUT, U_P, FP32, Paged, check, cu_of, garbage, run_paged, scalar, status_clear, values)
from oracle import codecs
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


# ------------------------------------------------------------------------ map --

def map_case(rng, batch, page, width, spare, q_hi=40, pad=0):
    held = rng.integers(0, page * width + 1, size=batch)
    new = np.where(rng.random(batch) < 0.3, 0, np.clip(held + rng.integers(-2 * page, 2 * page, size=batch), -3, None))
    count = np.minimum(rng.integers(0, q_hi + 1, size=batch), np.maximum(new, 0) + 2)   # some reach before position 0
    n_held = [op.pages(h, page, width) for h in held]
    n_pages = sum(n_held) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((batch, width), -7, dtype=np.int32)
    at = 0
    for i, h in enumerate(n_held):
        table[i, :h] = order[at:at + h]
        at += h
    F = np.full(max(1, n_pages), -5, dtype=np.int32)
    F[:spare] = order[at:]
    cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    return page, held.astype(np.int32), new.astype(np.int32), cu, int(cu[-1]) + pad, table, F, spare


def run_map(case, alias=False, positions=True, times=1):
    page, held, new, cu, total, table, F, n = case
    dev = "cuda"
    t, f = torch.from_numpy(table.copy()).to(dev), torch.from_numpy(F.copy()).to(dev)
    io = torch.tensor([n, 99], dtype=torch.int32, device=dev)
    out = io if alias else torch.zeros(2, dtype=torch.int32, device=dev)
    slots = torch.full((max(total, 1),), 12345, dtype=torch.int64, device=dev)
    pos = torch.full((max(total, 1),), 12345, dtype=torch.int32, device=dev) if positions else None
    for _ in range(times):
        b.kv_pages_map(page, torch.from_numpy(held).to(dev), torch.from_numpy(new).to(dev), torch.from_numpy(cu).to(dev),
                       total, t, f, io, out, slots, pos)
    torch.cuda.synchronize()
    return (t.cpu().numpy(), f.cpu().numpy(), tuple(out.cpu().tolist()), slots.cpu().numpy()[:total],
            pos.cpu().numpy()[:total] if positions else None)


def same_map(got, want):
    for g, w, n in zip(got, want, ("table", "free_pages", "free_out", "slots", "positions")):
        if g is not None:
            assert np.array_equal(np.asarray(g), np.asarray(w)), n


@pytest.mark.parametrize("batch,page,width,spare", [(1, 16, 1, 3), (7, 16, 9, 40), (33, 24, 5, 2), (300, 128, 4, 500),
                                                    (1500, 16, 3, 60), (3, 1, 700, 5000), (16384, 16, 2, 9000)])
def test_map(batch, page, width, spare):
    case = map_case(np.random.default_rng(batch), batch, page, width, spare, pad=5)
    same_map(run_map(case), op.map_pages(*case))


def test_map_runs_out_of_pages_and_says_so():
    page, held, new, cu, total, table, F, n = map_case(np.random.default_rng(5), 40, 16, 12, 0)
    case = (page, held, np.where(new > 0, np.minimum(held, 60) + 130, new).astype(np.int32), cu, total, table, F, n)
    want = op.map_pages(*case)
    assert want[2][1] > 0 and want[2][0] == 0 and (want[0] == -1).any() and (want[3] == -1).any()
    same_map(run_map(case), want)


def test_map_in_place_counter_repeats_and_no_positions():
    case = map_case(np.random.default_rng(6), 50, 32, 6, 100)
    want = op.map_pages(*case)
    same_map(run_map(case, alias=True), want)
    same_map(run_map(case, times=3), want)
    same_map(run_map(case, positions=False), want)


def test_map_of_pages_that_shortage_left_out():
    """A request that shrinks gives back only the pages it has."""
    page, held, new, cu = 16, np.array([64, 10], np.int32), np.array([0, 100], np.int32), np.array([0, 0, 3], np.int32)
    table = np.array([[4, -1, 2, -1, 9, 9, 9], [6, -7, -7, -7, -7, -7, -7]], np.int32)
    case = (page, held, new, cu, 3, table, np.array([1, 0, 0, 0], np.int32), 1)
    want = op.map_pages(*case)
    assert want[2] == (0, 3)
    same_map(run_map(case), want)


@pytest.mark.parametrize("free_in,capacity", [(-4, 8), (100, 8)])
def test_map_takes_a_counter_outside_its_list_as_the_nearest(free_in, capacity):
    F = np.arange(10, 10 + capacity, dtype=np.int32)
    case = (16, np.array([0, 0], np.int32), np.array([40, 20], np.int32), np.array([0, 40, 60], np.int32), 60,
            np.full((2, 4), -1, np.int32), F, free_in)
    same_map(run_map(case), op.map_pages(*case))


def test_map_without_rows():
    case = (16, np.array([5], np.int32), np.array([50], np.int32), np.array([0, 0], np.int32), 0,
            np.full((1, 4), 3, np.int32), np.arange(6, dtype=np.int32), 6)
    same_map(run_map(case), op.map_pages(*case))


# ---------------------------------------------------------------------- write --

def e4m3_of(x, descale):
    y = (x.float() / torch.tensor(descale, dtype=torch.float32)).numpy()
    return codecs.e4m3_encode(y.astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,h_kv,page,layout,fused", [(1, 1, 16, "row", False), (7, 2, 16, "row", True),
                                                         (333, 8, 64, "head", True), (1000, 5, 32, "row", False)])
def test_write(dtype, rows, h_kv, page, layout, fused):
    g = torch.Generator().manual_seed(rows)
    n_pages = -(-rows // page) + 3
    if fused:
        qkv = torch.randn((rows, 4 * h_kv, D), generator=g).to(torch.bfloat16).cuda()
        k, v = qkv[:, 2 * h_kv:3 * h_kv], qkv[:, 3 * h_kv:]
    else:
        k, v = (torch.randn((rows, h_kv, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    t = torch.bfloat16 if dtype == "bf16" else torch.uint8
    shape = (n_pages, page, h_kv, D) if layout == "row" else (n_pages, h_kv, page, D)
    kc, vc = (torch.full(shape, 3, dtype=t, device="cuda") for _ in range(2))
    if layout == "head":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    slots = torch.randperm(n_pages * page, generator=g)[:rows]
    slots[::5] = torch.tensor([-1, n_pages * page, -9, 1 << 40])[torch.arange((rows + 4) // 5) % 4]
    dk, dv = 0.013, 0.37
    b.kv_pages_write(b.kv_pages(kc, vc), k, v, slots.cuda(), scalar(dk, dtype), scalar(dv, dtype))
    torch.cuda.synchronize()
    for cache, x, d in ((kc, k, dk), (vc, v, dv)):
        want = torch.full((n_pages * page, h_kv, D), 3, dtype=t)
        keep = (slots >= 0) & (slots < n_pages * page)
        x = x.cpu()
        new = x if dtype == "bf16" else torch.from_numpy(e4m3_of(x, d)).view(torch.uint8).reshape(x.shape)
        want[slots[keep]] = new[keep]
        got = cache.cpu().reshape(n_pages * page, h_kv, D)
        assert torch.equal(got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


def test_write_special_values_to_e4m3():
    x = torch.zeros((2, 1, D), dtype=torch.bfloat16)
    x[0, 0, :8] = torch.tensor([float("inf"), -float("inf"), 1e30, -500.0, 448.0, 0.0, 1e-9, -0.0], dtype=torch.bfloat16)
    x[1, 0, :2] = torch.tensor([float("nan"), 1.0], dtype=torch.bfloat16)
    kc, vc = (torch.zeros((1, 16, 1, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    b.kv_pages_write(b.kv_pages(kc, vc), x.cuda(), x.cuda(), torch.tensor([0, 1], device="cuda"))
    got = kc.cpu()[0, :2, 0]
    assert got[0, :8].tolist() == [0x7E, 0xFE, 0x7E, 0xFE, 0x7E, 0x00, 0x00, 0x80]
    assert int(got[1, 0]) & 0x7F == 0x7F and int(got[1, 1]) == 0x38


@pytest.mark.parametrize("descale", [0.013, 1.0, 3.0, 1.9999999, 1e-20, 7e30, 2.0 ** -126, 1e-39, 0.0, float("inf")])
def test_write_divides_as_a_division_does(descale):
    """Every bf16 value (all 65,536 bit patterns) against e4m3 of the rounded fp32 quotient, at descales whose quotients
    fall on ties and outside the range of e4m3, of fp32, and of a reciprocal."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).reshape(512, 1, D)
    kc, vc = (torch.zeros((32, 16, 1, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    d = torch.tensor([descale], dtype=torch.float32, device="cuda")
    b.kv_pages_write(b.kv_pages(kc, vc), x.cuda(), x.cuda(), torch.arange(512, device="cuda"), d, d)
    with np.errstate(all="ignore"):
        q = x.reshape(-1).float().numpy() / np.float32(descale)      # IEEE division, subnormals and all
    got = kc.cpu().reshape(-1).numpy()
    nan = np.isnan(q)
    assert np.all((got[nan] & 0x7F) == 0x7F)
    want = codecs.e4m3_encode(np.clip(q[~nan], -448.0, 448.0).astype(np.float64))
    same = (got[~nan] == want) | (((got[~nan] | want) & 0x7F) == 0)   # either zero
    assert same.all(), (x.reshape(-1)[torch.from_numpy(~nan)][torch.from_numpy(~same)][:5], q[~nan][~same][:5])
    assert torch.equal(kc, vc)


def test_write_and_read_behind_32_bit_offsets():
    """Pages that lie more than 2^32 bytes from the base."""
    page, h_kv = 16, 1
    stride = (1 << 30) + 64                     # elements between pages: 2 GB each
    big = torch.zeros(4 * stride, dtype=torch.bfloat16, device="cuda")
    kc = big.as_strided((4, page, h_kv, D), (stride, 2 * D, D, 1))
    vc = big.as_strided((4, page, h_kv, D), (stride, 2 * D, D, 1), D)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((40, h_kv, D), generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[3, 0, 2]], dtype=torch.int32)
    pos = torch.arange(40)
    slots = table[0].long()[pos // page] * page + pos % page
    pages = b.kv_pages(kc, vc)
    b.kv_pages_write(pages, k.cuda(), v.cuda(), slots.cuda())
    assert torch.equal(kc[3, :, 0].cpu(), k[:16, 0]) and torch.equal(vc[2, :8, 0].cpu(), v[32:, 0])
    q = torch.randn((2, 4, D), generator=g).to(torch.bfloat16)
    plan = b.sdpa_paged_plan(1, 4, 1, D, "bf16", 2, 2, 40, force_splits=1)
    out = torch.empty((2, 4, D), device="cuda")
    b.sdpa_paged(plan, 2, q.cuda(), pages, table.cuda(), torch.tensor([40], dtype=torch.int32, device="cuda"),
                 cu_of([2]).cuda(), None, None, None, 0.1, "f32", 1.0, out)
    torch.cuda.synchronize()
    status_clear()
    seen = torch.ones((2, 40), dtype=torch.bool).numpy()
    seen[0, 39] = False
    ref = op.attend(q.double().numpy(), k.double().numpy(), v.double().numpy(), seen, 0.1)
    check(out.cpu(), None, None, ref, "bf16")
    del big, kc, vc
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- paged attention --

def paged_case(dtype, sq, kv, h_q, h_kv, page, seed=0, **kw):
    c = Paged(dtype, kv, h_kv, page, seed, **kw)
    q, dq = values(torch.Generator().manual_seed(seed + 1), (max(1, sum(sq)), h_q, D), dtype)
    return c, q, dq, cu_of(sq)


def go(dtype, sq, kv, h_q, h_kv, page, seed=0, layout="row", **kw):
    c, q, dq, cu = paged_case(dtype, sq, kv, h_q, h_kv, page, seed, layout=layout)
    ref = c.reference(q, dq, cu, kw.get("scale", 1 / math.sqrt(D)))
    check(*run_paged(c, q, dq, cu, h_q, **kw), ref, dtype, kw.get("out_dtype", "f32"), kw.get("inv_scale", 1.0))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("sq,kv", [
    ([1], [1]), ([1], [16]), ([1], [17]), ([1, 1, 1, 1], [5, 127, 129, 1000]), ([1] * 20, list(range(90, 490, 20))),
    ([2, 3, 1, 4], [30, 300, 700, 4]),
])
def test_decode(dtype, page, sq, kv):
    go(dtype, sq, kv, 8, 2, page, seed=page + len(sq))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("sq,kv", [
    ([5, 40, 1], [129, 300, 600]), ([33, 64, 100], [33, 64, 800]), ([300], [300]), ([257, 1, 129], [700, 90, 130]),
])
def test_chunk(dtype, page, sq, kv):
    go(dtype, sq, kv, 8, 2, page, seed=page + len(sq))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (8, 8), (5, 1), (14, 2), (16, 1), (24, 2), (64, 1), (128, 1), (100, 1)])
def test_group_sizes(dtype, h_q, h_kv):
    go(dtype, [1, 1, 1], [100, 257, 33], h_q, h_kv, 32, seed=h_q)
    go(dtype, [3, 17, 70], [100, 257, 70], h_q, h_kv, 32, seed=h_q + 1)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("S", [1, 2, 3, 7, 64])
def test_forced_splits(dtype, S):
    go(dtype, [1, 1, 1], [1000, 130, 5], 8, 2, 16, seed=S, force_splits=S)
    go(dtype, [40, 1, 150], [1000, 130, 150], 8, 2, 16, seed=S, force_splits=S)


@pytest.mark.parametrize("num_sms", [1, 5, 40])
def test_split_counts_from_the_lengths(num_sms):
    """Fewer SMs in the plan, fewer splits: same results."""
    go("e4m3", [1] * 6, [1900, 100, 700, 1, 1500, 33], 8, 2, 16, seed=1, num_sms=num_sms)
    go("bf16", [9, 30, 1], [1900, 100, 700], 8, 2, 16, seed=2, num_sms=num_sms)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("num_sms", [1, 3, 20])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_shares_that_cross_sequences(dtype, num_sms, page):
    """CTAs that take the end of one sequence, several whole ones and the start of another; more KV heads than CTAs."""
    rng = np.random.default_rng(num_sms)
    kv = [int(x) for x in rng.integers(0, 700, 45)]
    sq = [int(x) for x in rng.integers(0, 4, 45)]
    go(dtype, sq, kv, 8, 2, page, seed=num_sms, num_sms=num_sms, max_q=2)
    go(dtype, sq[:9], kv[:9], 10, 5, page, seed=num_sms, num_sms=num_sms, max_q=2)


@pytest.mark.parametrize("num_sms", [1, 3, 20])
@pytest.mark.parametrize("h_q,h_kv", [(8, 2), (10, 5), (96, 1)])
def test_chunk_shares_that_cross_sequences(num_sms, h_q, h_kv):
    """e4m3 over long tables: ranges that end in a sequence's query tiles, rows that see no key, one row block or two."""
    rng = np.random.default_rng(num_sms + h_q)
    kv = [int(x) for x in rng.integers(0, 900, 12)] + [0, 40, 1000]
    sq = [int(x) for x in rng.integers(0, 260, 12)] + [9, 90, 0]
    go("e4m3", sq, kv, h_q, h_kv, 32, seed=num_sms, num_sms=num_sms, max_kv=9000)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_q,max_kv", [(2, 60), (2, 500), (40, 60), (40, 500), (40, 9000)])
def test_hundreds_of_short_sequences(dtype, max_q, max_kv):
    """Job searches over many groups of sequences, empty ones among them."""
    rng = np.random.default_rng(max_q + max_kv)
    sq = [int(x) for x in rng.integers(0, 4, 700)]
    kv = [int(x) for x in rng.integers(0, 60, 700)]
    sq[300], kv[300] = (3, 400) if max_q == 2 else (150, 480)
    go(dtype, sq, kv, 8, 2, 16, seed=7, max_q=max_q, max_kv=max_kv)
    if max_kv == 60:
        run_prompt(dtype, sq, [max(n, m) for n, m in zip(sq, kv)], 8, 2, seed=7)


def test_decode_work_counted_in_coarser_units():
    """Tables so wide that the key tiles of all sequences could pass 32 bits: a unit of work is several tiles."""
    g = torch.Generator().manual_seed(5)
    batch, page, width = 600, 65536, 1 << 15
    c = types.SimpleNamespace(dtype="bf16", dk=1.0, dv=1.0)
    c.k, c.v = (torch.randn((2, page, 1, D), generator=g).to(torch.bfloat16) for _ in range(2))
    c.table = torch.full((batch, width), -1, dtype=torch.int32)
    c.table[:, 0] = torch.arange(batch) % 2
    c.kv_lens = torch.randint(0, 3000, (batch,), generator=g, dtype=torch.int32)
    c.kv_lens[7], c.kv_lens[500] = 60000, 20000
    q, dq = values(g, (batch, 4, D), "bf16")
    cu = cu_of([1] * batch)
    scale = 1 / math.sqrt(D)
    k, v = c.k.double().numpy(), c.v.double().numpy()
    ref = op.paged_attention(q.double().numpy(), k, v, c.table.numpy(), c.kv_lens.numpy(), cu.numpy(), scale)
    check(*run_paged(c, q, dq, cu, 4), ref, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("S", [0, 1, 3])
def test_rows_without_keys_and_empty_sequences(dtype, S):
    """More new tokens than keys (the first queries see nothing), no keys at all, no new tokens."""
    go(dtype, [6, 4, 0, 1, 0], [3, 0, 50, 20, 0], 8, 2, 16, force_splits=S)
    go(dtype, [160, 40, 0, 1], [100, 0, 50, 20], 8, 2, 16, force_splits=S)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("sq", [[1, 1, 1], [20, 70, 1]])
def test_pages_that_are_missing(dtype, sq):
    c, q, dq, cu = paged_case(dtype, sq, [150, 300, 64], 8, 2, 16, seed=3)
    c.table[0, 2] = -1
    c.table[1, 7] = c.num_pages
    c.table[1, 8] = 2 ** 31 - 1
    c.table[2, :] = -2 ** 31          # every key of the sequence is missing
    ref = c.reference(q, dq, cu, 1 / math.sqrt(D))
    for S in (0, 1, 2):
        check(*run_paged(c, q, dq, cu, 8, force_splits=S), ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("sq", [[1, 1], [30, 45]])
@pytest.mark.parametrize("S", [1, 3])
def test_nan_scores_give_nan_rows_and_touch_no_other(dtype, sq, S):
    """Sequence 1's keys are NaN: its O and LSE are NaN however it is split, sequence 0's are what they were."""
    c, q, dq, cu = paged_case(dtype, sq, [150, 500], 8, 2, 16, seed=9)
    O, L, A = c.reference(q, dq, cu, 1 / math.sqrt(D))
    held = c.table[1][c.table[1] >= 0].long()
    c.k[held] = float("nan") if dtype == "bf16" else 0x7F
    out, lse, _ = run_paged(c, q, dq, cu, 8, force_splits=S, amax=False)
    n = sq[0]
    check(out[:n], lse[:n], None, (O[:n], L[:n], A[:n]), dtype)
    assert torch.isnan(out[n:]).all() and torch.isnan(lse[n:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("sq", [[1, 1], [30, 45]])
@pytest.mark.parametrize("S", [0, 1, 3])
def test_padded_batch_rows_are_left_alone(dtype, sq, S):
    c, q, dq, cu = paged_case(dtype, sq, [150, 300], 8, 2, 16, seed=4)
    O, L, A = c.reference(q, dq, cu, 1 / math.sqrt(D))
    n = int(cu[-1])
    check(*run_paged(c, q, dq, cu, 8, rows=n + 37, force_splits=S), (O, L, A), dtype, untouched_from=n)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype,inv_scale", [("bf16", 1.0), ("e4m3", 64.0)])
@pytest.mark.parametrize("sq", [[1, 1], [30, 200]])
def test_output_types(dtype, out_dtype, inv_scale, sq):
    for S in (1, 0):
        go(dtype, sq, [150, 300], 8, 2, 16, out_dtype=out_dtype, inv_scale=inv_scale, force_splits=S)


@pytest.mark.parametrize("sq", [[1, 1], [30, 200]])
def test_head_major_pages_and_no_lse(sq):
    for dtype in ("bf16", "e4m3"):
        go(dtype, sq, [150, 300], 8, 2, 32, layout="head")
        go(dtype, sq, [150, 300], 8, 2, 32, lse=False, amax=False)


@pytest.mark.parametrize("sq", [[1, 1], [30, 200]])
@pytest.mark.parametrize("page", [16, 128])
def test_page_strides(sq, page):
    """Caches of one head, head-major pages, and pages inside a wider allocation (heads, rows and pages apart)."""
    for dtype in ("bf16", "e4m3"):
        go(dtype, sq, [150, 300], 4, 1, page, seed=page)
        go(dtype, sq, [150, 300], 8, 2, page, seed=page, layout="head")
        c, q, dq, cu = paged_case(dtype, sq, [150, 300], 8, 2, page, seed=page)
        ref = c.reference(q, dq, cu, 1 / math.sqrt(D))
        for x in ("k", "v"):
            t = getattr(c, x)
            wide = torch.empty((t.shape[0], page + 3, 2, 256), dtype=t.dtype)
            garbage(wide)
            wide[:, :page, :, :D] = t
            setattr(c, x, wide)

        class View:     # keeps the strides on the device
            def __init__(self, x):
                self.x, self.shape = x, (x.shape[0], page, 2, D)

            def to(self, dev):
                return self.x.to(dev)[:, :page, :, :D]

        c.k, c.v = View(c.k), View(c.v)
        check(*run_paged(c, q, dq, cu, 8), ref, dtype)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("sq", [[1, 1], [30, 200]])
def test_scales(scale, sq):
    """Zero and negative scales, and one that makes the softmax nearly one-hot. The products of e4m3 codes are exact,
    their sum is not: 128 fp32 additions (each up to 2^-24 of the partial sums, at most sum |q k| = 128 * 2/pi = 82 for
    N(0, 1) values) put 128 * 2^-24 * 82 * |scale| of natural-log error on a score, and that is p's relative error:
    1.9e-3 at scale 3."""
    c, q, dq, cu = paged_case("e4m3", sq, [150, 300], 8, 2, 16, seed=11)
    ref = c.reference(q, dq, cu, scale)
    out, lse, amax = run_paged(c, q, dq, cu, 8, scale=scale)
    if scale == 3.0:
        # scores up to 3 * 60 / ln 2 = 260 in log2 units: one fp32 rounding of the scaled score is 2^-16, two of them
        # and the sum 2^-14.5 in p and in the LSE
        ok = np.isfinite(ref[1])
        assert np.abs(lse.double().numpy()[ok] - ref[1][ok]).max() <= 2.0 ** -14
        lse = None
    check(out, lse, amax, ref, "e4m3", score_err=128 * 2.0 ** -24 * 82 * abs(scale))


def test_q_strides():
    """Q as the first heads of a fused projection's rows."""
    for sq in ([1, 1], [30, 200]):
        c, q, dq, cu = paged_case("bf16", sq, [150, 300], 8, 2, 16, seed=8)
        ref = c.reference(q, dq, cu, 1 / math.sqrt(D))
        wide = torch.full((q.shape[0], 12, D), float("nan"), dtype=torch.bfloat16)
        wide[:, :8] = q
        check(*run_paged_view(c, wide.cuda()[:, :8], cu), ref, "bf16")


def run_paged_view(c, qd, cu, stream=None, ws=None, plan=None):
    total, h_q = qd.shape[:2]
    plan = plan or b.sdpa_paged_plan(len(c.kv_lens), h_q, c.k.shape[2], D, c.dtype, int((cu[1:] - cu[:-1]).max()), total,
                                     int(c.kv_lens.max()))
    if ws is None and plan.workspace_bytes:
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out, L = torch.empty((total, h_q, D), device="cuda"), torch.empty((total, h_q), device="cuda")
    b.sdpa_paged(plan, total, qd, b.kv_pages(c.k.cuda(), c.v.cuda()), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), None,
                 None, None, 1 / math.sqrt(D), "f32", 1.0, out, L, None, ws)
    torch.cuda.synchronize()
    status_clear()
    return out.cpu(), L.cpu(), None


def test_longer_sequences_than_the_plan_expects():
    go("bf16", [1, 1], [900, 1500], 8, 2, 16, max_kv=20)
    go("e4m3", [40, 1], [900, 1500], 8, 2, 16, max_kv=20)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_more_tokens_than_the_plan_expects(dtype):
    """A plan for one token of 8 heads a KV head (16-row jobs), called with 3 to 40 of them."""
    assert b.sdpa_paged_plan(2, 16, 2, D, dtype, 1, 4, 300).row_kernel == 1
    go(dtype, [3, 1, 40], [150, 300, 90], 16, 2, 16, max_q=1)
    go(dtype, [3, 1, 40], [150, 300, 90], 16, 2, 16, max_q=1, force_splits=3)


@pytest.mark.parametrize("sq", [[1, 1, 1], [20, 70, 1]])
def test_graph_replayed_with_other_lengths(sq):
    """A captured call reads the lengths, tables and counts of the replay, not of the capture."""
    c, q, dq, cu = paged_case("bf16", sq, [1500, 300, 64], 8, 2, 16, seed=3)
    n, h_q = int(cu[-1]), 8
    plan = b.sdpa_paged_plan(3, h_q, 2, D, "bf16", max(sq), n, 1500)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda") if plan.workspace_bytes else None
    out, L = torch.empty((n, h_q, D), device="cuda"), torch.empty((n, h_q), device="cuda")
    kc, vc, table, lens, cud, qd = c.k.cuda(), c.v.cuda(), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), q.cuda()
    pages = b.kv_pages(kc, vc)
    call = lambda: b.sdpa_paged(plan, n, qd, pages, table, lens, cud, None, None, None, 0.1, "f32", 1.0, out, L, None, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([1500, 300, 64], [80, 290, 20], [1400, 70, 60]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        c.kv_lens = torch.tensor(new, dtype=torch.int32)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        status_clear()
        check(out.cpu(), L.cpu(), None, c.reference(q, dq, cu, 0.1), "bf16")


@pytest.mark.parametrize("sq", [[1, 1, 1], [20, 70, 1]])
def test_two_streams_with_workspaces_of_their_own(sq):
    cases = [paged_case("bf16", sq, [1500, 300, 64], 8, 2, 16, seed=s) for s in (3, 4)]
    state = []
    for c, q, dq, cu in cases:
        n = int(cu[-1])
        plan = b.sdpa_paged_plan(3, 8, 2, D, "bf16", max(sq), n, 1500)
        ws = torch.empty(max(16, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
        state.append((plan, n, q.cuda(), c.k.cuda(), c.v.cuda(), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(),
                      torch.empty((n, 8, D), device="cuda"), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for plan, n, q, k, v, t, l, cu, out, ws, st in state:
            b.sdpa_paged(plan, n, q, b.kv_pages(k, v), t, l, cu, None, None, None, 0.1, "f32", 1.0, out, None, None, ws,
                         stream=st)
    torch.cuda.synchronize()
    status_clear()
    for (c, q, dq, cu), s in zip(cases, state):
        check(s[8].cpu(), None, None, c.reference(q, dq, cu, 0.1), "bf16")


@pytest.mark.parametrize("S", [0, 2])
@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [4, 9, 2, 12], [0, 200, 10, 250], [-5, 7, 1 << 20, 3], [0, 0, 0, 0]])
def test_offsets_that_decrease_touch_nothing_outside(cu, S):
    """Rows are undefined then, but every write stays inside the buffers and every wait ends."""
    for dtype in ("bf16", "e4m3"):
        c, q, dq, _ = paged_case(dtype, [80, 80, 100], [500, 300, 64], 8, 2, 16, seed=6)
        total = 260
        plan = b.sdpa_paged_plan(3, 8, 2, D, dtype, 1 if max(cu) < 50 else 100, total, 500, force_splits=S)
        ws = torch.empty(max(16, plan.workspace_bytes) + 4096, dtype=torch.uint8, device="cuda")
        ws.fill_(0x5A)
        out = torch.full((total + 8, 8, D), 7.0, device="cuda")
        b.sdpa_paged(plan, total, q.cuda(), b.kv_pages(c.k.cuda(), c.v.cuda()), c.table.cuda(), c.kv_lens.cuda(),
                     torch.tensor(cu, dtype=torch.int32, device="cuda"), scalar(dq, dtype), scalar(c.dk, dtype),
                     scalar(c.dv, dtype), 0.1, "f32", 1.0, out, None, None, ws)
        torch.cuda.synchronize()
        status_clear()
        assert torch.all(out[total:] == 7.0) and torch.all(ws[-4096:] == 0x5A)


def test_repeated_calls_give_the_same_bits():
    for dtype, sq in (("bf16", [1, 1, 1]), ("e4m3", [1, 1, 1]), ("bf16", [20, 70, 1]), ("e4m3", [20, 70, 1])):
        c, q, dq, cu = paged_case(dtype, sq, [1500, 300, 64], 8, 2, 16, seed=3)
        a = run_paged(c, q, dq, cu, 8)
        z = run_paged(c, q, dq, cu, 8)
        assert torch.equal(a[0], z[0]) and torch.equal(a[1], z[1]) and a[2] == z[2]


@pytest.mark.parametrize("dtype,sq", [("bf16", [1, 1, 1]), ("bf16", [20, 300, 1]), ("e4m3", [20, 300, 1])])
def test_waits_that_run_out_end_the_call_with_a_status(dtype, sq):
    """With a limit far below a step's latency the kernels' waits run out: the call ends, says so, and the next one is
    right again. (100 ns, the shortest limit, and sequences long enough that their loads queue for memory. The 16-row
    kernel computes on e4m3 blocks for longer than their loads take, so there no wait need run out.)"""
    c, q, dq, cu = paged_case(dtype, sq, [20000, 9000, 64], 8, 2, 16, seed=3)
    ref = c.reference(q, dq, cu, 1 / math.sqrt(D))
    n = int(cu[-1])
    plan = b.sdpa_paged_plan(3, 8, 2, D, dtype, max(sq), n, 20000)
    ws = torch.empty(max(16, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    out = torch.empty((n, 8, D), device="cuda")
    args = [q.cuda(), b.kv_pages(c.k.cuda(), c.v.cuda()), c.table.cuda(), c.kv_lens.cuda(), cu.cuda()]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        b.mla_set_wait_limit_ns(100)
        flush.fill_(1)          # the keys are not in the cache
        b.sdpa_paged(plan, n, *args, scalar(dq, dtype), scalar(c.dk, dtype), scalar(c.dv, dtype), 0.1, "f32", 1.0, out, None,
                     None, ws)
        torch.cuda.synchronize()
        st, site = b.mla_get_status()
        assert st & b.MLA_STATUS_TIMEOUT and site != 0
    finally:
        b.mla_set_wait_limit_ns(0)
    check(*run_paged(c, q, dq, cu, 8), ref, dtype)


def test_waits_that_run_out_in_an_equal_share():
    """As above, in chunks over long e4m3 tables. (Few CTAs of the 16-row kernel have their loads in time: no wait of theirs
    need run out.)"""
    dtype, sq, kv = "e4m3", [40, 300, 70], [9000, 7000, 8000]
    c, q, dq, cu = paged_case(dtype, sq, kv, 8, 2, 16, seed=3)
    ref = c.reference(q, dq, cu, 1 / math.sqrt(D))
    n = int(cu[-1])
    plan = b.sdpa_paged_plan(len(sq), 8, 2, D, dtype, max(sq), n, 9000, num_sms=4)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty((n, 8, D), device="cuda")
    args = [q.cuda(), b.kv_pages(c.k.cuda(), c.v.cuda()), c.table.cuda(), c.kv_lens.cuda(), cu.cuda()]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        b.mla_set_wait_limit_ns(100)
        flush.fill_(1)          # the keys are not in the cache
        b.sdpa_paged(plan, n, *args, scalar(dq, dtype), scalar(c.dk, dtype), scalar(c.dv, dtype), 0.1, "f32", 1.0, out, None,
                     None, ws)
        torch.cuda.synchronize()
        st, site = b.mla_get_status()
        assert st & b.MLA_STATUS_TIMEOUT and site != 0
    finally:
        b.mla_set_wait_limit_ns(0)
    check(*run_paged(c, q, dq, cu, 8, num_sms=4, max_kv=9000), ref, dtype)


# ------------------------------------------------------------------------- prompt --

def run_prompt(dtype, sq, kv, h_q, h_kv, seed=0, scale=1 / math.sqrt(D), out_dtype="f32", inv_scale=1.0, fused=False, pad=0,
               tail=0):
    g = torch.Generator().manual_seed(seed)
    n, m = max(1, sum(sq)), max(1, sum(kv))
    t = torch.bfloat16 if dtype == "bf16" else torch.uint8
    if fused:
        qkv, dq = values(g, (max(n, m) + pad, h_q + 2 * h_kv, D), dtype)
        dk = dv = dq
        q, k, v = qkv[:n + pad, :h_q], qkv[:m + tail, h_q:h_q + h_kv], qkv[:m + tail, h_q + h_kv:]
    else:
        q, dq = values(g, (n + pad, h_q, D), dtype)
        k, dk = values(g, (m + tail, h_kv, D), dtype)
        v, dv = values(g, (m + tail, h_kv, D), dtype)
        if tail:
            garbage(k[m:])
            garbage(v[m:])
    cu, ck = cu_of(sq), cu_of(kv)
    dev = "cuda"
    if fused:
        base = qkv.to(dev)
        qd, kd, vd = base[:n + pad, :h_q], base[:m + tail, h_q:h_q + h_kv], base[:m + tail, h_q + h_kv:]
    else:
        qd, kd, vd = q.to(dev), k.to(dev), v.to(dev)
    out = torch.full((n + pad, h_q, D), 7, dtype=TORCH_OUT[out_dtype], device=dev)
    L, M = torch.full((n + pad, h_q), 7.0, device=dev), torch.full((1,), -1.0, device=dev)
    b.sdpa_prompt(len(sq), qd, kd, vd, cu.to(dev), ck.to(dev), scalar(dq, dtype), scalar(dk, dtype), scalar(dv, dtype),
                  scale, out_dtype, inv_scale, out, L, M)
    torch.cuda.synchronize()
    status_clear()
    ref = op.prompt_attention(op.decode_values(q, dq), op.decode_values(k, dk), op.decode_values(v, dv), cu.numpy(),
                              ck.numpy(), scale)
    check(out.cpu(), L.cpu(), float(M.cpu()[0]), ref, dtype, out_dtype, inv_scale, untouched_from=sum(sq))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255, 1, 257], [64, 65, 300, 7], [1000], [33] * 40])
def test_prompt(dtype, lens):
    run_prompt(dtype, lens, lens, 8, 2, seed=len(lens))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [40, 100, 170])
def test_many_short_jobs_a_cta(dtype, n):
    """Several jobs a CTA, each of two row blocks over one or two key tiles of which the last ends in the sequence: the V
    loads run ahead over more than one job's ragged end."""
    run_prompt(dtype, [n] * 70, [n] * 70, 32, 8, seed=n)
    go(dtype, [n] * 70, [n + 5] * 70, 32, 8, 16, seed=n, force_splits=1)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (8, 8), (5, 1), (14, 2), (16, 1), (64, 1), (128, 1)])
def test_prompt_groups(dtype, h_q, h_kv):
    run_prompt(dtype, [200, 3, 97], [200, 3, 97], h_q, h_kv, seed=h_q)


@pytest.mark.parametrize("out_dtype,inv_scale", [("f32", 1.0), ("bf16", 1.0), ("e4m3", 64.0)])
@pytest.mark.parametrize("max_q", [4, 200])
def test_outputs_that_are_16_byte_aligned_only(out_dtype, inv_scale, max_q):
    """Rows of out on odd 16-byte boundaries: unsplit rows of either kernel, split ones through the combine; prompts."""
    g = torch.Generator().manual_seed(3)
    scale = 1 / math.sqrt(D)
    sq, kv = ([1, 3], [300, 40]) if max_q == 4 else ([20, 200], [300, 210])
    c, q, dq, cu = paged_case("bf16", sq, kv, 8, 2, 16, seed=3)
    ref = c.reference(q, dq, cu, scale)
    n, dev, pages = sum(sq), "cuda", b.kv_pages(c.k.cuda(), c.v.cuda())
    esz = torch.tensor([], dtype=TORCH_OUT[out_dtype]).element_size()
    for S in (1, 3):
        plan = b.sdpa_paged_plan(2, 8, 2, D, "bf16", max_q, n, 300, force_splits=S)
        ws = torch.empty(max(16, plan.workspace_bytes), dtype=torch.uint8, device=dev)
        big = torch.full((16 // esz + n * 8 * D + 16 // esz,), 7, dtype=TORCH_OUT[out_dtype], device=dev)
        out = big[16 // esz:-(16 // esz)].view(n, 8, D)
        assert out.data_ptr() % 32 == 16
        b.sdpa_paged(plan, n, q.to(dev), pages, c.table.to(dev), c.kv_lens.to(dev), cu.to(dev), None, None, None, scale,
                     out_dtype, inv_scale, out, None, None, ws)
        torch.cuda.synchronize()
        status_clear()
        check(out.cpu(), None, None, ref, "bf16", out_dtype, inv_scale)
        assert torch.all(big[:16 // esz].float() == 7) and torch.all(big[-(16 // esz):].float() == 7)
    k, v = (torch.randn((n, 2, D), generator=g).to(torch.bfloat16) for _ in range(2))
    out.fill_(7)
    b.sdpa_prompt(2, q.to(dev), k.to(dev), v.to(dev), cu.to(dev), cu.to(dev), None, None, None, scale,
                  out_dtype, inv_scale, out)
    torch.cuda.synchronize()
    status_clear()
    ref = op.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), cu.numpy(), cu.numpy(), scale)
    check(out.cpu(), None, None, ref, "bf16", out_dtype, inv_scale)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompt_behind_a_prefix_and_with_fewer_keys(dtype):
    run_prompt(dtype, [20, 150, 0, 300, 9], [200, 150, 40, 100, 0], 8, 2)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype,inv_scale", [("bf16", 1.0), ("e4m3", 64.0)])
def test_prompt_output_types(dtype, out_dtype, inv_scale):
    run_prompt(dtype, [200, 77], [200, 77], 8, 2, out_dtype=out_dtype, inv_scale=inv_scale)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompt_strides_padding_and_what_lies_behind(dtype):
    run_prompt(dtype, [200, 77], [200, 77], 8, 2, fused=True)
    run_prompt(dtype, [200, 77], [200, 77], 8, 2, pad=300)
    run_prompt(dtype, [200, 77], [200, 77], 8, 2, tail=90)


def test_prompt_values_of_the_next_sequence_do_not_leak():
    """Sequence 1 holds NaN and infinity; sequence 0, whose last tile ends inside it, must not see them."""
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((300, h, D), generator=g).to(torch.bfloat16) for h in (8, 2, 2))
    k[100:] = float("nan")
    v[100:] = float("inf")
    cu = cu_of([100, 200])
    out = torch.empty((300, 8, D), device="cuda")
    b.sdpa_prompt(2, q.cuda(), k.cuda(), v.cuda(), cu.cuda(), cu.cuda(), None, None, None, 0.1, "f32", 1.0, out)
    torch.cuda.synchronize()
    status_clear()
    ref = op.prompt_attention(q[:100].double().numpy(), k[:100].double().numpy(), v[:100].double().numpy(),
                              np.array([0, 100]), np.array([0, 100]), 0.1)
    check(out[:100].cpu(), None, None, ref, "bf16")


def test_prompt_on_another_stream_and_repeated():
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((900, h, D), generator=g).to(torch.bfloat16) for h in (8, 2, 2))
    cu = cu_of([300, 17, 583])
    ref = op.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), cu.numpy(), cu.numpy(), 0.1)
    qd, kd, vd, cd = q.cuda(), k.cuda(), v.cuda(), cu.cuda()
    outs = [torch.empty((900, 8, D), device="cuda") for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        with torch.cuda.stream(streams[i % 2]):
            b.sdpa_prompt(3, qd, kd, vd, cd, cd, None, None, None, 0.1, "f32", 1.0, o)
    torch.cuda.synchronize()
    status_clear()
    check(outs[0].cpu(), None, None, ref, "bf16")
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_prompt_in_a_graph():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((300, h, D), generator=g).to(torch.bfloat16) for h in (8, 2, 2))
    out = torch.empty((300, 8, D), device="cuda")
    qd, kd, vd, cu = q.cuda(), k.cuda(), v.cuda(), cu_of([100, 200]).cuda()
    call = lambda: b.sdpa_prompt(2, qd, kd, vd, cu, cu, None, None, None, 0.1, "f32", 1.0, out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([100, 200], [7, 293], [300, 0]):
        cu.copy_(cu_of(lens))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        status_clear()
        ref = op.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), cu_of(lens).numpy(),
                                  cu_of(lens).numpy(), 0.1)
        check(out.cpu(), None, None, ref, "bf16")


# ----------------------------------------------------------------- a server's steps --

@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_steps_of_a_server(dtype):
    """Prompts, chunks, decode steps and an end, through the map, the append and the attention over pages, with the
    attention of whole prompts over the same keys beside them."""
    h_q, h_kv, page, W, cap = 8, 2, 16, 40, 90
    g = torch.Generator().manual_seed(5)
    rng = np.random.default_rng(5)
    dev, B = "cuda", 3
    t = torch.bfloat16 if dtype == "bf16" else torch.uint8
    kc, vc = (torch.empty((cap, page, h_kv, D), dtype=t) for _ in range(2))
    garbage(kc)
    garbage(vc)
    kc, vc = kc.to(dev), vc.to(dev)
    pages = b.kv_pages(kc, vc)
    descale = 0.012
    ds = scalar(descale, dtype)
    table = torch.full((B, W), -1, dtype=torch.int32, device=dev)
    free = torch.from_numpy(rng.permutation(cap).astype(np.int32)).to(dev)
    count = torch.tensor([cap, 0], dtype=torch.int32, device=dev)
    have = [0, 0, 0]
    hist = [[torch.zeros((0, h_kv, D), dtype=t) for _ in range(2)] for _ in range(B)]
    steps = [([130, 7, 40], None), ([1, 1, 1], None), ([60, 1, 3], None), ([1, 1, 0], 2), ([1, 200, 9], None), ([1, 1, 1], 0)]
    for add, ends in steps:
        held = list(have)
        if ends is not None:
            have[ends] = 0
            add = [0 if i == ends else n for i, n in enumerate(add)]
            hist[ends] = [torch.zeros((0, h_kv, D), dtype=t) for _ in range(2)]
        have = [a + n for a, n in zip(have, add)]
        n = sum(add)
        cu = cu_of(add)
        xk, xv = (torch.randn((n, h_kv, D), generator=g).to(torch.bfloat16) for _ in range(2))
        q, dq = values(g, (n, h_q, D), dtype)
        slots = torch.empty(n, dtype=torch.int64, device=dev)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        b.kv_pages_map(page, i32(held), i32(have), cu.to(dev), n, table, free, count, count, slots)
        b.kv_pages_write(pages, xk.to(dev), xv.to(dev), slots, ds, ds)
        out, L = torch.empty((n, h_q, D), device=dev), torch.empty((n, h_q), device=dev)
        plan = b.sdpa_paged_plan(B, h_q, h_kv, D, dtype, max(add), n, max(have))
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=dev) if plan.workspace_bytes else None
        b.sdpa_paged(plan, n, q.to(dev), pages, table, i32(have), cu.to(dev), scalar(dq, dtype), ds, ds, 0.1, "f32", 1.0,
                     out, L, None, ws)
        torch.cuda.synchronize()
        status_clear()
        assert int(count[1]) == 0 and int(count[0]) == cap - sum(-(-x // page) for x in have)
        for i in range(B):
            for w, x in ((0, xk), (1, xv)):
                x = x[int(cu[i]):int(cu[i + 1])]
                if dtype == "e4m3":
                    x = torch.from_numpy(e4m3_of(x, descale)).view(torch.uint8).reshape(x.shape)
                hist[i][w] = torch.cat([hist[i][w], x])
        K, V = (torch.cat([hist[i][w] for i in range(B)]) for w in (0, 1))
        ck = cu_of(have)
        d = 1.0 if dtype == "bf16" else descale
        ref = op.prompt_attention(op.decode_values(q, dq), op.decode_values(K, d), op.decode_values(V, d), cu.numpy(),
                                  ck.numpy(), 0.1)
        check(out.cpu(), L.cpu(), None, ref, dtype)
        out2 = torch.empty((n, h_q, D), device=dev)
        b.sdpa_prompt(B, q.to(dev), K.to(dev), V.to(dev), cu.to(dev), ck.to(dev), scalar(dq, dtype), ds, ds, 0.1, "f32",
                      1.0, out2)
        torch.cuda.synchronize()
        status_clear()
        check(out2.cpu(), None, None, ref, dtype)
