"""GPU tests of attention over a 4-bit paged cache, and of a server's steps that rotate, append and attend, against the fp64
oracle. Tolerances: _paged_util, P in f16."""
import math

import numpy as np
import pytest
import torch

import oracle.paged as op
from _four_bit_util import Paged4, caches, f32, run4, table_of
from _paged_util import D, check, cu_of, status_clear
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu
P_TYPE = "e4m3"      # of _paged_util's bounds: P in f16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


def queries(n, h_q, seed, scale=1.0):
    return (torch.randn((max(1, n), h_q, D), generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def go(sq, kv, h_q, h_kv, page, seed=0, layout="row", **kw):
    c, q, cu = Paged4(kv, h_kv, page, seed, layout), queries(sum(sq), h_q, seed + 1), cu_of(sq)
    ref = c.reference(q, cu, kw.get("scale", 1 / math.sqrt(D)))
    check(*run4(c, q, cu, h_q, **kw), ref, P_TYPE, kw.get("out_dtype", "f32"), kw.get("inv_scale", 1.0))


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("sq,kv", [
    ([1], [1]), ([1], [16]), ([1], [17]), ([1], [63]), ([1], [64]), ([1], [65]), ([1, 1, 1, 1], [5, 127, 129, 1000]),
    ([1] * 20, list(range(90, 490, 20))), ([2, 3, 1, 4], [30, 300, 700, 4]), ([2, 2, 1], [30, 300, 700]),
])
def test_decode(page, sq, kv):
    go(sq, kv, 8, 2, page, seed=page + len(sq))


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("sq,kv", [
    ([5, 40, 1], [129, 300, 600]), ([33, 64, 100], [33, 64, 800]), ([300], [300]), ([257, 1, 129], [700, 90, 130]),
])
def test_chunk(page, sq, kv):
    go(sq, kv, 8, 2, page, seed=page + len(sq))


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (8, 8), (5, 1), (14, 2), (16, 1), (24, 2), (9, 1), (7, 1), (8, 1), (64, 1), (128, 1), (100, 1)])
def test_group_sizes(h_q, h_kv):
    go([1, 1, 1], [100, 257, 33], h_q, h_kv, 32, seed=h_q)
    go([3, 17, 70], [100, 257, 70], h_q, h_kv, 32, seed=h_q + 1)


@pytest.mark.parametrize("S", [1, 2, 3, 7, 64])
def test_forced_splits(S):
    go([1, 1, 1], [1000, 130, 5], 8, 2, 16, seed=S, force_splits=S)
    go([40, 1, 150], [1000, 130, 150], 8, 2, 16, seed=S, force_splits=S)


@pytest.mark.parametrize("num_sms", [1, 3, 20])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("max_q", [1, 2, 4])
def test_shares_that_cross_sequences(num_sms, page, max_q):
    """CTAs that take the end of one sequence, several whole ones and the start of another; plans of the kernels of 8 and of 16 rows."""
    rng = np.random.default_rng(num_sms)
    kv = [int(x) for x in rng.integers(0, 700, 45)]
    sq = [int(x) for x in rng.integers(0, 4, 45)]
    go(sq, kv, 8, 2, page, seed=num_sms, num_sms=num_sms, max_q=max_q)
    go(sq[:9], kv[:9], 10, 5, page, seed=num_sms, num_sms=num_sms, max_q=max_q)


@pytest.mark.parametrize("num_sms", [1, 3, 20, 152])
@pytest.mark.parametrize("page", [16, 128])
def test_few_tokens_in_equal_shares(num_sms, page):
    """Sequences of one query tile in the kernel of 256-row jobs, cut where a CTA's share ends."""
    rng = np.random.default_rng(num_sms + page)
    kv = [int(x) for x in rng.integers(0, 1500, 30)]
    sq = [int(x) for x in rng.integers(0, 17, 30)]
    go(sq, kv, 8, 2, page, seed=num_sms, num_sms=num_sms, max_q=16, max_kv=2000)
    go(sq[:4], kv[:4], 32, 2, page, seed=num_sms, num_sms=num_sms, max_q=16, max_kv=1024)


@pytest.mark.parametrize("S", [0, 1, 3])
def test_rows_without_keys_and_empty_sequences(S):
    """More new tokens than keys (the first queries see nothing), no keys at all, no new tokens."""
    go([6, 4, 0, 1, 0], [3, 0, 50, 20, 0], 8, 2, 16, force_splits=S)
    go([2, 1, 0, 1, 0], [1, 0, 50, 20, 0], 8, 2, 16, force_splits=S)
    go([160, 40, 0, 1], [100, 0, 50, 20], 8, 2, 16, force_splits=S)


@pytest.mark.parametrize("sq", [[1, 1, 1], [3, 3, 1], [20, 70, 1]])
@pytest.mark.parametrize("page", [16, 32])
def test_pages_that_are_missing(sq, page):
    c, q, cu = Paged4([150, 300, 64], 2, page, seed=3), queries(sum(sq), 8, 4), cu_of(sq)
    c.table[0, 1], c.table[1, 0], c.table[1, 5], c.table[2, :] = -1, 1 << 20, -7, -1
    ref = c.reference(q, cu, 1 / math.sqrt(D))
    check(*run4(c, q, cu, 8), ref, P_TYPE)


@pytest.mark.parametrize("out_dtype,inv_scale", [("bf16", 1.0), ("e4m3", 64.0)])
@pytest.mark.parametrize("sq", [[1, 1], [3, 4], [40, 150]])
def test_output_types(out_dtype, inv_scale, sq):
    go(sq, [300, 900], 8, 2, 16, out_dtype=out_dtype, inv_scale=inv_scale)


@pytest.mark.parametrize("layout", ["row", "head"])
@pytest.mark.parametrize("sq", [[1, 2], [60, 3]])
def test_layouts(layout, sq):
    go(sq, [333, 70], 8, 2, 64, layout=layout)
    go(sq, [333, 70], 4, 4, 16, layout=layout)


@pytest.mark.parametrize("sq", [[1, 1], [2, 50]])
@pytest.mark.parametrize("scale", [0.0, -0.09])
def test_scales_that_are_not_positive(sq, scale):
    go(sq, [200, 90], 8, 2, 16, scale=scale)


@pytest.mark.parametrize("sq", [[1, 1], [4, 2], [2, 50]])
def test_a_descale_that_is_not_a_number(sq):
    c, q, cu = Paged4([200, 90], 2, 16, seed=5), queries(sum(sq), 8, 6), cu_of(sq)
    c.dk = float("nan")
    out, lse, _ = run4(c, q, cu, 8)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("sq", [[1, 1, 1], [2, 50, 1]])
def test_queries_of_any_size(sq):
    """Q is held in f16 at a power of two of its row: rows near bf16's ends, rows of zeros, and elements far below their row's largest."""
    c, q, cu = Paged4([200, 90, 33], 2, 16, seed=5), queries(sum(sq), 8, 6), cu_of(sq)
    for power in (-100, -30, 30, 100):
        x = (q.float() * 2.0 ** power).to(torch.bfloat16)
        x[:, 1] = 0
        x[:, 2, ::3] *= 2.0 ** -20
        kw = dict(scale=2.0 ** -power / math.sqrt(D))
        check(*run4(c, x, cu, 8, **kw), c.reference(x, cu, kw["scale"]), P_TYPE)


@pytest.mark.parametrize("sq", [[1], [4], [60]])
def test_a_query_that_is_not_a_number(sq):
    c, q, cu = Paged4([200], 2, 16, seed=5), queries(sum(sq), 8, 6), cu_of(sq)
    x = q.clone()
    x[0, 3, 5] = float("nan")
    out, lse, _ = run4(c, x, cu, 8)
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
    out[0, 3], lse[0, 3] = 0, 0
    ref = c.reference(q, cu, 1 / math.sqrt(D))
    ref[0][0, 3], ref[1][0, 3] = 0, 0
    check(out, lse, None, ref, P_TYPE)


@pytest.mark.parametrize("sq", [[1, 3], [2, 2], [70, 9]])
def test_rows_behind_the_last_sequence_are_left(sq):
    c, q, cu = Paged4([150, 40], 2, 16, seed=7), queries(sum(sq), 8, 8), cu_of(sq)
    n = sum(sq)
    ref = c.reference(torch.cat([q, q[:5]]), cu, 1 / math.sqrt(D))
    check(*run4(c, q, cu, 8, rows=n + 5, amax=False), ref, P_TYPE, untouched_from=n)


@pytest.mark.parametrize("sq", [[1], [3], [80]])
def test_small_weights_of_a_long_row_count(sq):
    """One key whose score is 20 above all others' and whose V is 0: what is left is the others' (2^-20 each of its weight)."""
    n = 4096
    c = Paged4([n], 1, 64, seed=9)
    page = c.table[0].long()
    c.k.fill_(0)                 # scores 0
    c.ks.fill_(0x38)
    c.v.fill_(0x22)              # ones
    c.vs.fill_(0x38)
    c.k[page[0], 0, 0] = 0x77    # 6 everywhere
    c.v[page[0], 0, 0] = 0
    c.dk = c.dv = 1.0
    q, cu = torch.full((sum(sq), 4, D), 1.0).to(torch.bfloat16), cu_of(sq)
    scale = 20 * math.log(2) / (6 * D)
    check(*run4(c, q, cu, 4, scale=scale), c.reference(q, cu, scale), P_TYPE)


def test_strided_queries_on_a_stream_of_their_own():
    c, cu = Paged4([500, 90], 2, 32, seed=11), cu_of([1, 2])
    x = queries(3, 24, 12)
    ref = c.reference(x[:, 8:16], cu, 1 / math.sqrt(D))
    dev, pages = x.cuda(), c.pages()
    plan = b.sdpa_paged_plan(2, 8, 2, D, "e2m1", 2, 3, 500)
    ws = torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((3, 8, D), device="cuda"), torch.empty((3, 8), device="cuda")
    args = [c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), None, f32(c.dk), f32(c.dv)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    b.sdpa_paged(plan, 3, dev[:, 8:16], pages, *args, 1 / math.sqrt(D), "f32", 1.0, out, lse, None, ws, stream=st)
    torch.cuda.synchronize()
    check(out.cpu(), lse.cpu(), None, ref, P_TYPE)


@pytest.mark.parametrize("sq,kv", [([1] * 40, 3000), ([200] * 6, 900), ([64] * 200, 300)])
def test_waits_that_run_out(sq, kv):
    """Limits below a load's latency: the call ends, the status says so, and the next call is right. (Single tokens: the kernel of
    8 rows computes on a block for longer than its loads take, so there no wait need run out.)"""
    kv = [kv] * len(sq)
    c, q, cu = Paged4(kv, 2, 64, seed=13), queries(sum(sq), 8, 14), cu_of(sq)
    plan = b.sdpa_paged_plan(len(kv), 8, 2, D, "e2m1", max(sq), sum(sq), max(kv))
    ws = torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    out = torch.empty((sum(sq), 8, D), device="cuda")
    args = [q.cuda(), c.pages(), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), None, f32(c.dk), f32(c.dv), 1 / math.sqrt(D), "f32", 1.0, out,
            None, None, ws]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    seen = 0
    try:
        for limit in (200, 500, 1000, 2000, 4000, 8000):
            b.mla_set_wait_limit_ns(limit)
            flush.fill_(1)          # the keys are not in the cache
            b.sdpa_paged(plan, sum(sq), *args)
            torch.cuda.synchronize()
            st, site = b.mla_get_status()
            assert st in (0, b.MLA_STATUS_TIMEOUT) and (site != 0) == (st != 0), (limit, st, site)
            seen += st
    finally:
        b.mla_set_wait_limit_ns(0)
    assert seen or max(sq) == 1, "no wait ran out"
    check(*run4(c, q, cu, 8), c.reference(q, cu, 1 / math.sqrt(D)), P_TYPE)


# ------------------------------------------------------------ a server's steps --

@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
def test_steps_of_a_server(dtype):
    """Prompts, a chunk and decode steps: map, rotating append and attention, captured once a shape and replayed, against the oracle
    on the values that the cache holds, which in turn are those of the rotated rows."""
    page, width, h_q, h_kv, rot = 16, 12, 8, 2, 64
    g = torch.Generator().manual_seed(3)
    cs = table_of(page * width, rot)
    mem = caches(dtype, 30, page, h_kv, device="cuda", fill=0x7F)
    pages = b.kv_pages(*mem)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((3, width), -1, **i32)
    free, count = torch.arange(30, **i32), torch.tensor([30, 0], **i32)
    held, new, cu = torch.zeros(3, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32)
    dq, dk, dv = (None, None, None) if dtype == "bf16" else (f32(0.012), f32(0.012), f32(0.012)) if dtype == "e4m3" else (None, f32(0.004), f32(0.004))
    scale = 1 / math.sqrt(D)
    so_far = [0, 0, 0]
    graphs = {}
    for counts in [(40, 7, 0), (1, 1, 33), (1, 1, 1), (1, 1, 1), (20, 1, 1), (1, 1, 1)]:
        n = sum(counts)
        shape = max(counts) > 1, n
        if shape not in graphs:
            s = dict(qkv=torch.zeros((n, h_q + 2 * h_kv, D), dtype=torch.bfloat16, device="cuda"),
                     slots=torch.zeros(n, dtype=torch.int64, device="cuda"), pos=torch.zeros(n, **i32),
                     q=torch.zeros((n, h_q, D), dtype=torch.uint8 if dtype == "e4m3" else torch.bfloat16, device="cuda"),
                     out=torch.zeros((n, h_q, D), device="cuda"), lse=torch.zeros((n, h_q), device="cuda"),
                     k=torch.zeros((n, h_kv, D), dtype=torch.bfloat16, device="cuda"), v=torch.zeros((n, h_kv, D), dtype=torch.bfloat16, device="cuda"))
            plan = b.sdpa_paged_plan(3, h_q, h_kv, D, dtype, max(counts), n, page * width)
            s["ws"] = torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
            tab = cs.cuda()

            def step(s=s, plan=plan, n=n, tab=tab):
                x = s["qkv"]
                b.kv_pages_map(page, held, new, cu, n, table, free, count, count, s["slots"], s["pos"])
                b.kv_pages_write_rotary(pages, x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], s["pos"], tab, s["slots"], s["q"],
                                        descale_q=dq, descale_k=dk, descale_v=dv)
                b.sdpa_paged(plan, n, s["q"], pages, table, new, cu, dq, dk, dv, scale, "f32", 1.0, s["out"], s["lse"], None, s["ws"])
                b.kv_pages_read(pages, s["slots"], s["k"], s["v"], dk, dv)

            s["graph"] = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(s["graph"]):
                step()
            graphs[shape] = s
        s = graphs[shape]
        x = torch.randn((n, h_q + 2 * h_kv, D), generator=g).to(torch.bfloat16)
        s["qkv"].copy_(x)
        held.copy_(torch.tensor(so_far, dtype=torch.int32))
        so_far = [a + c for a, c in zip(so_far, counts)]
        new.copy_(torch.tensor(so_far, dtype=torch.int32))
        cu.copy_(cu_of(counts))
        s["graph"].replay()
        torch.cuda.synchronize()
        status_clear()
        pos = s["pos"].cpu().numpy()
        assert pos.tolist() == [p for a, c in zip(so_far, counts) for p in range(a - c, a)]
        # the append: what the cache holds of the new rows
        y = op.rotate(x[:, h_q:h_q + h_kv].float().numpy(), cs.numpy(), pos)
        for got, want in ((s["k"], y), (s["v"], x[:, h_q + h_kv:].float().numpy())):
            err = np.abs(got.cpu().double().numpy() - want)
            if dtype == "e2m1":   # half a step of e2m1 at its group's largest is the scale, (1 + 2^-4) / 6 of it at most; then bf16
                top = np.repeat(np.abs(want).reshape(n, h_kv, 8, 16).max(-1), 16, -1)
                assert np.all(err <= top / 6 * (1 + 2.0 ** -4) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * top)
            else:
                assert np.all(err <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -4 + 2.0 ** -7) * np.abs(want) + 2.0 ** -10 * 0.013)
        # the attention: over the values that the cache holds, queries as rotated
        if dtype == "e2m1":
            kc, vc = (op.four_bit_decode(c.cpu().numpy(), z.cpu().numpy()) * np.float32(0.004) for c, z in ((mem[0], mem[2]), (mem[1], mem[3])))
        else:
            kc, vc = (op.decode_values(c, 1.0 if dtype == "bf16" else np.float32(0.012)) for c in mem[:2])
        qv = op.decode_values(s["q"], np.float32(0.012) if dtype == "e4m3" else 1.0)
        ref = op.paged_attention(qv, kc, vc, table.cpu().numpy(), np.array(so_far), cu_of(counts).numpy(), scale)
        check(s["out"].cpu(), s["lse"].cpu(), None, ref, "bf16" if dtype == "bf16" else P_TYPE)


def test_a_prefix_read_back_for_packed_attention():
    """Values of a 4-bit cache as bf16 rows, attended by sdpa_prompt: what sdpa_paged gives over the pages, to bf16's rounding of the rows."""
    c, q, cu = Paged4([300, 41], 2, 16, seed=15), queries(20 + 41, 8, 16), cu_of([20, 41])
    pages = c.pages()
    pos = [torch.arange(m) for m in (300, 41)]
    slots = torch.cat([c.table[i].long()[p // 16] * 16 + p % 16 for i, p in enumerate(pos)]).cuda()
    k, v = (torch.zeros((341, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b.kv_pages_read(pages, slots, k, v, f32(c.dk), f32(c.dv))
    out = torch.empty((61, 8, D), device="cuda")
    b.sdpa_prompt(2, q.cuda(), k, v, cu.cuda(), cu_of([300, 41]).cuda(), None, None, None, 1 / math.sqrt(D), "f32", 1.0, out)
    torch.cuda.synchronize()
    status_clear()
    ref = op.prompt_attention(q.double().numpy(), k.cpu().double().numpy(), v.cpu().double().numpy(), cu.numpy(), cu_of([300, 41]).numpy(),
                              1 / math.sqrt(D))
    check(out.cpu(), None, None, ref, "bf16")
    kk, vv = c.values()
    sel = slots.cpu().numpy()
    kk, vv = kk.reshape(-1, 2, D)[sel], vv.reshape(-1, 2, D)[sel]
    assert np.all(np.abs(k.cpu().double().numpy() - kk) <= 2.0 ** -8 * np.abs(kk) * (1 + 2.0 ** -8))
    assert np.all(np.abs(v.cpu().double().numpy() - vv) <= 2.0 ** -8 * np.abs(vv) * (1 + 2.0 ** -8))


# --------------------------------------------------------------- what else a caller may do --

def test_a_scale_of_the_queries_applies():
    sq = [1, 3]
    c, q, cu = Paged4([200, 90], 2, 16, seed=17), queries(4, 8, 18), cu_of(sq)
    ref = c.reference((q.float() * 0.5).to(torch.bfloat16), cu, 1 / math.sqrt(D))     # (exact: a power of two)
    check(*run4(c, q, cu, 8, descale_q=0.5), ref, P_TYPE)


@pytest.mark.parametrize("max_q", [1, 4, 40])
def test_pages_that_sequences_share(max_q):
    """Five requests over one prefix of 10 pages, and a page that stands twice in one table."""
    c = Paged4([300, 64, 64, 64, 64], 2, 16, seed=19)
    c.table[1:, :10] = c.table[0, :10]
    c.table[4, 7] = c.table[4, 2]
    c.kv_lens[1:] = 160
    sq = [1] * 5 if max_q < 40 else [1, 30, 1, 40, 7]
    q, cu = queries(sum(sq), 8, 20), cu_of(sq)
    check(*run4(c, q, cu, 8, max_q=max_q), c.reference(q, cu, 1 / math.sqrt(D)), P_TYPE)


@pytest.mark.parametrize("max_q,max_kv", [(1, 60), (2, 500), (4, 500), (40, 60), (40, 9000)])
def test_hundreds_of_short_sequences(max_q, max_kv):
    rng = np.random.default_rng(max_q + max_kv)
    sq = [int(x) for x in rng.integers(0, 4, 500)]
    kv = [int(x) for x in rng.integers(0, 60, 500)]
    sq[300], kv[300] = (3, 400) if max_q < 40 else (150, 480)
    go(sq, kv, 8, 2, 16, seed=7, max_q=max_q, max_kv=max_kv)


@pytest.mark.parametrize("max_kv", [200, 9000])
@pytest.mark.parametrize("S", [0, 1])
@pytest.mark.parametrize("each", [[(64, 200), (3, 40), (2, 9)], [(64, 64), (40, 50), (1, 1), (9, 130)], [(50, 90), (33, 33)]])
def test_short_jobs_behind_long_ones(each, S, max_kv):
    """Several jobs a CTA, those of one key tile and one or two row blocks behind jobs with rows to write for long: what a job's
    rows were scaled by has to be its own."""
    sq, kv = ([x[k] for x in each] * 40 for k in (0, 1))
    c, q, cu = Paged4(kv, 8, 16, seed=len(each)), queries(sum(sq), 32, 21), cu_of(sq)
    x = (q.float() * 2.0 ** torch.randint(-12, 12, (len(q), 32, 1), generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    x /= x.float().abs().amax(-1, keepdim=True).clamp(min=1).to(torch.bfloat16)
    check(*run4(c, x, cu, 32, force_splits=S, max_kv=max_kv), c.reference(x, cu, 1 / math.sqrt(D)), P_TYPE)


@pytest.mark.parametrize("page,h_q,h_kv", [(1024, 8, 1), (65536, 4, 2), (16, 32, 8)])
def test_pages_of_any_size(page, h_q, h_kv):
    go([1, 2, 1], [1500, 700, 64], h_q, h_kv, page, seed=page)
    go([50, 2, 1], [1500, 700, 64], h_q, h_kv, page, seed=page)


@pytest.mark.parametrize("max_q", [1, 3, 100])
def test_repeated_calls_give_the_same_bits(max_q):
    sq = [1, 1, 1] if max_q < 100 else [20, 70, 1]
    c, q, cu = Paged4([1500, 300, 64], 2, 16, seed=3), queries(sum(sq), 8, 4), cu_of(sq)
    a, z = (run4(c, q, cu, 8, max_q=max_q) for _ in range(2))
    assert torch.equal(a[0], z[0]) and torch.equal(a[1], z[1]) and a[2] == z[2]


@pytest.mark.parametrize("S", [0, 2])
@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [4, 9, 2, 12], [0, 200, 10, 250], [-5, 7, 1 << 20, 3], [0, 0, 0, 0]])
@pytest.mark.parametrize("max_q", [1, 4, 100])
def test_offsets_that_decrease_touch_nothing_outside(cu, S, max_q):
    """Rows are undefined then, but every write stays inside the buffers and every wait ends."""
    c, total = Paged4([500, 300, 64], 2, 16, seed=6), 260
    plan = b.sdpa_paged_plan(3, 8, 2, D, "e2m1", max_q, total, 500, force_splits=S)
    ws = torch.empty(max(16, plan.workspace_bytes) + 4096, dtype=torch.uint8, device="cuda")
    ws.fill_(0x5A)
    out = torch.full((total + 8, 8, D), 7.0, device="cuda")
    b.sdpa_paged(plan, total, queries(total, 8, 7).cuda(), c.pages(), c.table.cuda(), c.kv_lens.cuda(),
                 torch.tensor(cu, dtype=torch.int32, device="cuda"), None, f32(c.dk), f32(c.dv), 0.1, "f32", 1.0, out, None, None, ws)
    torch.cuda.synchronize()
    status_clear()
    assert torch.all(out[total:] == 7.0) and torch.all(ws[-4096:] == 0x5A)


def test_calls_on_two_streams_at_once():
    """Four calls of different kinds in flight together, five times over, each with a workspace of its own."""
    cases, state = [], []
    for i, sq in enumerate(([1] * 12, [4] * 5, [90, 200, 1], [1, 1])):
        kv = [int(x) for x in np.random.default_rng(i).integers(max(sq), 2500, len(sq))]
        c, q, cu = Paged4(kv, 2, 32, seed=30 + i), queries(sum(sq), 8, 40 + i), cu_of(sq)
        plan = b.sdpa_paged_plan(len(sq), 8, 2, D, "e2m1", max(sq), sum(sq), max(kv))
        ws = torch.full((max(1, plan.workspace_bytes),), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros((sum(sq), 8, D), device="cuda"), torch.zeros((sum(sq), 8), device="cuda")
        cases.append((c, q, cu))
        state.append((plan, sum(sq), q.cuda(), c.pages(), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), None, f32(c.dk), f32(c.dv),
                      1 / math.sqrt(D), "f32", 1.0, out, lse, None, ws))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(state):
            b.sdpa_paged(*s, stream=streams[i & 1])
    torch.cuda.synchronize()
    status_clear()
    for (c, q, cu), s in zip(cases, state):
        check(s[13].cpu(), s[14].cpu(), None, c.reference(q, cu, 1 / math.sqrt(D)), P_TYPE)


def test_graphs_of_two_plans_share_a_workspace():
    """Decode and chunk captured apart over one workspace of the larger size, replayed in turn with other lengths."""
    c = Paged4([900, 700, 64], 2, 16, seed=50)
    plans = [b.sdpa_paged_plan(3, 8, 2, D, "e2m1", n, 3 * n, 1000) for n in (1, 50)]
    ws = torch.full((max(p.workspace_bytes for p in plans),), 0xFF, dtype=torch.uint8, device="cuda")
    pages, table, lens = c.pages(), c.table.cuda(), torch.zeros(3, dtype=torch.int32, device="cuda")
    graphs = []
    for p, n in zip(plans, (1, 50)):
        q = queries(3 * n, 8, 60 + n)
        dev, cu, out = q.cuda(), cu_of([n] * 3).cuda(), torch.zeros((3 * n, 8, D), device="cuda")
        args = (p, 3 * n, dev, pages, table, lens, cu, None, f32(c.dk), f32(c.dv), 1 / math.sqrt(D), "f32", 1.0, out, None, None, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.sdpa_paged(*args)
        graphs.append((g, args, q, n, out))
    for kv in ([900, 700, 64], [60, 650, 50], [800, 51, 64]):
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        c.kv_lens = torch.tensor(kv, dtype=torch.int32)
        for g, _, q, n, out in graphs + graphs[::-1]:
            g.replay()
            torch.cuda.synchronize()
            status_clear()
            check(out.cpu(), None, None, c.reference(q, cu_of([n] * 3), 1 / math.sqrt(D)), P_TYPE)


def test_codes_behind_32_bit_offsets():
    """Pages of codes and scales that lie more than 2^32 bytes from their bases."""
    page, stride = 16, (1 << 31) + 4096
    big = torch.zeros(3 * stride, dtype=torch.uint8, device="cuda")
    view = lambda last, at: big.as_strided((3, page, 1, last), (stride, last, page * last, 1), at)
    k, v, ks, vs = view(D // 2, 0), view(D // 2, 1024), view(8, 2048), view(8, 2048 + 128)
    c = Paged4([40], 1, page, seed=70, spare=0)
    for dst, src in ((k, c.k), (v, c.v), (ks, c.ks), (vs, c.vs)):
        dst.copy_(src)
    for sq in ([2], [30]):
        q, cu = queries(sum(sq), 4, 71), cu_of(sq)
        plan = b.sdpa_paged_plan(1, 4, 1, D, "e2m1", sq[0], sq[0], 40, force_splits=1)
        out = torch.empty((sq[0], 4, D), device="cuda")
        b.sdpa_paged(plan, sq[0], q.cuda(), b.kv_pages(k, v, ks, vs), c.table.cuda(), c.kv_lens.cuda(), cu.cuda(), None, f32(c.dk), f32(c.dv),
                     0.1, "f32", 1.0, out)
        torch.cuda.synchronize()
        status_clear()
        check(out.cpu(), None, None, c.reference(q, cu, 0.1), P_TYPE)
    del big, k, v, ks, vs
    torch.cuda.empty_cache()
