"""GPU tests of attention rows whose result lies in many small weights: one key far above the others (an attention sink) whose
V is 0, so that O comes out of the rest alone; and rows of V = 1, whose O is the quotient of the two sums.

Tolerances (as in _paged_util, with nothing added for weights below f16's normal range but what the kernels' own reference
leaves): p of the largest weight 1, u_P the half step of P's type (bf16 2^-8; its pair in the 16-row kernel 2^-16; f16
2^-11). f16 P is 2^(s - m + 7) with m at most the row's maximum: below 2^-14, so p below 2^-21, its half step is 2^-25, so
2^-32 = u_P 2^-21 of p. With A(f) = sum max(p, f) |v| / sum p, and N keys:
    |O - O_ref| <= u_P A(f) + (2^-12 + N 2^-24) A(0),    f = 2^-21 for e4m3, 0 for bf16;
2^-12 as there (scores: the products and sums of these inputs are exact, 26 log2 units times the scale's two roundings and the
exponent's one are 2^-18 of p; the exponential 2^-22), N 2^-24 a worst case of the fp32 sums of N terms."""
import math

import numpy as np
import pytest
import torch

import oracle.paged as op
from _paged_util import D, LSE_ATOL, cu_of, scalar, status_clear
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu

KINDS = ["decode", "chunk", "prompt"]
FLOOR = {"bf16": 0.0, "e4m3": 2.0 ** -21}


def half_step(dtype, kind):
    return 2.0 ** -11 if dtype == "e4m3" else 2.0 ** -16 if kind == "decode" else 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


def codes(x, dtype):
    return x.to(torch.bfloat16) if dtype == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)


def run(kind, dtype, q, k, v, scale, S=1):
    """One sequence: q [n, h_q, D], k and v [m, h_kv, D] on the host. (out fp32, lse)"""
    n, h_q, m, h_kv, dev = q.shape[0], q.shape[1], k.shape[0], k.shape[1], "cuda"
    out, lse = torch.full((n, h_q, D), 7.0, device=dev), torch.full((n, h_q), 7.0, device=dev)
    one = scalar(1.0, dtype)
    if kind == "prompt":
        b.sdpa_prompt(1, q.to(dev), k.to(dev), v.to(dev), cu_of([n]).to(dev), cu_of([m]).to(dev), one, one, one, scale, "f32",
                      1.0, out, lse)
    else:
        page = 64
        held = -(-m // page)
        kc, vc = (torch.zeros((held * page, h_kv, D), dtype=k.dtype) for _ in range(2))
        kc[:m], vc[:m] = k, v
        pages = b.kv_pages(kc.view(held, page, h_kv, D).to(dev), vc.view(held, page, h_kv, D).to(dev))
        plan = b.sdpa_paged_plan(1, h_q, h_kv, D, dtype, n, n, m, force_splits=S)
        assert plan.row_kernel == (kind == "decode")
        ws = torch.full((max(16, plan.workspace_bytes),), 0xFF, dtype=torch.uint8, device=dev)
        b.sdpa_paged(plan, n, q.to(dev), pages, torch.arange(held, dtype=torch.int32, device=dev)[None],
                     torch.tensor([m], dtype=torch.int32, device=dev), cu_of([n]).to(dev), one, one, one, scale, "f32", 1.0,
                     out, lse, None, ws)
    torch.cuda.synchronize()
    status_clear()
    return out.cpu().double().numpy(), lse.cpu().double().numpy()


def exact(q, k, v, scale, floor):
    """(O, LSE2, A(floor), A(0)) in 64 bits."""
    q, k, v = (op.decode_values(x, 1.0) for x in (q, k, v))
    n, h_q, m, h_kv = q.shape[0], q.shape[1], k.shape[0], k.shape[1]
    seen = np.arange(m)[None, :] <= m - n + np.arange(n)[:, None]
    O, L, _ = op.attend(q, k, v, seen, scale)
    A = [np.zeros(O.shape), np.zeros(O.shape)]
    for j in range(h_q):
        s = np.where(seen, scale * (q[:, j] @ k[:, j * h_kv // h_q].T), -np.inf)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        for a, f in zip(A, (floor, 0.0)):
            a[:, j] = (np.where(seen, np.maximum(p, f), 0.0) @ np.abs(v[:, j * h_kv // h_q])) / p.sum(axis=1)[:, None]
    return O, L, A[0], A[1]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("keys,below,at", [(16384, 25.3, 0), (32768, 26, 0), (9001, 20, 5000), (700, 12, 0)])
def test_weights_far_below_a_sink(dtype, kind, keys, below, at):
    g = torch.Generator().manual_seed(keys)
    n, h_q, h_kv = (1 if kind == "decode" else 40), 8, 2
    q, k = torch.ones((n, h_q, D)), torch.zeros((keys, h_kv, D))
    k[:, :, 0] = torch.randint(-8, 9, (keys, h_kv), generator=g) / 8.0     # scores up to below / 192 apart
    k[at] = 1.5                                                            # a raw score of 192
    v = 1 + torch.randn((keys, h_kv, D), generator=g)
    v[at] = 0
    q, k, v = (codes(x, dtype) for x in (q, k, v))
    scale = below * math.log(2) / 192
    O, _, Af, A0 = exact(q, k, v, scale, FLOOR[dtype])
    tol = half_step(dtype, kind) * Af + (2.0 ** -12 + keys * 2.0 ** -24) * A0
    for S in ((1,) if kind == "prompt" else (1, 3, 0)):
        out, _ = run(kind, dtype, q, k, v, scale, S)
        err = np.abs(out - O)
        assert np.all(err <= tol), (S, (err / tol).max(), (err / np.abs(O).max()).max())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("unit", [1.0, 1 / 8, 1 / 64, 1 / 4096, 1e-6])
def test_rows_of_ones_at_scores_up_to_2_to_the_25(dtype, kind, unit):
    """V = 1: O is sum P / sum p, so 1 whatever the scores are and however coarsely fp32 holds them: 127 * 448^2 = 2^24.6 in
    units of `unit` log2, the keys in rising order, so that a row's reference lags as far as it may."""
    g = torch.Generator().manual_seed(1)
    n, h_q, h_kv, keys = (1 if kind == "decode" else 40), 8, 2, 1500
    q, k = torch.full((n, h_q, D), 448.0), torch.full((keys, h_kv, D), 448.0)
    q[:, :, 5] = 4.0
    k[:, :, 5] = torch.sort(torch.rand((keys, h_kv), generator=g) * min(448.0, 8.0 / unit), dim=0).values
    q, k, v = (codes(x, dtype) for x in (q, k, torch.ones((keys, h_kv, D))))
    tol = half_step(dtype, kind) + 2.0 ** -12 + keys * (2.0 ** -24 + 2.0 ** -32)
    for S in ((1,) if kind == "prompt" else (1, 3)):
        out, lse = run(kind, dtype, q, k, v, unit * math.log(2), S)
        assert np.all(np.isfinite(lse)) and np.abs(out - 1).max() <= tol, np.abs(out - 1).max()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("keys,below", [(16384, 25.3), (100000, 25.3), (60000, 23.0), (100000, 31.3)])
def test_lse_of_many_weights_below_the_sums_last_bit(dtype, kind, keys, below):
    """Weights under half the last bit of a sum that a far larger one began: added one by one in fp32 none of them would
    count. The library's 1e-5 on the LSE holds for any number of keys: the sums of a block or tile have at most 128 terms,
    and their running sum is compensated, so its error is a few 2^-24, 4e-7 of the LSE, whatever their number."""
    g = torch.Generator().manual_seed(keys)
    n, h_q, h_kv = (1 if kind == "decode" else 40), 8, 2
    q, k, v = torch.ones((n, h_q, D)), torch.zeros((keys, h_kv, D)), torch.ones((keys, h_kv, D))
    k[:, :, 0] = torch.randint(-8, 9, (keys, h_kv), generator=g) / 8.0
    k[0] = 1.5
    q, k, v = (codes(x, dtype) for x in (q, k, v))
    scale = below * math.log(2) / 192
    _, L, _, _ = exact(q, k, v, scale, 0.0)
    for S in ((1,) if kind == "prompt" else (1, 0)):
        out, lse = run(kind, dtype, q, k, v, scale, S)
        assert np.abs(lse - L).max() <= LSE_ATOL, (S, np.abs(lse - L).max())
        assert np.abs(out - 1).max() <= half_step(dtype, kind) + 2.0 ** -12 + keys * 2.0 ** -24


@pytest.mark.parametrize("keys", [2, 5, 17, 60, 300])
def test_decode_rounds_bf16_weights_to_a_pair(keys):
    """The 16-row kernel's P is bf16 hi + lo: 2^-16 a term, where one bf16 costs 2^-8, which a few keys show. 2^-12 for fp32 as
    above (the scores of N(0, 1) values: 128 products, 2^-13.6)."""
    for seed in range(4):
        g = torch.Generator().manual_seed(100 * keys + seed)
        q, k, v = (codes(torch.randn((m, h, D), generator=g), "bf16") for m, h in ((1, 8), (keys, 2), (keys, 2)))
        scale = 1 / math.sqrt(D)
        O, L, _, A0 = exact(q, k, v, scale, 0.0)
        out, lse = run("decode", "bf16", q, k, v, scale)
        assert np.all(np.abs(out - O) <= (2.0 ** -16 + 2.0 ** -12) * A0), (np.abs(out - O) / A0).max()
        assert np.abs(lse - L).max() <= LSE_ATOL
