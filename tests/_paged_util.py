"""Inputs and tolerances of the tests of the paged KV cache and of prompt attention.

Tolerances, from the arithmetic (u = half a step of a type: bf16 2^-8, f16 2^-11, e4m3 2^-4, fp32 2^-24):
  * O, element by element, against the fp64 oracle, with A = sum_j softmax_j |v_j|:
        |O - O_ref| <= (u_P + 2^-12) A        (fp32 output)
    (softmax_j = p_j / sum p taken with p_j >= 2^-14, below which f16 is subnormal and its half step 2^-25 = u 2^-14).
    u_P is the half step of the type that P is rounded to (bf16 for bf16 V, f16 for e4m3 V). 2^-12 covers fp32: the
    score's 128 products (128 * 2^-24 of sum |q k| scale, about 10 in log2 units for N(0, 1) inputs: 2^-13.6), the
    exponential (2^-22 of p), the sum and the product over up to 2,048 keys (2,048 * 2^-24 = 2^-13 of A).
    A bf16 output adds 2^-8 |O_ref|, an e4m3 output 2^-4 |O_ref| (half its smallest step, 2^-10 / inv_scale, at least).
  * LSE (log2): 1e-5 absolute, the library's contract; -inf must match.
  * amax: that of the worst element's bound.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle.paged as op
from oracle import codecs
from split_kv_sparse_gb300 import binding as b

U_P = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}
FP32 = 2.0 ** -12
LSE_ATOL = 1e-5
D = 128
TORCH_OUT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}


def cu_of(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)


def values(g, shape, dtype, scale=1.0):
    """(tensor of the type, descale): N(0, scale^2) values."""
    x = torch.randn(shape, generator=g) * scale
    if dtype == "bf16":
        return x.to(torch.bfloat16), 1.0
    descale = 0.012 * scale
    return (x / descale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), descale


def garbage(x):
    """Fills a tensor with NaN (bf16) or the e4m3 NaN code, and some infinities in bf16."""
    if x.dtype == torch.bfloat16:
        x.fill_(float("nan"))
        x.view(-1)[::7] = float("inf")
    else:
        x.fill_(0x7F)


class Paged:
    """A paged cache filled with the keys of sequences; every row that belongs to none, and every unused page, is NaN."""

    def __init__(self, dtype, kv, h_kv, page, seed=0, layout="row", spare=5):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        held = [-(-m // page) for m in kv]
        self.num_pages = sum(held) + spare
        order = rng.permutation(self.num_pages)
        W = max(max(held), 1) + 2
        self.table = torch.full((len(kv), W), -1, dtype=torch.int32)
        shape = (self.num_pages, page, h_kv, D) if layout == "row" else (self.num_pages, h_kv, page, D)
        t = torch.bfloat16 if dtype == "bf16" else torch.uint8
        self.k, self.v = torch.empty(shape, dtype=t), torch.empty(shape, dtype=t)
        garbage(self.k)
        garbage(self.v)
        if layout != "row":
            self.k, self.v = self.k.permute(0, 2, 1, 3), self.v.permute(0, 2, 1, 3)
        self.dk = self.dv = 1.0
        at = 0
        for i, m in enumerate(kv):
            pg = order[at:at + held[i]]
            at += held[i]
            self.table[i, :held[i]] = torch.from_numpy(pg.astype(np.int32))
            K, self.dk = values(g, (m, h_kv, D), dtype)
            V, self.dv = values(g, (m, h_kv, D), dtype)
            for e in range(held[i]):
                n = min(page, m - e * page)
                self.k[int(pg[e]), :n] = K[e * page:e * page + n]
                self.v[int(pg[e]), :n] = V[e * page:e * page + n]
        self.kv_lens = torch.tensor(kv, dtype=torch.int32)
        self.dtype, self.page = dtype, page

    def reference(self, q, dq, cu_q, scale):
        return op.paged_attention(op.decode_values(q, dq), op.decode_values(self.k, self.dk),
                                  op.decode_values(self.v, self.dv), self.table.numpy(), self.kv_lens.numpy(),
                                  cu_q.numpy(), scale)


def scalar(x, dtype):
    return None if dtype == "bf16" else torch.tensor([x], dtype=torch.float32, device="cuda")


def status_clear():
    st, site = b.mla_get_status()
    assert st == 0, f"device status {st:#x}, first timed-out wait site {site}"


def run_paged(c, q, dq, cu_q, h_q, *, scale=1 / math.sqrt(D), out_dtype="f32", inv_scale=1.0, force_splits=0, max_q=None,
              rows=None, lse=True, amax=True, num_sms=0, max_kv=None):
    """The call on the current stream; `rows` pads the batch's rows. Returns (out, lse, amax) on the host."""
    h_kv = c.k.shape[2]
    n = (cu_q[1:] - cu_q[:-1])
    total = rows or max(1, int(cu_q[-1]))
    plan = b.sdpa_paged_plan(len(c.kv_lens), h_q, h_kv, D, c.dtype, max_q or max(1, int(n.max())), total,
                             max_kv or max(1, int(c.kv_lens.max())), force_splits=force_splits, num_sms=num_sms)
    dev = "cuda"
    qd = q.to(dev)
    if qd.shape[0] < total:
        qd = torch.cat([qd, torch.zeros((total - qd.shape[0],) + qd.shape[1:], dtype=qd.dtype, device=dev)])
    # .to keeps the strides of a permuted cache
    kc, vc = c.k.to(dev), c.v.to(dev)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=dev) if plan.workspace_bytes else None
    if ws is not None:
        ws.fill_(0xFF)          # NaN everywhere: nothing may be read before it is written
    out = torch.full((total, h_q, D), 7, dtype=TORCH_OUT[out_dtype], device=dev)
    L = torch.full((total, h_q), 7.0, device=dev) if lse else None
    M = torch.full((1,), -1.0, device=dev) if amax else None
    b.sdpa_paged(plan, total, qd, b.kv_pages(kc, vc), c.table.to(dev), c.kv_lens.to(dev), cu_q.to(dev),
                 scalar(dq, c.dtype), scalar(c.dk, c.dtype), scalar(c.dv, c.dtype), scale, out_dtype, inv_scale, out, L, M,
                 ws)
    torch.cuda.synchronize()
    status_clear()
    return out.cpu(), (L.cpu() if lse else None), (float(M.cpu()[0]) if amax else None)


def check(out, lse, amax, ref, dtype, out_dtype="f32", inv_scale=1.0, untouched_from=None, score_err=0.0):
    """score_err: relative error of P that large scores add (the module's bound holds for scale 1 / sqrt(128))."""
    O, L, A = ref
    if untouched_from is not None:
        assert torch.all(out[untouched_from:].float() == 7), "rows behind the last sequence were written"
        if lse is not None:
            assert torch.all(lse[untouched_from:] == 7)
        out, O, A, L = out[:untouched_from], O[:untouched_from], A[:untouched_from], L[:untouched_from]
        lse = None if lse is None else lse[:untouched_from]
    if out.dtype == torch.uint8:
        got = codecs.e4m3_decode(out.numpy()) / inv_scale
    else:
        got = out.double().numpy()
    tol = (U_P[dtype] + FP32 + score_err) * A
    bound = tol.max() if tol.size else 0.0
    if out_dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(O)
    elif out_dtype == "e4m3":
        tol = tol + np.maximum(2.0 ** -4 * np.abs(O), 2.0 ** -10 / inv_scale)
    assert np.all(np.isfinite(got)), "non-finite values"
    err = np.abs(got - O)
    worst = np.max(err - tol) if err.size else 0.0
    assert worst <= 0, f"O: {int((err > tol).sum())} of {err.size} off by up to {err.max():.3e} (excess {worst:.3e})"
    if lse is not None:
        g = lse.double().numpy()
        dead = np.isneginf(L)
        assert np.array_equal(np.isneginf(g), dead), "LSE: -inf pattern differs"
        if (~dead).any():
            d = np.abs(g[~dead] - L[~dead]).max()
            assert d <= LSE_ATOL, f"LSE off by {d:.3e}"
    if amax is not None:
        top = np.abs(O).max() if O.size else 0.0
        assert abs(amax - top) <= bound, (amax, top)
