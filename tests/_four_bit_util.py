"""Inputs of the tests of the 4-bit paged cache and of the append that rotates. Tolerances of attention: those of _paged_util
with P in f16 (Q's own rounding, 2^-39 of a row's largest element, is far below their fp32 term)."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle.paged as op
from _paged_util import D, TORCH_OUT, status_clear
from split_kv_sparse_gb300 import binding as b


def table_of(positions, rot, base=10000.0):
    """cos_sin of a model's rotation, fp32 [positions, rot]."""
    f = base ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(positions)[:, None] * f[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def caches(dtype, num_pages, page, h_kv, layout="row", device="cpu", fill=None):
    """(k, v, k_scales, v_scales) as views [num_pages, page, h_kv, ..]; scales None but in 4 bits. fill: a byte for all."""
    def one(last, t, head_first):
        shape = (num_pages, h_kv, page, last) if head_first else (num_pages, page, h_kv, last)
        x = torch.zeros(shape, dtype=t, device=device)
        if fill is not None:
            x.view(torch.uint8).fill_(fill)
        return x.permute(0, 2, 1, 3) if head_first else x
    if dtype == "e2m1":
        return tuple(one(D // 2, torch.uint8, layout != "row") for _ in range(2)) + tuple(one(D // 16, torch.uint8, True) for _ in range(2))
    t = torch.bfloat16 if dtype == "bf16" else torch.uint8
    return one(D, t, layout != "row"), one(D, t, layout != "row"), None, None


def on_gpu(x):
    """.cuda() keeps the strides of a permuted cache."""
    return None if x is None else x.cuda()


def f32(x):
    return None if x is None else torch.tensor([x], dtype=torch.float32, device="cuda")


class Paged4:
    """A 4-bit cache filled with the keys of sequences; every row that belongs to none, and every unused page, holds -6 under
    scales of NaN."""

    dtype = "e2m1"

    def __init__(self, kv, h_kv, page, seed=0, layout="row", spare=5, scale=1.0):
        rng = np.random.default_rng(seed)
        held = [-(-m // page) for m in kv]
        n = sum(held) + spare
        order = rng.permutation(n)
        self.table = torch.full((len(kv), max(max(held), 1) + 2), -1, dtype=torch.int32)
        self.k, self.v, self.ks, self.vs = caches("e2m1", n, page, h_kv, layout, fill=0x7F)
        self.k.fill_(0xFF)
        self.v.fill_(0xFF)
        self.dk, self.dv = 0.004 * scale, 0.003 * scale
        at = 0
        for i, m in enumerate(kv):
            pg = order[at:at + held[i]]
            at += held[i]
            self.table[i, :held[i]] = torch.from_numpy(pg.astype(np.int32))
            for cache, scales, d in ((self.k, self.ks, self.dk), (self.v, self.vs, self.dv)):
                c, s = op.four_bit_encode(rng.standard_normal((m, h_kv, D)) * scale / d)
                for e in range(held[i]):
                    w = min(page, m - e * page)
                    cache[int(pg[e]), :w] = torch.from_numpy(c[e * page:e * page + w])
                    scales[int(pg[e]), :w] = torch.from_numpy(s[e * page:e * page + w])
        self.kv_lens = torch.tensor(kv, dtype=torch.int32)

    def values(self):
        return (op.four_bit_decode(self.k.numpy(), self.ks.numpy()) * np.float32(self.dk),
                op.four_bit_decode(self.v.numpy(), self.vs.numpy()) * np.float32(self.dv))

    def reference(self, q, cu_q, scale):
        k, v = self.values()
        return op.paged_attention(q.double().numpy(), k, v, self.table.numpy(), self.kv_lens.numpy(), cu_q.numpy(), scale)

    def pages(self):
        return b.kv_pages(*(on_gpu(x) for x in (self.k, self.v, self.ks, self.vs)))


def run4(c, q, cu_q, h_q, *, scale=1 / math.sqrt(D), out_dtype="f32", inv_scale=1.0, force_splits=0, max_q=None, rows=None, num_sms=0,
         max_kv=None, descale_q=None, lse=True, amax=True):
    """As run_paged, over a 4-bit cache."""
    h_kv = c.k.shape[2]
    n = cu_q[1:] - cu_q[:-1]
    total = rows or max(1, int(cu_q[-1]))
    plan = b.sdpa_paged_plan(len(c.kv_lens), h_q, h_kv, D, "e2m1", max_q or max(1, int(n.max())), total,
                             max_kv or max(1, int(c.kv_lens.max())), force_splits=force_splits, num_sms=num_sms)
    qd = q.cuda()
    if qd.shape[0] < total:
        qd = torch.cat([qd, torch.zeros((total - qd.shape[0],) + qd.shape[1:], dtype=qd.dtype, device="cuda")])
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda") if plan.workspace_bytes else None
    if ws is not None:
        ws.fill_(0xFF)          # NaN everywhere: nothing may be read before it is written
    out = torch.full((total, h_q, D), 7, dtype=TORCH_OUT[out_dtype], device="cuda")
    L = torch.full((total, h_q), 7.0, device="cuda") if lse else None
    M = torch.full((1,), -1.0, device="cuda") if amax else None
    b.sdpa_paged(plan, total, qd, c.pages(), c.table.cuda(), c.kv_lens.cuda(), cu_q.cuda(), f32(descale_q), f32(c.dk), f32(c.dv),
                 scale, out_dtype, inv_scale, out, L, M, ws)
    torch.cuda.synchronize()
    status_clear()
    return out.cpu(), (L.cpu() if lse else None), (float(M.cpu()[0]) if amax else None)
