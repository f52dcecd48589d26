"""fp64 / integer oracle for the paged KV cache and for attention over pages and packed prompts
(test infrastructure only; plain loops, no code shared with the GPU path)."""
from __future__ import annotations

import numpy as np

from . import codecs

LN2 = float(np.log(2.0))

# The weight below which the e4m3 kernels' P has an absolute error: they hold 2^(s - m + 7) in f16, subnormal below 2^-14.
F16_FLOOR = 2.0 ** -21


def pages(n: int, page_size: int, width: int) -> int:
    return min(max(0, -(-int(n) // page_size)), width)


def map_pages(page_size, held, new, cu_q, total_q, table, free_pages, free_in):
    """The bookkeeping of kv_pages_map, request by request: (table, free_pages, (left, short), slots, positions)."""
    table, F = np.array(table, dtype=np.int32), np.array(free_pages, dtype=np.int32)
    B, W = len(held), table.shape[1]
    cap = len(F)
    n = min(max(int(free_in), 0), cap)
    for b in range(B):
        for e in range(pages(new[b], page_size, W), pages(held[b], page_size, W)):
            if table[b, e] >= 0 and n < cap:
                F[n] = table[b, e]
                n += 1
    short = 0
    for b in range(B):
        for e in range(pages(held[b], page_size, W), pages(new[b], page_size, W)):
            if n > 0:
                n -= 1
                table[b, e] = F[n]
            else:
                table[b, e] = -1
                short += 1
    slots = np.full(total_q, -1, dtype=np.int64)
    positions = np.full(total_q, -1, dtype=np.int32)
    for b in range(B):
        count = int(cu_q[b + 1]) - int(cu_q[b])
        for i in range(count):
            p, r = int(new[b]) - count + i, int(cu_q[b]) + i
            if p < 0 or p // page_size >= W or r >= total_q:
                continue
            positions[r] = p
            page = int(table[b, p // page_size])
            if page >= 0:
                slots[r] = page * page_size + p % page_size
    return table, F, (n, short), slots, positions


def attend(q, keys, values, seen, sm_scale, floor=F16_FLOOR):
    """One sequence: q [n, h_q, d] (fp64), keys and values [m, h_kv, d], seen bool [n, m]. Returns (O [n, h_q, d],
    LSE2 [n, h_q], A [n, h_q, d]) with A = sum_j max(p_j, floor) |v_j| / sum_j p_j, p_j = exp(s_j - max s), the scale of
    rounding errors of P and of the sum: below the floor an e4m3 kernel's p has an error of u floor, not of u p. floor = 0
    for bf16, whose P has fp32's range, and for what is relative to the sum itself."""
    n, h_q, d = q.shape
    group = h_q // max(1, keys.shape[1])
    O, A = np.zeros((n, h_q, d)), np.zeros((n, h_q, d))
    L = np.full((n, h_q), -np.inf)
    if keys.shape[0] == 0 or n == 0:
        return O, L, A
    has = seen.any(axis=1)
    any_key = seen.any(axis=0)
    keys = np.where(any_key[:, None, None], keys, 0.0)       # what nobody sees reaches nothing
    values = np.where(any_key[:, None, None], values, 0.0)
    for j in range(h_q):
        K, V = keys[:, j // group], values[:, j // group]
        s = np.where(seen, sm_scale * (q[:, j] @ K.T), -np.inf)
        m = np.where(has, s.max(axis=1), 0.0)
        p = np.exp(s - m[:, None])
        z = np.where(has, p.sum(axis=1), 1.0)
        O[:, j] = (p @ V) / z[:, None]
        A[:, j] = (np.where(seen, np.maximum(p, floor), 0.0) @ np.abs(V)) / z[:, None]
        L[:, j] = np.where(has, (m + np.log(z)) / LN2, -np.inf)
    return O, L, A


def decode_values(x, descale: float) -> np.ndarray:
    """fp64 values of a bf16 tensor, or of e4m3 codes (uint8 or float8 tensor), times the descale."""
    import torch
    x = x.detach().cpu()
    if x.dtype == torch.bfloat16:
        return x.double().numpy() * descale
    return codecs.e4m3_decode(x.contiguous().view(torch.uint8).numpy()) * descale


def paged_attention(q, k_cache, v_cache, table, kv_lens, cu_q, sm_scale, floor=F16_FLOOR):
    """q [total_q, h_q, d], caches [num_pages, page_size, h_kv, d] as fp64 values; returns (O, LSE2, A); rows outside the
    sequences are NaN."""
    n_pages, ps = k_cache.shape[:2]
    W = table.shape[1]
    total_q, h_q, d = q.shape
    O, A = np.full((total_q, h_q, d), np.nan), np.full((total_q, h_q, d), np.nan)
    L = np.full((total_q, h_q), np.nan)
    for b in range(len(kv_lens)):
        q0, q1 = int(cu_q[b]), int(cu_q[b + 1])
        m = min(max(int(kv_lens[b]), 0), W * ps)
        pos = np.arange(m)
        page = table[b][pos // ps].astype(np.int64)
        ok = (page >= 0) & (page < n_pages)
        K = k_cache[np.where(ok, page, 0), pos % ps]
        V = v_cache[np.where(ok, page, 0), pos % ps]
        at = m - (q1 - q0) + np.arange(q1 - q0)
        seen = (pos[None, :] <= at[:, None]) & ok[None, :]
        O[q0:q1], L[q0:q1], A[q0:q1] = attend(q[q0:q1], K, V, seen, sm_scale, floor)
    return O, L, A


def prompt_attention(q, k, v, cu_q, cu_kv, sm_scale, floor=F16_FLOOR):
    total_q, h_q, d = q.shape
    O, A = np.full((total_q, h_q, d), np.nan), np.full((total_q, h_q, d), np.nan)
    L = np.full((total_q, h_q), np.nan)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_kv[b]), int(cu_kv[b + 1])
        at = (k1 - k0) - (q1 - q0) + np.arange(q1 - q0)
        seen = np.arange(k1 - k0)[None, :] <= at[:, None]
        O[q0:q1], L[q0:q1], A[q0:q1] = attend(q[q0:q1], k[k0:k1], v[k0:k1], seen, sm_scale, floor)
    return O, L, A


GROUP4 = 16     # dims of a 4-bit cache that share a scale


def four_bit_encode(y):
    """y [..., 128], the values over the descale: (codes [..., 64], scales [..., 8]) as bytes. The quotients are those of y's own
    type, so fp32 values give the codes of fp32 divisions."""
    y = np.asarray(y)
    g = y.reshape(*y.shape[:-1], y.shape[-1] // GROUP4, GROUP4)
    amax = np.abs(g).max(-1)
    with np.errstate(all="ignore"):
        scales = codecs.e4m3_encode((amax / y.dtype.type(6)).astype(np.float64))
        s = codecs.e4m3_decode(scales).astype(y.dtype)[..., None]
        q = np.where(s > 0, g / s, np.copysign(y.dtype.type(0), g))
    c = codecs.e2m1_encode(np.clip(q, -1e6, 1e6).astype(np.float64)).reshape(y.shape)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), scales


def four_bit_decode(codes, scales) -> np.ndarray:
    """fp64 values (without the descale) of codes [..., 64] and scales [..., 8]."""
    codes = np.asarray(codes)
    v = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]))
    v[..., 0::2], v[..., 1::2] = codecs.e2m1_decode(codes & 15), codecs.e2m1_decode(codes >> 4)
    return v * np.repeat(codecs.e4m3_decode(scales), GROUP4, axis=-1)


def rotate(x, cos_sin, positions, interleaved=False):
    """x [rows, heads, 128] turned by the angles of its rows' positions, cos_sin [positions, R]; in x's own type, every
    product and sum rounded. Rows without a position are left."""
    x = np.array(x)
    R = cos_sin.shape[1]
    for r, p in enumerate(positions):
        if p < 0 or p >= len(cos_sin):
            continue
        c, s = cos_sin[p, :R // 2].astype(x.dtype), cos_sin[p, R // 2:].astype(x.dtype)
        i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        a, b = x[r, :, i].copy(), x[r, :, j].copy()
        x[r, :, i] = a * c - b * s
        x[r, :, j] = b * c + a * s
    return x
