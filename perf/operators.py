"""Cases of the paged KV cache (block tables and slot maps, the append, attention over its pages) and of prompt attention.

A case is a dict of plain values. ``prepare`` makes what a server has in hand before the call, ``run`` is one
pass through one operator: in its plain form (elementary torch operations in fp32, rounded once) where ``own``
is false, and through the library's entry points where it is true.
"""
import math
import random

import torch

own = False

D = 128
DESCALE = {"q": 0.0117, "k": 0.0121, "v": 0.0113}   # about 5.2 standard deviations to e4m3's 448


# --------------------------------------------------------------------------- cases --

def listed():
    return [
        # a decode step of a small server: one new token for each of 8 requests, one page of 16 in a while
        dict(name="map decode", op="map", batch=8, page=16, decode=1.0, finish=0.0, q_hi=1, kv_hi=16384, mix=1),
        # a mixed step: most requests decode, some bring prompts of up to 1000 tokens, some end and give pages back
        dict(name="map mixed", op="map", batch=256, page=16, decode=0.8, finish=0.1, q_hi=1000, kv_hi=8192, mix=2),
        # the rows of one decode step into an e4m3 cache: latency
        dict(name="write decode", op="write", dtype="e4m3", rows=8, h_kv=8, page=16, pages=4096, drop=0.0, fused=True),
        # prompt rows out of a fused projection into a bf16 cache, a few of them padding
        dict(name="write prompt", op="write", dtype="bf16", rows=16001, h_kv=8, page=64, pages=512, drop=0.01, fused=True),
        # single-token decode of 8 requests at the dense workload's lengths, e4m3
        dict(name="decode e4m3 b8", op="paged", dtype="e4m3", batch=8, h_q=32, h_kv=8, page=64, q_lo=1, q_hi=1,
             kv_lo=1024, kv_hi=16384, mix=3),
        # single-token decode of a full server, bf16, pages of 16
        dict(name="decode bf16 b96", op="paged", dtype="bf16", batch=96, h_q=32, h_kv=8, page=16, q_lo=1, q_hi=1,
             kv_lo=100, kv_hi=12000, mix=4),
        # the dense workload itself over pages: 1 to 16 new tokens a sequence (speculative decoding)
        dict(name="few tokens e4m3 b8", op="paged", dtype="e4m3", batch=8, h_q=32, h_kv=8, page=128, q_lo=1, q_hi=16,
             kv_lo=1024, kv_hi=16384, mix=5),
        # chunked prefill: ragged chunks of up to 600 tokens over long cached contexts, bf16, pages of 16
        dict(name="chunk bf16 ragged", op="paged", dtype="bf16", batch=5, h_q=32, h_kv=8, page=16, q_lo=1, q_hi=600,
             kv_lo=2000, kv_hi=16384, mix=6),
        # one long chunk over a long e4m3 cache
        dict(name="chunk e4m3 2048", op="paged", dtype="e4m3", batch=1, h_q=32, h_kv=8, page=64, q_lo=2048, q_hi=2048,
             kv_lo=32768, kv_hi=32768, mix=7),
        # short prompts, packed
        dict(name="prompt bf16 short", op="prompt", dtype="bf16", batch=9, h_q=32, h_kv=8, lo=1, hi=333, mix=8),
        # one long prompt
        dict(name="prompt bf16 16384", op="prompt", dtype="bf16", batch=1, h_q=32, h_kv=8, lo=16384, hi=16384, mix=9),
        # packed prompts of different lengths, e4m3, 16 query heads over 2
        dict(name="prompt e4m3 ragged", op="prompt", dtype="e4m3", batch=7, h_q=16, h_kv=2, lo=700, hi=5000, mix=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "write", "paged", "paged", "paged", "prompt", "prompt"])
    mix = rng.randrange(1 << 20)
    if op == "map":
        return dict(op=op, batch=_log(rng, 1, 512), page=rng.choice([16, 32, 64, 128]), decode=rng.choice([1.0, 0.8, 0.5]),
                    finish=rng.choice([0.0, 0.1, 0.3]), q_hi=_log(rng, 1, 1000), kv_hi=_log(rng, 16, 16384), mix=mix)
    if op == "write":
        return dict(op=op, dtype=rng.choice(["bf16", "e4m3"]), rows=_log(rng, 1, 16000), h_kv=rng.choice([1, 2, 4, 8]),
                    page=rng.choice([16, 32, 64, 128]), pages=1024, drop=rng.choice([0.0, 0.02]), fused=rng.random() < 0.5)
    h_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 4, 7, 8, 16] if h_kv <= 2 else [1, 2, 4, 4, 5, 8] if h_kv == 4 else [1, 2, 4])
    dtype = rng.choice(["bf16", "e4m3"])
    if op == "paged":
        kind = rng.choice(["decode", "few", "chunk"])
        batch = _log(rng, 1, 64) if kind == "decode" else _log(rng, 1, 12) if kind == "few" else _log(rng, 1, 4)
        q_hi = 1 if kind == "decode" else _log(rng, 2, 24) if kind == "few" else _log(rng, 33, 1000)
        kv_hi = _log(rng, max(64, q_hi), 16384)
        return dict(op=op, dtype=dtype, batch=batch, h_q=h_kv * group, h_kv=h_kv, page=rng.choice([16, 32, 64, 128, 256]),
                    q_lo=1, q_hi=q_hi, kv_lo=_log(rng, 1, kv_hi), kv_hi=kv_hi, mix=mix)
    batch = _log(rng, 1, 12)
    hi = _log(rng, 4, int(16000 / math.sqrt(batch)))
    return dict(op=op, dtype=dtype, batch=batch, h_q=h_kv * group, h_kv=h_kv, lo=_log(rng, 1, hi), hi=hi, mix=mix)


def _lens(case):
    """(new tokens, keys) of each sequence: a property of the case, not of the seed of its values."""
    rng = random.Random(case["mix"])
    if case["op"] == "prompt":
        n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
        return n, n
    sq = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    kv = [max(rng.randint(case["kv_lo"], case["kv_hi"]), n) for n in sq]
    return sq, kv


def _requests(case):
    """(positions held before, positions after, new tokens) of each request of a map case."""
    rng = random.Random(case["mix"])
    out = []
    for _ in range(case["batch"]):
        kind, cached = rng.random(), rng.randint(1, case["kv_hi"])
        if kind < case["decode"]:
            out.append((cached, cached + 1, 1))
        elif kind < case["decode"] + case["finish"]:
            out.append((cached, 0, 0))
        else:
            n = rng.randint(1, case["q_hi"])
            out.append((0, n, n))
    return out


def _pages(n, page):
    return (n + page - 1) // page


def work(case):
    if case["op"] == "map":
        req = _requests(case)
        moved = sum(abs(_pages(b, case["page"]) - _pages(a, case["page"])) for a, b, _ in req)
        return {"bytes": 12 * len(req) + 8 * moved + 12 * sum(n for _, _, n in req) + 12, "flops": 0}
    if case["op"] == "write":
        e = 2 if case["dtype"] == "bf16" else 1
        return {"bytes": case["rows"] * (2 * case["h_kv"] * D * (2 + e) + 8), "flops": 0}
    sq, kv = _lens(case)
    e = 2 if case["dtype"] == "bf16" else 1
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(sq, kv))
    moved = sum(sq) * case["h_q"] * (D * (e + 2) + 4) + sum(kv) * 2 * case["h_kv"] * D * e
    if case["op"] == "paged":
        moved += 4 * sum(_pages(m, case["page"]) for m in kv)
    return {"bytes": moved, "flops": 4 * D * case["h_q"] * pairs}


# -------------------------------------------------------------------------- inputs --

def _cu(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _values(shape, dtype, which, g):
    x = torch.randn(shape, dtype=torch.float32, device="cuda", generator=g)
    if dtype == "bf16":
        return x.to(torch.bfloat16)
    return (x / DESCALE[which]).clamp(-448, 448).to(torch.float8_e4m3fn)


def _descales(dtype):
    if dtype == "bf16":
        return None, None, None
    return tuple(torch.tensor([DESCALE[w]], dtype=torch.float32, device="cuda") for w in "qkv")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "map":
        req, P = _requests(case), case["page"]
        held = [a for a, _, _ in req]
        after = [b for _, b, _ in req]
        width = _pages(max(max(held), max(after), 1), P)
        n_held = sum(_pages(a, P) for a in held)
        s["capacity"] = n_held + sum(_pages(b, P) for b in after) + 64
        order = torch.randperm(s["capacity"], device="cuda", generator=g).to(torch.int32)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, a in enumerate(held):
            table[b, :_pages(a, P)] = order[at:at + _pages(a, P)]
            at += _pages(a, P)
        s["free_pages"] = torch.full((s["capacity"],), -1, dtype=torch.int32, device="cuda")
        s["free_pages"][:s["capacity"] - n_held] = order[n_held:]
        s["free_in"] = torch.tensor([s["capacity"] - n_held], dtype=torch.int32, device="cuda")
        s["free_out"] = torch.zeros(2, dtype=torch.int32, device="cuda")
        s["held"] = torch.tensor(held, dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(after, dtype=torch.int32, device="cuda")
        s["cu_q"] = _cu([n for _, _, n in req])
        s["total_q"] = max(1, sum(n for _, _, n in req))
        s["table"], s["width"] = table, width
        s["slots"] = torch.empty(s["total_q"], dtype=torch.int64, device="cuda")
        s["positions"] = torch.empty(s["total_q"], dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "write":
        n, h, P, pages = case["rows"], case["h_kv"], case["page"], case["pages"]
        if case["fused"]:   # K and V as slices of a fused projection's output, beside 4 query heads a KV head
            qkv = torch.randn((n, 6 * h, D), dtype=torch.float32, device="cuda", generator=g).to(torch.bfloat16)
            s["k"], s["v"] = qkv[:, 4 * h:5 * h], qkv[:, 5 * h:]
        else:
            s["k"], s["v"] = _values((n, h, D), "bf16", "k", g), _values((n, h, D), "bf16", "v", g)
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float8_e4m3fn
        s["k_cache"] = torch.zeros((pages, P, h, D), dtype=t, device="cuda")
        s["v_cache"] = torch.zeros((pages, P, h, D), dtype=t, device="cuda")
        # rows fill pages that lie anywhere in the cache, in order within a page
        order = torch.randperm(pages, device="cuda", generator=g)[:_pages(n, P)]
        slots = (order[:, None] * P + torch.arange(P, device="cuda")[None, :]).reshape(-1)[:n]
        drop = torch.rand(n, device="cuda", generator=g) < case["drop"]
        s["slots"] = torch.where(drop, torch.full_like(slots, -1), slots).contiguous()
        _, s["descale_k"], s["descale_v"] = _descales(case["dtype"])
        if own:
            import split_kv_sparse_gb300 as skv
            s["pages_desc"] = skv.kv_pages(s["k_cache"], s["v_cache"])
        return s
    sq, kv = _lens(case)
    h_q, h_kv, dtype = case["h_q"], case["h_kv"], case["dtype"]
    s["total_q"], s["max_q"], s["max_kv"] = sum(sq), max(sq), max(kv)
    s["q"] = _values((s["total_q"], h_q, D), dtype, "q", g)
    s["cu_q"], s["scale"] = _cu(sq), 1 / math.sqrt(D)
    s["descales"] = _descales(dtype)
    s["out"] = torch.empty((s["total_q"], h_q, D), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((s["total_q"], h_q), dtype=torch.float32, device="cuda")
    if case["op"] == "prompt":
        s["total_kv"] = sum(kv)
        s["k"] = _values((s["total_kv"], h_kv, D), dtype, "k", g)
        s["v"] = _values((s["total_kv"], h_kv, D), dtype, "v", g)
        s["cu_kv"] = _cu(kv)
        return s
    P = case["page"]
    held = [_pages(m, P) for m in kv]
    order = torch.randperm(sum(held) + 8, device="cuda", generator=g).to(torch.int32)
    s["k_cache"] = _values((sum(held) + 8, P, h_kv, D), dtype, "k", g)
    s["v_cache"] = _values((sum(held) + 8, P, h_kv, D), dtype, "v", g)
    s["table"] = torch.full((case["batch"], max(held)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        s["table"][b, :n] = order[at:at + n]
        at += n
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    if own:
        import split_kv_sparse_gb300 as skv
        s["pages_desc"] = skv.kv_pages(s["k_cache"], s["v_cache"])
        s["plan"] = skv.sdpa_paged_plan(case["batch"], h_q, h_kv, D, dtype, s["max_q"], s["total_q"], s["max_kv"])
        n = s["plan"].workspace_bytes
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    return s


# --------------------------------------------------------------------- plain forms --

def _map_plain(s):
    P, W = s["page"], s["width"]
    table, n = s["table"], s["free_in"].long()
    h = ((s["held"].long().clamp(min=0) + P - 1) // P).clamp(max=W)[:, None]
    p = ((s["lens"].long().clamp(min=0) + P - 1) // P).clamp(max=W)[:, None]
    e = torch.arange(W, device="cuda")[None, :]
    back = ((e >= p) & (e < h) & (table >= 0)).reshape(-1)
    to = torch.where(back, n + back.long().cumsum(0) - 1, s["capacity"])
    stack = torch.cat([s["free_pages"], s["free_pages"][:1]])
    stack = stack.scatter(0, to, table.reshape(-1))[:-1]
    n = n + back.sum()
    want = (e >= h) & (e < p)
    src = n - 1 - (want.reshape(-1).long().cumsum(0) - 1).reshape(want.shape)
    page = torch.where(src >= 0, stack[src.clamp(min=0, max=s["capacity"] - 1)], -1)
    table = torch.where(want, page, table)
    need = want.sum()
    left = torch.cat([(n - need).clamp(min=0), (need - n).clamp(min=0)]).to(torch.int32)
    r = torch.arange(s["total_q"], device="cuda")
    cu = s["cu_q"].long()
    b = torch.searchsorted(cu[1:], r, right=True)
    live = b < cu.numel() - 1
    b = b.clamp(max=cu.numel() - 2)
    pos = s["lens"].long()[b] - (cu[b + 1] - r)
    live = live & (pos >= 0) & (pos // P < W)
    page = table[b, (pos // P).clamp(min=0, max=W - 1)].long()
    slots = torch.where(live & (page >= 0), page * P + pos % P, -1)
    return {"table": table, "free_pages": stack, "free": left, "slots": slots,
            "positions": torch.where(live, pos, -1).to(torch.int32)}


def _write_plain(s):
    slots = s["slots"]
    out = []
    for x, cache, d in ((s["k"], s["k_cache"], s["descale_k"]), (s["v"], s["v_cache"], s["descale_v"])):
        rows = cache.view(-1, cache.shape[2], cache.shape[3])
        if d is not None:
            x = (x.float() / d).clamp(-448, 448).to(torch.float8_e4m3fn)
            rows, x = rows.view(torch.uint8), x.view(torch.uint8)
        # a row without a slot goes where the first row that has one goes, with that row's values
        keep = slots >= 0
        first = keep.long().argmax()
        src = torch.where(keep, torch.arange(slots.numel(), device="cuda"), first)
        rows[slots[src]] = x[src]
        out.append(cache)
    return {"k_cache": out[0], "v_cache": out[1]}


def _attend_plain(s, K, V, kv_len):
    """K, V fp32 [batch][keys][h_kv][D], padded; kv_len [batch]."""
    dq = s["descales"][0]
    B, L, h_kv, _ = K.shape
    h_q, M = s["h_q"], s["max_q"]
    group = h_q // h_kv
    cu = s["cu_q"].long()
    sq = cu[1:] - cu[:-1]
    i = torch.arange(M, device="cuda")
    rows = (cu[:-1, None] + i[None, :]).clamp(max=s["total_q"] - 1)
    q = s["q"].view(torch.uint8)[rows].view(s["q"].dtype).float() if dq is not None else s["q"][rows].float()
    if dq is not None:
        q = q * dq
    q = q.view(B, M, h_kv, group, D).permute(0, 2, 3, 1, 4).reshape(B, h_kv, group * M, D)
    x = torch.matmul(q, K.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, h_kv, group, M, L)
    pos = (kv_len - sq)[:, None] + i[None, :]
    hidden = torch.arange(L, device="cuda")[None, None, :] > pos[:, :, None]
    x.masked_fill_(hidden[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1) / math.log(2)
    V = torch.where((torch.arange(L, device="cuda")[None, :] < kv_len[:, None])[:, :, None, None], V, 0.0)
    o = torch.matmul(x.view(B, h_kv, group * M, L), V.permute(0, 2, 1, 3)).view(B, h_kv, group, M, D)
    o = o / torch.where(l == 0, 1.0, l)
    r = torch.arange(s["total_q"], device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True)
    i = r - cu[b]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, M, h_q, D)[b, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, M, h_q)[b, i]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _widen(x, d):
    return x.float() if d is None else x.view(torch.uint8).view(torch.float8_e4m3fn).float() * d


def _paged_plain(s):
    P = s["page"]
    j = torch.arange(s["max_kv"], device="cuda")
    slot = s["table"].long()[:, j // P].clamp(min=0) * P + j % P
    _, dk, dv = s["descales"]
    h_kv = s["h_kv"]

    def rows(cache, d):
        flat = cache.view(-1, h_kv, D)
        return _widen(flat[slot] if d is None else flat.view(torch.uint8)[slot], d)

    return _attend_plain(s, rows(s["k_cache"], dk), rows(s["v_cache"], dv), s["kv_lens"].long())


def _prompt_plain(s):
    cu = s["cu_kv"].long()
    j = (cu[:-1, None] + torch.arange(s["max_kv"], device="cuda")[None, :]).clamp(max=s["total_kv"] - 1)
    _, dk, dv = s["descales"]

    def rows(x, d):
        return _widen(x[j] if d is None else x.view(torch.uint8)[j], d)

    return _attend_plain(s, rows(s["k"], dk), rows(s["v"], dv), cu[1:] - cu[:-1])


# --------------------------------------------------------------------------- a pass --

def run(s):
    op = s["op"]
    if not own:
        return {"map": _map_plain, "write": _write_plain, "paged": _paged_plain, "prompt": _prompt_plain}[op](s)
    import split_kv_sparse_gb300 as skv
    if op == "map":
        skv.kv_pages_map(s["page"], s["held"], s["lens"], s["cu_q"], s["total_q"], s["table"], s["free_pages"],
                         s["free_in"], s["free_out"], s["slots"], s["positions"])
        return {"table": s["table"], "free_pages": s["free_pages"], "free": s["free_out"], "slots": s["slots"],
                "positions": s["positions"]}
    if op == "write":
        skv.kv_pages_write(s["pages_desc"], s["k"], s["v"], s["slots"], s["descale_k"], s["descale_v"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    dq, dk, dv = s["descales"]
    if op == "paged":
        skv.sdpa_paged(s["plan"], s["total_q"], s["q"], s["pages_desc"], s["table"], s["kv_lens"], s["cu_q"], dq, dk, dv,
                       s["scale"], "bf16", 1.0, s["out"], s["lse"], None, s["workspace"])
    else:
        skv.sdpa_prompt(s["batch"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_kv"], dq, dk, dv, s["scale"], "bf16", 1.0,
                        s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------- 64-bit values --

def exact(case, seed):
    if case["op"] == "map":
        return None          # whole numbers
    s = prepare(case, seed)
    if case["op"] == "write":
        # what a row's slot holds, from the nearest code of the quotient in 64 bits
        got = {}
        for name, w in (("k", "k"), ("v", "v")):
            cache = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device="cuda")
            flat = cache.view(-1, case["h_kv"], D)
            x = s[name].double()
            if case["dtype"] == "e4m3":
                x = x / s["descale_" + name].double()
                top = x.abs().clamp(max=448.0, min=2.0 ** -30)
                step = torch.exp2(torch.floor(torch.log2(top)).clamp(min=-6) - 3)
                x = torch.sign(x) * torch.round(top / step) * step
            keep = s["slots"] >= 0
            flat[s["slots"][keep]] = x[keep]
            got[name + "_cache"] = cache
        return got
    sq, kv = _lens(case)
    h_q, h_kv = case["h_q"], case["h_kv"]
    group = h_q // h_kv
    d = [1.0 if x is None else float(x.double().cpu()) for x in s["descales"]]
    out = torch.zeros((s["total_q"], h_q, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total_q"], h_q), dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(sq, kv)):
        if case["op"] == "paged":
            page = s["table"][b, :_pages(m, case["page"])].long()
            K, V = ((c.view(torch.uint8)[page].view(c.dtype) if c.dtype != torch.bfloat16 else c[page]).reshape(-1, h_kv, D)[:m]
                    for c in (s["k_cache"], s["v_cache"]))
        else:
            K, V = s["k"][k0:k0 + m], s["v"][k0:k0 + m]
        for j in range(h_kv):
            Kj, Vj = K[:, j].double() * d[1], V[:, j].double() * d[2]
            for t0 in range(0, n, 1024):
                t1 = min(n, t0 + 1024)
                end = m - n + t1      # keys that the block's last query sees
                qj = s["q"][q0 + t0:q0 + t1, j * group:(j + 1) * group].double() * d[0]
                x = torch.einsum("tgd,kd->tgk", qj, Kj[:end]) * s["scale"]
                at = torch.arange(m - n + t0, end, device="cuda")
                x = torch.where(torch.arange(end, device="cuda")[None, None, :] <= at[:, None, None], x, -math.inf)
                lse[q0 + t0:q0 + t1, j * group:(j + 1) * group] = torch.logsumexp(x, -1) / math.log(2)
                out[q0 + t0:q0 + t1, j * group:(j + 1) * group] = torch.einsum("tgk,kd->tgd", torch.softmax(x, -1), Vj[:end])
        q0 += n
        k0 += m
    return {"out": out, "lse": lse}
