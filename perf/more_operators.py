"""Cases of the append with the position rotation, of a K/V cache held in 4 bits (append, read-back) and of attention over it.

A case is a dict of plain values. ``prepare`` makes what a server has in hand before the call, ``run`` is one
pass through one operator: in its plain form (elementary torch operations in fp32, rounded once) where ``own``
is false, and through the library's entry points where it is true.

The 4-bit form: 16 consecutive dims share a scale in e4m3, e4m3(max|y| / 6) with y = x / descale, and each is
held as the e2m1 code of y / scale (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign; two codes a byte, the first in the low half).
"""
import math
import random

import torch

own = False

D = 128
GROUP = 16                                           # dims that share a scale
DESCALE8 = {"q": 0.0234, "k": 0.0242, "v": 0.0226}   # e4m3: about 5.2 of the largest standard deviations to 448
DESCALE4 = {"k": 0.0045, "v": 0.0043}                # 4 bits: as many to the largest scale, 448
FAR = 131072                                         # positions of the rotation's table


# --------------------------------------------------------------------------- cases --

def listed():
    return [
        # the rows of one decode step, queries and cache in e4m3: latency
        dict(name="rotary decode e4m3", op="rotary", dtype="e4m3", rows=8, h_q=32, h_kv=8, rot=128, inter=False, page=16,
             drop=0.0, mix=1),
        # a mixed step into a bf16 cache: half the dims rotated, neighbouring ones paired, padded to a captured size
        dict(name="rotary mixed bf16", op="rotary", dtype="bf16", rows=1037, h_q=16, h_kv=2, rot=64, inter=True, page=64,
             drop=0.1, mix=2),
        # prompt rows out of a fused projection into a bf16 cache
        dict(name="rotary prompt bf16", op="rotary", dtype="bf16", rows=16001, h_q=32, h_kv=8, rot=128, inter=False, page=64,
             drop=0.01, mix=3),
        # prompt rows into a 4-bit cache, and the cache's values of them for attention over the packed prompt
        dict(name="rotary prompt 4 bit", op="rotary", dtype="e2m1", rows=8192, h_q=32, h_kv=8, rot=128, inter=False, page=32,
             drop=0.0, mix=4),
        # one decode step's rows of a full server into a 4-bit cache without a rotation, and back
        dict(name="write read 4 bit", op="store", dtype="e2m1", rows=96, h_kv=8, page=16, drop=0.0, mix=5),
        # a cached prefix of 20,000 positions read back for attention over packed keys
        dict(name="read prefix 4 bit", op="read", dtype="e2m1", rows=20000, h_kv=8, page=64, drop=0.0, mix=6),
        # single-token decode of 8 requests over a 4-bit cache
        dict(name="decode 4 bit b8", op="paged", batch=8, h_q=32, h_kv=8, page=64, q_lo=1, q_hi=1, kv_lo=1024, kv_hi=16384,
             mix=7),
        # single-token decode of a full server, pages of 16
        dict(name="decode 4 bit b96", op="paged", batch=96, h_q=32, h_kv=8, page=16, q_lo=1, q_hi=1, kv_lo=100, kv_hi=12000,
             mix=8),
        # single-token decode at long contexts, 64 query heads over 8
        dict(name="decode 4 bit long", op="paged", batch=4, h_q=64, h_kv=8, page=128, q_lo=1, q_hi=1, kv_lo=100000,
             kv_hi=131072, mix=9),
        # 1 to 16 new tokens a sequence (speculative decoding)
        dict(name="few tokens 4 bit b8", op="paged", batch=8, h_q=32, h_kv=8, page=128, q_lo=1, q_hi=16, kv_lo=1024,
             kv_hi=16384, mix=10),
        # chunked prefill: ragged chunks of up to 600 tokens over long cached contexts, pages of 16
        dict(name="chunk 4 bit ragged", op="paged", batch=5, h_q=32, h_kv=8, page=16, q_lo=1, q_hi=600, kv_lo=2000,
             kv_hi=16384, mix=11),
        # one long chunk over a long cache
        dict(name="chunk 4 bit 2048", op="paged", batch=1, h_q=32, h_kv=8, page=64, q_lo=2048, q_hi=2048, kv_lo=32768,
             kv_hi=32768, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "store", "read", "paged", "paged", "paged", "paged"])
    mix = rng.randrange(1 << 20)
    h_kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        return dict(op=op, dtype=rng.choice(["bf16", "e4m3", "e2m1"]), rows=_log(rng, 1, 16000),
                    h_q=h_kv * rng.choice([1, 4, 5, 8] if h_kv < 8 else [1, 4]), h_kv=h_kv, rot=rng.choice([32, 64, 96, 128, 128]),
                    inter=rng.random() < 0.4, page=page, drop=rng.choice([0.0, 0.02, 0.2]), mix=mix)
    if op in ("store", "read"):
        return dict(op=op, dtype="e2m1" if op == "store" else rng.choice(["e2m1", "e2m1", "e4m3", "bf16"]),
                    rows=_log(rng, 1, 16000), h_kv=h_kv, page=page, drop=rng.choice([0.0, 0.05]), mix=mix)
    group = rng.choice([1, 2, 4, 4, 7, 8, 16] if h_kv <= 2 else [1, 2, 4, 4, 5, 8] if h_kv == 4 else [1, 2, 4, 8])
    kind = rng.choice(["decode", "decode", "few", "chunk"])
    batch = _log(rng, 1, 64) if kind == "decode" else _log(rng, 1, 12) if kind == "few" else _log(rng, 1, 4)
    q_hi = 1 if kind == "decode" else _log(rng, 2, 24) if kind == "few" else _log(rng, 33, 1000)
    kv_hi = _log(rng, max(64, q_hi), 16384)
    return dict(op=op, batch=batch, h_q=h_kv * group, h_kv=h_kv, page=rng.choice([16, 32, 64, 128, 256]), q_lo=1, q_hi=q_hi,
                kv_lo=_log(rng, 1, kv_hi), kv_hi=kv_hi, mix=mix)


def _lens(case):
    """(new tokens, keys) of each sequence: a property of the case, not of the seed of its values."""
    rng = random.Random(case["mix"])
    sq = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    kv = [max(rng.randint(case["kv_lo"], case["kv_hi"]), n) for n in sq]
    return sq, kv


def _positions(case):
    """Positions of the rows, sequence by sequence: runs of tokens that begin anywhere below FAR."""
    rng = random.Random(case["mix"])
    out = []
    while len(out) < case["rows"]:
        n = min(rng.randint(1, 1 + 2 * case["rows"] // 3), case["rows"] - len(out))
        first = rng.randint(0, FAR - n)
        out += range(first, first + n)
    return out


def _dropped(case):
    """Rows that a padded batch carries behind its tokens: no position, no slot."""
    return int(case["rows"] * case["drop"])


def _pages(n, page):
    return (n + page - 1) // page


_BYTES = {"bf16": 2 * D, "e4m3": D, "e2m1": D // 2 + D // GROUP}   # of a row and head of the cache


def work(case):
    if case["op"] == "rotary":
        live = case["rows"] - _dropped(case)
        q_out = D if case["dtype"] == "e4m3" else 2 * D
        moved = live * (case["h_q"] * (2 * D + q_out) + 2 * case["h_kv"] * (2 * D + _BYTES[case["dtype"]]) + 4 * case["rot"])
        if case["dtype"] == "e2m1":
            moved += live * 2 * case["h_kv"] * (_BYTES["e2m1"] + 2 * D)
        return {"bytes": moved + 12 * case["rows"], "flops": 0}
    if case["op"] in ("store", "read"):
        live, b = case["rows"] - _dropped(case), _BYTES[case["dtype"]]
        return {"bytes": live * 2 * case["h_kv"] * (2 * D + b) * (2 if case["op"] == "store" else 1) + 8 * case["rows"], "flops": 0}
    sq, kv = _lens(case)
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(sq, kv))
    moved = sum(sq) * case["h_q"] * (4 * D + 4) + sum(kv) * 2 * case["h_kv"] * _BYTES["e2m1"]
    moved += 4 * sum(_pages(m, case["page"]) for m in kv)
    return {"bytes": moved, "flops": 4 * D * case["h_q"] * pairs}


# ------------------------------------------------------------------- the 4-bit form --

def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _steps(a):
    """The nearest e2m1 magnitude of a >= 0, ties to the even code, at most 6."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return (torch.round(a / step) * step).clamp(max=6)


def _encode(y):
    """y [..., 128] (already divided by the descale) -> codes [..., 64], scales [..., 8], both bytes."""
    g = y.reshape(*y.shape[:-1], D // GROUP, GROUP)
    s = _e4m3(g.abs().amax(-1) / 6)
    w = s.float()[..., None]
    m = _steps(torch.where(w > 0, g.abs() / w, torch.zeros_like(g)))
    code = torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(g).to(torch.uint8) << 3)).reshape(y.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _decode(codes, scales):
    """The values, without the descale, in fp32 (exact)."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D)
    m = (c & 7).float()
    m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(c > 7, -m, m)
    return v * scales.view(torch.float8_e4m3fn).float().repeat_interleave(GROUP, -1)


# -------------------------------------------------------------------------- inputs --

def _cu(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _one(x):
    return torch.tensor([x], dtype=torch.float32, device="cuda")


def _keys(shape, g):
    """Normal values whose dims differ in size, as a projection's do."""
    x = torch.randn(shape, dtype=torch.float32, device="cuda", generator=g)
    return x.mul_(torch.exp2(torch.linspace(-1, 1, D, device="cuda")))


def _filled(which, pages, page, heads, g):
    """A 4-bit cache of earlier rows: codes [pages, page, heads, 64], scales [pages, heads, page, 8] as [pages, page, heads, 8]."""
    codes = torch.empty((pages, page, heads, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, heads, page, D // GROUP), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (page * heads * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        codes[p:p + n], s = _encode(_keys((n, page, heads, D), g) / DESCALE4[which])
        scales[p:p + n] = s.permute(0, 2, 1, 3)
    return codes, scales.permute(0, 2, 1, 3)


def _empty(dtype, pages, page, heads):
    if dtype == "e2m1":
        return (torch.zeros((pages, page, heads, D // 2), dtype=torch.uint8, device="cuda"),
                torch.zeros((pages, heads, page, D // GROUP), dtype=torch.uint8, device="cuda").permute(0, 2, 1, 3))
    t = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    return torch.zeros((pages, page, heads, D), dtype=t, device="cuda"), None


def _descales(dtype):
    if dtype == "bf16":
        return {"q": None, "k": None, "v": None}
    if dtype == "e4m3":
        return {w: _one(DESCALE8[w]) for w in "qkv"}
    return {"q": None, "k": _one(DESCALE4["k"]), "v": _one(DESCALE4["v"])}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    s["descales"] = _descales(case.get("dtype", "e2m1"))
    if case["op"] in ("rotary", "store", "read"):
        n, h, P, dtype = case["rows"], case["h_kv"], case["page"], case["dtype"]
        pages = _pages(n, P) + 8
        # rows fill pages that lie anywhere in the cache, in order within a page; the padding behind them has no slot
        order = torch.randperm(pages, device="cuda", generator=g)[:_pages(n, P)]
        slots = (order[:, None] * P + torch.arange(P, device="cuda")[None, :]).reshape(-1)[:n].clone()
        slots[n - _dropped(case):] = -1
        s["slots"] = slots
        if case["op"] == "read" and dtype == "e2m1":
            s["k_cache"], s["k_scales"] = _filled("k", pages, P, h, g)
            s["v_cache"], s["v_scales"] = _filled("v", pages, P, h, g)
        else:
            s["k_cache"], s["k_scales"] = _empty(dtype, pages, P, h)
            s["v_cache"], s["v_scales"] = _empty(dtype, pages, P, h)
            if case["op"] == "read":
                for w in "kv":
                    x = _keys((pages, P, h, D), g)
                    s[w + "_cache"] = x.to(torch.bfloat16) if dtype == "bf16" else _e4m3(x / DESCALE8[w])
        if case["op"] != "read":
            # queries, keys and values side by side, as a fused projection leaves them
            h_q = case.get("h_q", 4 * h)
            qkv = _keys((n, h_q + 2 * h, D), g).to(torch.bfloat16)
            s["q"], s["k"], s["v"] = qkv[:, :h_q], qkv[:, h_q:h_q + h], qkv[:, h_q + h:]
        if case["op"] == "rotary":
            pos = torch.tensor(_positions(case), dtype=torch.int32, device="cuda")
            pos[n - _dropped(case):] = -1
            s["positions"] = pos
            R = case["rot"]
            f = torch.pow(torch.tensor(500000.0, dtype=torch.float64, device="cuda"),
                          -torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
            angle = torch.arange(FAR, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
            s["q_out"] = torch.zeros((n, case["h_q"], D), device="cuda",
                                     dtype=torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16)
        s["k_out"], s["v_out"] = (torch.zeros((n, h, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if own:
            import split_kv_sparse_gb300 as skv
            s["pages_desc"] = skv.kv_pages(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
        return s
    sq, kv = _lens(case)
    h_q, h_kv, P = case["h_q"], case["h_kv"], case["page"]
    s["total_q"], s["max_q"], s["max_kv"] = sum(sq), max(sq), max(kv)
    s["q"] = torch.randn((s["total_q"], h_q, D), dtype=torch.float32, device="cuda", generator=g).to(torch.bfloat16)
    s["cu_q"], s["scale"] = _cu(sq), 1 / math.sqrt(D)
    s["out"] = torch.empty((s["total_q"], h_q, D), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((s["total_q"], h_q), dtype=torch.float32, device="cuda")
    held = [_pages(m, P) for m in kv]
    order = torch.randperm(sum(held) + 8, device="cuda", generator=g).to(torch.int32)
    s["k_cache"], s["k_scales"] = _filled("k", sum(held) + 8, P, h_kv, g)
    s["v_cache"], s["v_scales"] = _filled("v", sum(held) + 8, P, h_kv, g)
    s["table"] = torch.full((case["batch"], max(held)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        s["table"][b, :n] = order[at:at + n]
        at += n
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    if own:
        import split_kv_sparse_gb300 as skv
        s["pages_desc"] = skv.kv_pages(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
        s["plan"] = skv.sdpa_paged_plan(case["batch"], h_q, h_kv, D, "e2m1", s["max_q"], s["total_q"], s["max_kv"])
        n = s["plan"].workspace_bytes
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    return s


# --------------------------------------------------------------------- plain forms --

def _rotate(x, table, rot, inter):
    """x [rows, heads, 128] fp32 by the angles of its rows' positions: table [rows, rot], cosines then sines."""
    c, n = table[:, None, :rot // 2], table[:, None, rot // 2:]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _put(s, w, x, keep, src):
    """x [rows, heads, 128] fp32 into its slots; a row without one writes what row `src` says once more."""
    cache, scales, d = s[w + "_cache"], s[w + "_scales"], s["descales"][w]
    P = s["page"]
    page, row = s["slots"][src] // P, s["slots"][src] % P
    if s["dtype"] == "bf16":
        cache[page, row] = x.to(torch.bfloat16)[src]
    elif s["dtype"] == "e4m3":
        cache.view(torch.uint8)[page, row] = _e4m3(x / d).view(torch.uint8)[src]
    else:
        codes, sc = _encode(x / d)
        cache[page, row] = codes[src]
        scales[page, row] = sc[src]


def _get(s, w, keep, src):
    """The values of the rows' slots in bf16; a row without one keeps what its place holds."""
    cache, scales, d = s[w + "_cache"], s[w + "_scales"], s["descales"][w]
    P, out = s["page"], s[w + "_out"]
    page, row = s["slots"][src] // P, s["slots"][src] % P
    if s["dtype"] == "bf16":
        x = cache[page, row]
    elif s["dtype"] == "e4m3":
        x = (cache.view(torch.uint8)[page, row].view(torch.float8_e4m3fn).float() * d).to(torch.bfloat16)
    else:
        x = (_decode(cache[page, row], scales[page, row]) * d).to(torch.bfloat16)
    out.copy_(torch.where(keep[:, None, None], x, out))
    return out


def _live(s):
    keep = s["slots"] >= 0
    at = torch.arange(keep.numel(), device="cuda")
    return keep, torch.where(keep, at, keep.long().argmax())


def _rows_plain(s):
    keep, src = _live(s)
    got = {}
    if s["op"] != "read":
        k, v = s["k"].float(), s["v"].float()
        if s["op"] == "rotary":
            table = s["cos_sin"][s["positions"].long().clamp(min=0)]
            k = _rotate(k, table, s["rot"], s["inter"])
            q = _rotate(s["q"].float(), table, s["rot"], s["inter"])
            if s["dtype"] == "e4m3":
                q = _e4m3(q / s["descales"]["q"]).view(torch.uint8)
                out = s["q_out"].view(torch.uint8)
            else:
                q, out = q.to(torch.bfloat16), s["q_out"]
            out.copy_(torch.where(keep[:, None, None], q, out))
            got["q"] = s["q_out"]
        _put(s, "k", k, keep, src)
        _put(s, "v", v, keep, src)
    if s["op"] == "rotary" and s["dtype"] != "e2m1":
        return {**got, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {**got, "k": _get(s, "k", keep, src), "v": _get(s, "v", keep, src)}


def _attend_plain(s):
    P = s["page"]
    j = torch.arange(s["max_kv"], device="cuda")
    page = s["table"].long()[:, j // P].clamp(min=0)
    row = (j % P).expand_as(page)
    B, L, M = s["batch"], s["max_kv"], s["max_q"]
    h_q, h_kv = s["h_q"], s["h_kv"]
    group = h_q // h_kv
    K, V = (_decode(s[w + "_cache"][page, row], s[w + "_scales"][page, row]).mul_(s["descales"][w]) for w in "kv")
    cu, kv_len = s["cu_q"].long(), s["kv_lens"].long()
    sq = cu[1:] - cu[:-1]
    i = torch.arange(M, device="cuda")
    q = s["q"][(cu[:-1, None] + i[None, :]).clamp(max=s["total_q"] - 1)].float()
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


# --------------------------------------------------------------------------- a pass --

def run(s):
    op = s["op"]
    if not own:
        return _attend_plain(s) if op == "paged" else _rows_plain(s)
    import split_kv_sparse_gb300 as skv
    d = s["descales"]
    if op == "paged":
        skv.sdpa_paged(s["plan"], s["total_q"], s["q"], s["pages_desc"], s["table"], s["kv_lens"], s["cu_q"], None, d["k"],
                       d["v"], s["scale"], "bf16", 1.0, s["out"], s["lse"], None, s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    got = {}
    if op == "rotary":
        skv.kv_pages_write_rotary(s["pages_desc"], s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["q_out"],
                                  interleaved=s["inter"], descale_q=d["q"], descale_k=d["k"], descale_v=d["v"])
        got["q"] = s["q_out"]
        if s["dtype"] != "e2m1":
            return {**got, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    elif op == "store":
        skv.kv_pages_write(s["pages_desc"], s["k"], s["v"], s["slots"], d["k"], d["v"])
    skv.kv_pages_read(s["pages_desc"], s["slots"], s["k_out"], s["v_out"], d["k"], d["v"])
    return {**got, "k": s["k_out"], "v": s["v_out"]}


# --------------------------------------------------------------------- 64-bit values --

_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values64(codes, scales):
    """What the codes and scales of a 4-bit cache stand for, from the table of its 16 values."""
    t = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float64, device="cuda")
    v = torch.empty((*codes.shape[:-1], D), dtype=torch.float64, device="cuda")
    v[..., 0::2], v[..., 1::2] = t[(codes & 15).long()], t[(codes >> 4).long()]
    return (v.unflatten(-1, (D // GROUP, GROUP)) * scales.view(torch.float8_e4m3fn).double()[..., None]).flatten(-2)


def _near8(x):
    """The nearest e4m3 value."""
    top = x.abs().clamp(max=448.0, min=2.0 ** -30)
    step = torch.exp2(torch.floor(torch.log2(top)).clamp(min=-6) - 3)
    return torch.sign(x) * torch.round(top / step) * step


def _near4(x):
    """The value that 16 dims of x are held as."""
    g = x.unflatten(-1, (D // GROUP, GROUP))
    s = _near8(g.abs().amax(-1, keepdim=True) / 6)
    a = torch.where(s > 0, g.abs() / s, 0.0)
    t = torch.tensor(_VALUES, dtype=torch.float64, device="cuda")
    best = torch.zeros_like(a)
    for k in range(1, 8):      # from value k on, where a lies past the middle (a tie goes to the even code)
        mid = (t[k - 1] + t[k]) / 2
        best = torch.where((a > mid) | ((a == mid) & (k % 2 == 0)), t[k], best)
    return (torch.sign(g) * best * s).flatten(-2)


def _exact_rows(case, s):
    keep = s["slots"] >= 0
    dtype, d = case["dtype"], {w: 1.0 if x is None else float(x.double().cpu()) for w, x in s["descales"].items()}
    got, P = {}, case["page"]
    if case["op"] != "read":
        x = {w: s[w].double() for w in "qkv"}
        if case["op"] == "rotary":
            R, t = case["rot"], s["cos_sin"][s["positions"].long().clamp(min=0)].double()
            turn = torch.complex(t[:, :R // 2], t[:, R // 2:])[:, None]
            for w in "qk":
                a = x[w][..., :R]
                pair = a.unflatten(-1, (R // 2, 2)) if case["inter"] else a.unflatten(-1, (2, R // 2)).transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
                z = z if case["inter"] else z.transpose(-1, -2)
                x[w] = torch.cat([z.flatten(-2), x[w][..., R:]], -1)
            q = x["q"] if dtype != "e4m3" else _near8(x["q"] / d["q"])
            got["q"] = torch.where(keep[:, None, None], q, 0.0)
        for w in "kv":
            y = x[w] if dtype == "bf16" else _near8(x[w] / d[w]) if dtype == "e4m3" else _near4(x[w] / d[w]) * d[w]
            if dtype == "e2m1":
                got[w] = torch.where(keep[:, None, None], y, 0.0)
            else:
                cache = torch.zeros(s[w + "_cache"].shape, dtype=torch.float64, device="cuda")
                cache.view(-1, case["h_kv"], D)[s["slots"][keep]] = y[keep]
                got[w + "_cache"] = cache
        return got
    at = s["slots"].clamp(min=0)
    for w in "kv":
        cache = s[w + "_cache"]
        if dtype == "e2m1":
            y = _values64(cache[at // P, at % P], s[w + "_scales"][at // P, at % P])
        elif dtype == "e4m3":
            y = cache.view(torch.uint8)[at // P, at % P].view(torch.float8_e4m3fn).double()
        else:
            y = cache[at // P, at % P].double()
        got[w] = torch.where(keep[:, None, None], y * d[w], 0.0)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "paged":
        return _exact_rows(case, s)
    sq, kv = _lens(case)
    h_q, h_kv = case["h_q"], case["h_kv"]
    group = h_q // h_kv
    d = {w: float(s["descales"][w].double().cpu()) for w in "kv"}
    out = torch.zeros((s["total_q"], h_q, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total_q"], h_q), dtype=torch.float64, device="cuda")
    q0 = 0
    for b, (n, m) in enumerate(zip(sq, kv)):
        page = s["table"][b, :_pages(m, case["page"])].long()
        for j in range(h_kv):
            K, V = (_values64(s[w + "_cache"][page, :, j].reshape(-1, D // 2)[:m],
                              s[w + "_scales"][page, :, j].reshape(-1, D // GROUP)[:m]) * d[w] for w in "kv")
            for t0 in range(0, n, 1024):
                t1 = min(n, t0 + 1024)
                end = m - n + t1      # keys that the block's last query sees
                qj = s["q"][q0 + t0:q0 + t1, j * group:(j + 1) * group].double()
                x = torch.einsum("tgd,kd->tgk", qj, K[:end]) * s["scale"]
                at = torch.arange(m - n + t0, end, device="cuda")
                x = torch.where(torch.arange(end, device="cuda")[None, None, :] <= at[:, None, None], x, -math.inf)
                lse[q0 + t0:q0 + t1, j * group:(j + 1) * group] = torch.logsumexp(x, -1) / math.log(2)
                out[q0 + t0:q0 + t1, j * group:(j + 1) * group] = torch.einsum("tgk,kd->tgd", torch.softmax(x, -1), V[:end])
        q0 += n
    return {"out": out, "lse": lse}
