"""GPU tests of the append that rotates (kv_pages_write_rotary), of the append into 4-bit pages and of the way back
(kv_pages_read), against the oracle.

Tolerances against the fp64 values, from the arithmetic: a rotated value is two products and a sum in fp32, each off by at
most 2^-24 of itself, so y is off by at most t = 2^-23 (|x_i c| + |x_j s|). Beside that a bf16 result is off by 2^-8 |y|, an e4m3
one (of y / descale, one more rounding of 2^-24, within t / descale as |y| <= |x_i c| + |x_j s|, doubled below) by 2^-4 |y| or half its smallest step, 2^-10
descale. A 4-bit value under scale s is off by half a step of e2m1, s / 4 up to 2 s, s / 2 up to 4 s, s above (its saturation
at 6 too: s is at least (1 - 2^-4) of amax / 6, so y / s ends at 6.4). Bytes are held to the same arithmetic in fp32 exactly."""
import numpy as np
import pytest
import torch

import oracle.paged as op
from _four_bit_util import caches, f32, on_gpu, table_of
from _paged_util import D, status_clear
from oracle import codecs
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


def bf16_bytes(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def held(y, d, dtype):
    """The bytes of fp32 values y: bf16, e4m3 codes, or (codes, scales)."""
    if dtype == "bf16":
        return bf16_bytes(y), None
    with np.errstate(all="ignore"):
        q = (y / np.float32(d)).astype(np.float32)
    if dtype == "e4m3":
        return torch.from_numpy(codecs.e4m3_encode(np.clip(q, -448, 448).astype(np.float64))), None
    c, s = op.four_bit_encode(q)
    return torch.from_numpy(c), torch.from_numpy(s)


def slots_of(rows, n_slots, g, drop):
    slots = torch.randperm(n_slots, generator=g)[:rows]
    if drop:
        slots[1::5] = torch.tensor([-1, n_slots, -9, 1 << 40])[torch.arange(len(slots[1::5])) % 4]
    return slots


def same_rows(cache, want, slots, fill):
    """Rows of the cache by slot: those named are `want`, all others still hold the byte `fill`."""
    flat = cache.cpu().contiguous().view(torch.uint8).flatten(0, 1)
    full = torch.full_like(flat, fill)
    keep = (slots >= 0) & (slots < flat.shape[0])
    full[slots[keep]] = want.contiguous().view(torch.uint8).reshape(len(slots), *flat.shape[1:])[keep]
    assert torch.equal(flat, full)


def turned_error(x, cs, pos, inter):
    """|x_i c| + |x_j s| of every dim: the scale of a rotation's rounding errors."""
    a = op.rotate(np.abs(x), np.abs(cs) * np.concatenate([np.ones(cs.shape[1] // 2), -np.ones(cs.shape[1] // 2)]), pos, inter)
    z = op.rotate(np.abs(x), np.abs(cs), pos, inter)
    return np.maximum(np.abs(a), np.abs(z))


def go(dtype, rows, h_q, h_kv, rot, inter, page=16, layout="row", fused=True, q_type="bf16", k_out=False, drop=True, pad=0, in_place=False,
       seed=0):
    g = torch.Generator().manual_seed(seed + rows)
    n_pages = -(-rows // page) + 3
    dq, dk, dv = 0.021, 0.013 if dtype == "e4m3" else 0.004, 0.017 if dtype == "e4m3" else 0.003
    x = torch.randn((rows, h_q + 2 * h_kv, D), generator=g).to(torch.bfloat16)
    positions = torch.randint(0, 500, (rows,), generator=g, dtype=torch.int32)
    if pad:
        positions[rows - pad:] = torch.tensor([-1, 500, 1 << 30], dtype=torch.int32)[torch.arange(pad) % 3]
    cs = table_of(500, rot)
    slots = slots_of(rows, n_pages * page, g, drop)
    dev = x.cuda()
    if not fused:
        q, k, v = (dev[:, i:j].contiguous() for i, j in ((0, h_q), (h_q, h_q + h_kv), (h_q + h_kv, h_q + 2 * h_kv)))
    else:
        q, k, v = dev[:, :h_q], dev[:, h_q:h_q + h_kv], dev[:, h_q + h_kv:]
    fill = 3
    mem = [on_gpu(c) for c in caches(dtype, n_pages, page, h_kv, layout, fill=fill)]
    q_out = None if in_place or not h_q else torch.full((rows, h_q, D), 9, dtype=torch.bfloat16 if q_type == "bf16" else torch.uint8, device="cuda")
    ko = (k if in_place else torch.full((rows, h_kv, D), 9, dtype=torch.bfloat16, device="cuda")) if k_out else None
    b.kv_pages_write_rotary(b.kv_pages(*mem), q if h_q else None, k, v, positions.cuda(), cs.cuda(), slots.cuda(), q_out, ko, interleaved=inter,
                            descale_q=f32(dq) if q_type == "e4m3" else None, descale_k=f32(dk), descale_v=f32(dv))
    torch.cuda.synchronize()
    f = x.float().numpy()
    pos, c = positions.numpy(), cs.numpy()
    live = torch.from_numpy((pos >= 0) & (pos < 500))
    y = op.rotate(f[:, :h_q + h_kv], c, pos, inter)
    exact = op.rotate(f[:, :h_q + h_kv].astype(np.float64), c.astype(np.float64), pos, inter)
    t = 2.0 ** -23 * turned_error(f[:, :h_q + h_kv].astype(np.float64), c.astype(np.float64), pos, inter)
    slots = torch.where(live, slots, -1)
    if h_q:
        got = (q if in_place else q_out).cpu()
        want = held(y[:, :h_q], dq, q_type)[0]
        old = x[:, :h_q] if in_place else torch.full_like(want, 9)
        assert torch.equal(got.view(torch.uint8), torch.where(live[:, None, None], want, old).view(torch.uint8))
        value = got[live].double().numpy() if q_type == "bf16" else codecs.e4m3_decode(got[live].numpy()) * np.float32(dq)
        e, tt = exact[:, :h_q][live.numpy()], t[:, :h_q][live.numpy()]
        assert np.all(np.abs(value - e) <= (2.0 ** -8 * np.abs(e) + tt if q_type == "bf16"
                                            else np.maximum(2.0 ** -4 * np.abs(e), 2.0 ** -10 * dq) + 2 * tt))
    if k_out:
        old = x[:, h_q:h_q + h_kv] if in_place else torch.full((rows, h_kv, D), 9, dtype=torch.bfloat16)
        assert torch.equal(ko.cpu(), torch.where(live[:, None, None], bf16_bytes(y[:, h_q:]), old))
    for cache, scales, z, e, tt, d in ((mem[0], mem[2], y[:, h_q:], exact[:, h_q:], t[:, h_q:], dk),
                                       (mem[1], mem[3], f[:, h_q + h_kv:], f[:, h_q + h_kv:].astype(np.float64), 0 * t[:, h_q:], dv)):
        codes, s = held(z, d, dtype)
        same_rows(cache, codes, slots, fill)
        if dtype == "e2m1":
            same_rows(scales, s, slots, fill)
            sc = np.repeat(codecs.e4m3_decode(s.numpy()), 16, -1) * np.float32(d)
            err = np.abs(op.four_bit_decode(codes.numpy(), s.numpy()) * np.float32(d) - e)
            a = np.abs(e)
            assert np.all(err <= np.where(a < 2 * sc, sc / 4, np.where(a < 4 * sc, sc / 2, sc)) + 2 * tt + 2.0 ** -20 * a)
        elif dtype == "bf16":
            assert np.all(np.abs(codes.double().numpy() - e) <= 2.0 ** -8 * np.abs(e) + tt)
        else:
            err = np.abs(codecs.e4m3_decode(codes.numpy()) * np.float32(d) - e)
            assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(e), 2.0 ** -10 * d) + 2 * tt)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (64, False), (64, True), (32, False), (96, False), (96, True)])
def test_rotary_forms(dtype, rot, inter):
    go(dtype, 37, 8, 2, rot, inter, seed=rot)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("rows,h_q,h_kv,page,layout,fused", [
    (1, 1, 1, 16, "row", False), (7, 5, 1, 16, "head", True), (333, 32, 8, 64, "head", True), (1000, 14, 2, 32, "row", False),
    (1500, 32, 8, 128, "row", True), (50, 0, 3, 16, "row", True)])
def test_rotary_sizes(dtype, rows, h_q, h_kv, page, layout, fused):
    go(dtype, rows, h_q, h_kv, 128, False, page, layout, fused, pad=min(3, rows - 1), seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("in_place", [False, True])
def test_rotary_into_codes_in_place_and_beside(dtype, in_place):
    """Queries as e4m3 codes; queries and keys turned in place; rotated keys beside the cache."""
    if not in_place:
        go(dtype, 65, 8, 2, 128, False, q_type="e4m3", k_out=True, pad=4, seed=2)
        go(dtype, 65, 8, 2, 64, True, q_type="e4m3", k_out=True, pad=4, seed=2)
    for fused in (True, False):
        go(dtype, 65, 8, 2, 128, False, k_out=True, in_place=in_place, fused=fused, pad=4, seed=3)
        go(dtype, 2000, 32, 8, 96, True, k_out=True, in_place=in_place, fused=fused, pad=4, seed=3)


def test_rotary_without_rows_and_with_all_rows_padding():
    x = torch.ones((3, 4, D), dtype=torch.bfloat16, device="cuda")
    k, v = caches("bf16", 2, 16, 1, device="cuda")[:2]
    pages, cs = b.kv_pages(k, v), table_of(8, 128).cuda()
    b.kv_pages_write_rotary(pages, x[:0, :2], x[:0, 2:3], x[:0, 3:], torch.zeros(0, dtype=torch.int32, device="cuda"), cs,
                            torch.zeros(0, dtype=torch.int64, device="cuda"))
    b.kv_pages_write_rotary(pages, x[:, :2], x[:, 2:3], x[:, 3:], torch.full((3,), 8, dtype=torch.int32, device="cuda"), cs,
                            torch.arange(3, device="cuda"))
    torch.cuda.synchronize()
    assert not k.any() and not v.any() and (x == 1).all()


# ------------------------------------------------------------------------ 4 bits --

@pytest.mark.parametrize("rows,h_kv,page,layout", [(1, 1, 16, "row"), (7, 2, 16, "head"), (333, 8, 64, "row"), (2500, 5, 32, "row")])
def test_write_four_bits(rows, h_kv, page, layout):
    g = torch.Generator().manual_seed(rows)
    n_pages = -(-rows // page) + 3
    qkv = (torch.randn((rows, 4 * h_kv, D), generator=g) * torch.exp2(torch.linspace(-6, 6, D))).to(torch.bfloat16)
    k, v = qkv[:, 2 * h_kv:3 * h_kv], qkv[:, 3 * h_kv:]
    mem = [on_gpu(c) for c in caches("e2m1", n_pages, page, h_kv, layout, fill=3)]
    slots = slots_of(rows, n_pages * page, g, True)
    d = 0.037
    dev = qkv.cuda()
    b.kv_pages_write(b.kv_pages(*mem), dev[:, 2 * h_kv:3 * h_kv], dev[:, 3 * h_kv:], slots.cuda(), f32(d), None)
    torch.cuda.synchronize()
    for cache, scales, x, by in ((mem[0], mem[2], k, d), (mem[1], mem[3], v, 1.0)):
        c, s = held(x.float().numpy(), by, "e2m1")
        same_rows(cache, c, slots, 3)
        same_rows(scales, s, slots, 3)


def test_write_four_bits_special_values():
    """Infinities and values past the largest end at 6 * 448, a NaN makes its 16 dims NaN and no others, groups that are zero or
    too small for a scale are zeros, ties go to the even code."""
    x = torch.zeros((1, 1, D), dtype=torch.bfloat16)
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2] = float("inf"), -float("inf"), 448.0
    x[0, 0, 16], x[0, 0, 17] = float("nan"), 3.0
    x[0, 0, 32:36] = torch.tensor([1e-5, -1e-5, 2e-5, -0.0])
    x[0, 0, 48:64] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5])
    x[0, 0, 64], x[0, 0, 65] = 1e30, 2688.0
    mem = caches("e2m1", 1, 16, 1, device="cuda")
    pages, at = b.kv_pages(*mem), torch.zeros(1, dtype=torch.int64, device="cuda")
    b.kv_pages_write(pages, x.cuda(), x.cuda(), at)
    out = [torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    b.kv_pages_read(pages, at, *out)
    torch.cuda.synchronize()
    y = out[0].cpu()[0, 0].float()
    assert torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))
    assert y[:3].tolist() == [2688.0, -2688.0, 448.0] and not y[3:16].any()
    assert torch.isnan(y[16:32]).all()
    assert not y[32:48].any()
    up = [6, 0, 1, 1, 2, 2, 4, 4]
    assert y[48:64].tolist() == up + [-u for u in up]
    assert y[64:66].tolist() == [2688.0, 2688.0] and not y[66:].any()


@pytest.mark.parametrize("descale", [0.013, 1.0, 3.0, 1e-20, 7e30, 2.0 ** -126, 1e-39, 0.0, float("inf")])
def test_four_bit_codes_divide_as_divisions_do(descale):
    """Every finite bf16 value, in groups of like and of unlike magnitude, at descales whose quotients leave every range."""
    bits = torch.arange(65536, dtype=torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    bits = torch.cat([bits, bits[torch.randperm(len(bits), generator=torch.Generator().manual_seed(1))]])
    x = bits[:len(bits) // D * D].to(torch.int16).view(torch.bfloat16).reshape(-1, 1, D)
    n = x.shape[0]
    mem = caches("e2m1", -(-n // 16), 16, 1, device="cuda")
    b.kv_pages_write(b.kv_pages(*mem), x.cuda(), x.cuda(), torch.arange(n, device="cuda"), f32(descale), f32(descale))
    with np.errstate(all="ignore"):
        y = (x.float().numpy() / np.float32(descale)).astype(np.float32)     # IEEE division, subnormals and all
    amax = np.abs(y.reshape(n, 8, 16)).max(-1)
    nan = np.isnan(y.reshape(n, 8, 16)).any(-1)
    got_c, got_s = mem[0].cpu().reshape(-1, D // 2)[:n].numpy(), mem[2].cpu().reshape(-1, 8)[:n].numpy()
    assert np.all((got_s[nan] & 0x7F) == 0x7F)
    with np.errstate(all="ignore"):
        want_s = codecs.e4m3_encode(np.minimum((amax / np.float32(6)).astype(np.float32), 448).astype(np.float64))
    assert np.array_equal(got_s[~nan], want_s[~nan])
    want_c, _ = op.four_bit_encode(np.clip(np.nan_to_num(y, nan=0.0, posinf=1e30, neginf=-1e30), -1e30, 1e30)[:, 0])
    a, w = (op.four_bit_decode(c, np.full((n, 8), 0x38)).reshape(n, 8, 16) for c in (got_c, want_c))
    assert np.array_equal(a[~nan], w[~nan])
    assert torch.equal(mem[0], mem[1]) and torch.equal(mem[2], mem[3])


# ------------------------------------------------------------------------- read --

@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("rows,h_kv,page,layout", [(1, 1, 16, "row"), (9, 2, 16, "head"), (700, 8, 64, "row"), (3000, 3, 16, "head")])
def test_read(dtype, rows, h_kv, page, layout):
    """Every code under every scale that is a number; slots in any order, some twice, some outside the cache."""
    g = torch.Generator().manual_seed(rows)
    n_pages = 40
    mem = caches(dtype, n_pages, page, h_kv, layout)
    for c in mem:
        if c is not None:
            c.copy_(torch.randint(0, 256, c.shape, generator=g, dtype=torch.uint8) if c.dtype == torch.uint8
                    else torch.randn(c.shape, generator=g).to(torch.bfloat16))
    for c in (mem if dtype == "e4m3" else mem[2:]):
        if c is not None:
            c[(c & 0x7F) == 0x7F] = 0x11
    slots = torch.randint(-3, n_pages * page + 3, (rows,), generator=g)
    dk, dv = 0.013, 1.7
    kv = torch.full((rows, 2 * h_kv + 1, D), 9, dtype=torch.bfloat16, device="cuda")
    b.kv_pages_read(b.kv_pages(*(on_gpu(c) for c in mem)), slots.cuda(), kv[:, 1:1 + h_kv], kv[:, 1 + h_kv:], f32(dk), f32(dv))
    torch.cuda.synchronize()
    got = kv.cpu()
    assert (got[:, 0] == 9).all()
    keep = (slots >= 0) & (slots < n_pages * page)
    for i, (c, s, d) in enumerate(((mem[0], mem[2], dk), (mem[1], mem[3], dv))):
        flat = c.reshape(n_pages * page, h_kv, -1)
        if dtype == "bf16":
            want = flat
        else:
            value = codecs.e4m3_decode(flat.numpy()) if dtype == "e4m3" else op.four_bit_decode(flat.numpy(), s.reshape(n_pages * page, h_kv, -1).numpy())
            want = bf16_bytes(value.astype(np.float32) * np.float32(d))
        want = torch.where(keep[:, None, None], want[slots.clamp(0, n_pages * page - 1)], torch.tensor(9, dtype=torch.bfloat16))
        assert torch.equal(got[:, 1 + i * h_kv:1 + (i + 1) * h_kv], want)


def test_rows_behind_32_bit_offsets():
    """Pages of codes that lie more than 2^32 bytes from the base."""
    page, stride = 16, (1 << 31) + 4096
    big = torch.zeros(3 * stride, dtype=torch.uint8, device="cuda")
    k = big.as_strided((3, page, 1, D // 2), (stride, D, D, 1))
    v = big.as_strided((3, page, 1, D // 2), (stride, D, D, 1), D // 2)
    ks = big.as_strided((3, page, 1, 8), (stride, 8, 16 * page, 1), 8192 - 4096)
    vs = big.as_strided((3, page, 1, 8), (stride, 8, 16 * page, 1), 8192 - 4096 + 512)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((20, 2, D), generator=g).to(torch.bfloat16)
    slots = torch.arange(20) + page + 4
    pages = b.kv_pages(k, v, ks, vs)
    b.kv_pages_write(pages, x[:, :1].cuda(), x[:, 1:].cuda(), slots.cuda(), f32(0.004), f32(0.004))
    out = [torch.zeros((20, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    b.kv_pages_read(pages, slots.cuda(), *out, f32(0.004), f32(0.004))
    torch.cuda.synchronize()
    for i in range(2):
        c, s = held(x[:, i:i + 1].float().numpy(), 0.004, "e2m1")
        assert torch.equal(out[i].cpu(), bf16_bytes(op.four_bit_decode(c.numpy(), s.numpy()).astype(np.float32) * np.float32(0.004)))
    del big, k, v, ks, vs
    torch.cuda.empty_cache()


def test_positions_behind_32_bit_offsets():
    """A table of rotations of more than 2^31 entries, read at its end: a quarter turn there takes a head's halves into one another."""
    n = (1 << 24) + 6
    cs = torch.zeros((n, D), device="cuda")
    cs[n - 1, D // 2:] = 1
    x = torch.randn((1, 3, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    k, v = caches("bf16", 1, 16, 1, device="cuda")[:2]
    dev, out = x.cuda(), torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    b.kv_pages_write_rotary(b.kv_pages(k, v), dev[:, :1], dev[:, 1:2], dev[:, 2:], torch.tensor([n - 1], dtype=torch.int32, device="cuda"), cs,
                            torch.tensor([3], device="cuda"), out)
    torch.cuda.synchronize()
    turn = lambda y: torch.cat([-y[..., D // 2:], y[..., :D // 2]], -1)
    assert torch.equal(out.cpu(), turn(x[:, :1])) and torch.equal(k[0, 3].cpu(), turn(x[0, 1:2])) and torch.equal(v[0, 3].cpu(), x[0, 2:])
    del cs
    torch.cuda.empty_cache()
