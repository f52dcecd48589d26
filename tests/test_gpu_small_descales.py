"""GPU tests of the appends at descales near fp32's smallest numbers: codes are those of fp32 divisions there too, bit for bit.
The short way to a quotient needs its residual exactly, which fp32 does not hold below 2^-149; the descales are such that a
quotient lies within a rounding of the middle of two codes, or of two scales, and those where the two ways meet."""
import numpy as np
import pytest
import torch

import oracle.paged as op
from _four_bit_util import caches, f32
from _paged_util import D, status_clear
from oracle import codecs
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu

DESCALES = [float.fromhex(h) for h in (
    "0x1.fffffep-125", "0x1.ef7be0p-126", "0x1.e38e3ap-124", "0x1.3dcb08p-126", "0x1.fffffep-119", "0x1.d55554p-119", "0x1.a9fffep-116",
    "0x1.aaaaacp-123", "0x1.fb8240p-123", "0x1.04bda2p-125", "0x1.555556p-109", "0x1.fffffep-91", "0x1p-90", "0x1.000002p-90", "-0x1.ef7be0p-126")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


def rows():
    """Every finite bf16 value, 16 times in a group of its own, then all of them in groups of unlike ones: [n, 1, 128]."""
    bits = torch.arange(65536, dtype=torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    mixed = bits[torch.randperm(len(bits), generator=torch.Generator().manual_seed(1))]
    bits = torch.cat([bits.repeat_interleave(16), mixed])
    return bits[:len(bits) // D * D].to(torch.int16).view(torch.bfloat16).reshape(-1, 1, D)


def quotients(x, d):
    with np.errstate(all="ignore"):
        return (x.float().numpy() / np.float32(d)).astype(np.float32)


@pytest.mark.parametrize("rotary", [False, True])
@pytest.mark.parametrize("dtype", ["e4m3", "e2m1"])
@pytest.mark.parametrize("descale", DESCALES)
def test_codes_divide_as_divisions_do(descale, dtype, rotary):
    x = rows()
    n = x.shape[0]
    mem = caches(dtype, -(-n // 16), 16, 1, device="cuda")
    pages, dev, slots = b.kv_pages(*mem), x.cuda(), torch.arange(n, device="cuda")
    if rotary:
        # (by a quarter turn a pair (x, 0) becomes (0, x): k's second half is 0, and its first arrives there)
        k = dev.clone()
        k[..., D // 2:] = 0
        cs = torch.cat([torch.zeros((1, D // 2)), torch.ones((1, D // 2))], 1).cuda()
        b.kv_pages_write_rotary(pages, None, k, dev, torch.zeros(n, dtype=torch.int32, device="cuda"), cs, slots, descale_k=f32(descale),
                                descale_v=f32(descale))
        turned = torch.zeros_like(x)
        turned[..., D // 2:] = x[..., :D // 2]
    else:
        b.kv_pages_write(pages, dev, dev, slots, f32(descale), f32(descale))
        turned = x
    torch.cuda.synchronize()
    for i, rows_in in enumerate((turned, x)):
        y = quotients(rows_in, descale)
        got = mem[i].cpu().reshape(-1, mem[i].shape[-1])[:n].numpy()
        if dtype == "e4m3":
            want = codecs.e4m3_encode(np.clip(y[:, 0], -448, 448).astype(np.float64))
            # (the sign of a turned half's zeros is that of 0 - x 1 or x 1 + 0 0)
            assert np.array_equal(np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want))
            continue
        scales = mem[2 + i].cpu().reshape(-1, 8)[:n].numpy()
        with np.errstate(all="ignore"):
            amax = np.abs(y.reshape(n, 8, 16)).max(-1)
            want_s = codecs.e4m3_encode(np.minimum((amax / np.float32(6)).astype(np.float32), 448).astype(np.float64))
        assert np.array_equal(scales, want_s)
        want, _ = op.four_bit_encode(np.clip(y, -1e30, 1e30)[:, 0])
        a, w = (op.four_bit_decode(c, np.full((n, 8), 0x38)) for c in (got, want))
        assert np.array_equal(a, w)
