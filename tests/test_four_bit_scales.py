"""Codes of a 4-bit cache under every scale. A quotient by a scale goes by its reciprocal: an approximation within 1 ulp (which
the instruction promises) and one Newton step in FMAs, which has to be the rounded reciprocal for the quotients to be rounded divisions."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import codecs
from split_kv_sparse_gb300 import binding as b

SCALES = codecs.e4m3_decode(np.arange(1, 127, dtype=np.uint8))
TIES = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def rounded(x):
    """The fp32 value nearest to a fraction in the range of normal numbers, ties to even."""
    if x == 0:
        return Fraction(0)
    a, e = abs(x), 0
    while a >= 2:
        a, e = a / 2, e + 1
    while a < 1:
        a, e = a * 2, e - 1
    step = Fraction(2) ** (e - 23)
    return round(x / step) * step      # (round of a fraction takes ties to even)


@pytest.mark.parametrize("off", [-1, 0, 1])
def test_one_newton_step_gives_the_rounded_reciprocal(off):
    assert len(SCALES) == 126 and SCALES[-1] == 448
    for s in SCALES:
        s = Fraction(float(s))
        want = rounded(1 / s)
        r = Fraction(float(np.float32(float(want))))
        for _ in range(abs(off)):
            r = Fraction(float(np.nextafter(np.float32(float(r)), np.float32(off * 1e30))))
        error = rounded(1 - s * r)
        assert rounded(r + error * r) == want, float(s)


@pytest.mark.gpu
def test_codes_at_the_middles_of_two_under_every_scale():
    """The largest of 16 dims is 6 scales, so the scale is known; the others lie at the middles of two codes, which go to the even
    one, and a bf16 step on either side."""
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    groups = []
    for s in SCALES:
        mid = torch.tensor([t * s for t in TIES], dtype=torch.bfloat16)
        assert torch.equal(mid.double(), torch.tensor([t * s for t in TIES], dtype=torch.float64))
        bits = mid.view(torch.int16)
        y = torch.cat([mid, (bits + 1).view(torch.bfloat16), (bits - 1).view(torch.bfloat16)])
        y = torch.cat([y, -y, y[:3]])
        for part in y.split(15):
            groups.append(torch.cat([torch.tensor([6 * s], dtype=torch.bfloat16), part]))
    x = torch.stack(groups)
    want_s = np.repeat(np.arange(1, 127, dtype=np.uint8), len(groups) // 126)
    n = -(-len(groups) // 8)
    rows = torch.zeros((n * 8, 16), dtype=torch.bfloat16)
    rows[:len(groups)] = x
    rows = rows.reshape(n, 1, 128)
    mem = [torch.zeros((-(-n // 16), 16, 1, w), dtype=torch.uint8, device="cuda") for w in (64, 64, 8, 8)]
    b.kv_pages_write(b.kv_pages(*mem), rows.cuda(), (-rows).cuda(), torch.arange(n, device="cuda"))
    torch.cuda.synchronize()
    y = x.double().numpy() / codecs.e4m3_decode(want_s)[:, None]
    for i, sign in ((0, 1.0), (1, -1.0)):
        got_s = mem[2 + i].cpu().numpy().reshape(-1)[:len(groups)]
        assert np.array_equal(got_s, want_s)
        c = mem[i].cpu().numpy().reshape(-1, 8)[:len(groups)]
        got = np.stack([c & 15, c >> 4], -1).reshape(-1, 16)
        assert np.array_equal(got, codecs.e2m1_encode(sign * y))
