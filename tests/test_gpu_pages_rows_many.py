"""GPU tests of the rotating append, of the append into 4 bits and of the read-back with as many rows as fill the SMs, where a warp
takes several chunks of a row one after the other (its next loads on their way), or four heads' loads at once. The inputs, the oracle and
the tolerances are those of the tests of few rows."""
import pytest
import torch

import test_gpu_pages_rows as few
from _four_bit_util import caches, f32, on_gpu
from _paged_util import D, status_clear
from split_kv_sparse_gb300 import binding as b

pytestmark = pytest.mark.gpu
SM_WARPS = 16    # an SM's warps below which a call takes the smallest pieces


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    b.lib()
    status_clear()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def rows_past(chunks):
    """Rows from which on a warp takes more than one of a row's chunks, and some."""
    return 12 * SM_WARPS * sms() // chunks + 40


def chunks_of(h_q, h_kv):
    return (h_q + 3) // 4 + (h_kv + 1) // 2


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("h_q,h_kv,rot,inter", [
    (32, 8, 128, False),    # 12 chunks of four heads
    (28, 8, 96, True),      # 11
    (30, 7, 64, False),     # heads of q, and of k and v, that leave a part of a chunk; v begins inside one
    (0, 5, 128, False),     # no queries
    (20, 4, 128, True),     # 7
])
def test_rotary(dtype, h_q, h_kv, rot, inter):
    few.go(dtype, rows_past(chunks_of(h_q, h_kv)), h_q, h_kv, rot, inter, k_out=True, pad=4, seed=h_q)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("q_type,in_place,inter", [("e4m3", False, False), ("e4m3", False, True), ("bf16", True, False), ("bf16", True, True)])
def test_rotary_into_codes_and_in_place(dtype, q_type, in_place, inter):
    h_q, h_kv = 18, 3       # 5 + 2 chunks, none of the two whole
    few.go(dtype, rows_past(chunks_of(h_q, h_kv)), h_q, h_kv, 64, inter, page=32, layout="head", q_type=q_type, k_out=True, in_place=in_place,
           fused=in_place, pad=5, seed=7)


@pytest.mark.parametrize("dtype", ["bf16", "e2m1"])
def test_rotary_of_many_heads(dtype):
    """Rows of 48 chunks, too few rows for a warp to take a whole one."""
    few.go(dtype, 680, 64, 64, 128, False, seed=9)


@pytest.mark.parametrize("h_kv,page,layout", [(5, 16, "row"), (8, 64, "head"), (1, 128, "row")])
def test_write_four_bits(h_kv, page, layout):
    rows = rows_past(chunks_of(0, h_kv))
    g = torch.Generator().manual_seed(h_kv)
    n_pages = -(-rows // page) + 3
    x = torch.randn((rows, 2 * h_kv + 1, D), generator=g).to(torch.bfloat16)
    mem = [on_gpu(c) for c in caches("e2m1", n_pages, page, h_kv, layout, fill=3)]
    slots = few.slots_of(rows, n_pages * page, g, True)
    dev, dk, dv = x.cuda(), 0.0045, 0.037
    b.kv_pages_write(b.kv_pages(*mem), dev[:, 1:1 + h_kv], dev[:, 1 + h_kv:], slots.cuda(), f32(dk), f32(dv))
    torch.cuda.synchronize()
    for cache, scales, rows_in, d in ((mem[0], mem[2], x[:, 1:1 + h_kv], dk), (mem[1], mem[3], x[:, 1 + h_kv:], dv)):
        codes, s = few.held(rows_in.float().numpy(), d, "e2m1")
        few.same_rows(cache, codes, slots, 3)
        few.same_rows(scales, s, slots, 3)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("h_kv,page,layout", [(8, 16, "row"), (3, 64, "head"), (9, 16, "row")])
def test_read(dtype, h_kv, page, layout):
    """16 heads of K and V a warp: whole, and with a part of it past the last."""
    few.test_read(dtype, 16 * SM_WARPS * sms() // (2 * h_kv) + 30, h_kv, page, layout)
