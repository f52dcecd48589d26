"""The descriptor of a bf16 or e4m3 cache may end before the four fields of the 4-bit form, as the header says: they are not read.
A child process lays the descriptor's first 64 bytes at the end of a page of memory whose next page cannot be read, so that
reading on ends the process."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import ctypes, math, mmap
import torch
from split_kv_sparse_gb300 import binding as b
libc = ctypes.CDLL(None, use_errno=True)
libc.mmap.restype = ctypes.c_void_p
libc.mmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long]
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
size = mmap.PAGESIZE
base = libc.mmap(None, 2 * size, 3, 0x22, -1, 0)
assert base not in (None, ctypes.c_void_p(-1).value) and libc.mprotect(base + size, size, 0) == 0
dtype = "%s"
t = torch.bfloat16 if dtype == "bf16" else torch.uint8
k, v = (torch.zeros((4, 16, 2, 128), dtype=t, device="cuda") for _ in range(2))
whole = b.kv_pages(k, v)
short = b.KvPages.k_scales.offset
assert short == 64
ctypes.memmove(base + size - short, ctypes.byref(whole), short)
pages = ctypes.cast(base + size - short, ctypes.POINTER(b.KvPages))
g = torch.Generator().manual_seed(1)
x = torch.randn((20, 12, 128), generator=g).to(torch.bfloat16).cuda()
slots = torch.arange(20, device="cuda")
pos = torch.arange(20, dtype=torch.int32, device="cuda")
cs = torch.cat([torch.ones((20, 64)), torch.zeros((20, 64))], 1).cuda()
q_out = torch.zeros((20, 8, 128), dtype=t, device="cuda")
out = [torch.zeros((20, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
lib, p = b.lib(), (lambda z: z.data_ptr())
q, kn, vn = x[:, :8], x[:, 8:10], x[:, 10:]
ts, hs = kn.stride()[:2]
assert lib.kv_pages_write(pages, 20, p(kn), p(vn), ts, hs, p(slots), None, None, None) == 0
torch.cuda.synchronize()
first = k.clone()
k.zero_()
assert lib.kv_pages_write_rotary(pages, 20, 8, p(q), ts, hs, p(kn), p(vn), ts, hs, p(pos), p(cs), 20, 128, 0, p(slots), None, None, None,
                                 b._SDPA_DTYPES[dtype], p(q_out), 1024, 128, None, 0, 0, None) == 0
assert lib.kv_pages_read(pages, 20, p(slots), None, None, p(out[0]), p(out[1]), 256, 128, None) == 0
torch.cuda.synchronize()
assert torch.equal(k, first) and first.any()
if dtype == "bf16":
    assert torch.equal(out[0], kn) and torch.equal(out[1], vn)
plan = b.sdpa_paged_plan(1, 8, 2, 128, dtype, 1, 1, 20, force_splits=1)
table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
lens, cu = torch.tensor([20], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
o = [torch.zeros((1, 8, 128), device="cuda") for _ in range(2)]
args = [p(table), 2, p(lens), p(cu), None, None, None, 1 / math.sqrt(128), 0, 1.0]
for i, desc in enumerate((pages, ctypes.byref(whole))):
    assert lib.sdpa_paged(ctypes.byref(plan), 1, p(q_out), 1024, 128, desc, *args, p(o[i]), None, None, None, None) == 0
torch.cuda.synchronize()
assert torch.equal(o[0], o[1]) and o[0].any()
print("done")
"""


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_descriptor_without_the_fields_of_scales(dtype):
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA GPU"
    r = subprocess.run([sys.executable, "-c", CHILD % dtype], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "done", (r.returncode, r.stdout[-500:], r.stderr[-2000:])
