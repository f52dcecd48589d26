"""The binding's checks of where tensors lie (no GPU needed: the tensors below only say that they lie on a device)."""
import os

import pytest
import torch

from split_kv_sparse_gb300 import binding as b
from split_kv_sparse_gb300 import build as bld


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(b.LIB_PATH):
        bld.build()
    return b.lib()


class On:
    """What the binding asks of a tensor, for one that lies on CUDA device `dev`."""

    def __init__(self, dev, shape, dtype):
        self.x, self.dev = torch.empty(shape, dtype=dtype), dev
        self.shape, self.dtype, self.nbytes = self.x.shape, dtype, self.x.nbytes

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 1 << 20     # never dereferenced

    def __getattr__(self, name):
        return getattr(self.x, name)


@pytest.fixture
def current(monkeypatch):
    dev = [0]
    monkeypatch.setattr(b, "_device", lambda where: dev[0])
    monkeypatch.setattr(b, "_on", lambda stream, d: None)
    return dev


def test_pages_of_another_device_are_refused(current):
    """A descriptor holds bare addresses: one made on device 0 is of no use to a call on device 1."""
    cache = [On(0, (8, 16, 2, 128), torch.bfloat16) for _ in range(2)]
    pages = b.kv_pages(*cache)
    assert pages.tensors == tuple(cache)
    current[0] = 1
    i32 = lambda *shape: On(1, shape, torch.int32)
    new = On(1, (3, 2, 128), torch.bfloat16)
    with pytest.raises(b.SplitKVError, match="pages lie on CUDA device 0") as e:
        b.kv_pages_write(pages, new, new, On(1, (3,), torch.int64))
    assert e.value.status == b.MLA_ERR_INVALID_ARG
    plan = b.sdpa_paged_plan(1, 8, 2, 128, "bf16", 1, 1, 100, num_sms=152, force_splits=1)
    with pytest.raises(b.SplitKVError, match="pages lie on CUDA device 0") as e:
        b.sdpa_paged(plan, 1, On(1, (1, 8, 128), torch.bfloat16), pages, i32(1, 8), i32(1), i32(2), None, None, None, 0.1,
                     "f32", 1.0, On(1, (1, 8, 128), torch.float32))
    assert e.value.status == b.MLA_ERR_INVALID_ARG
