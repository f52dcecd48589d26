"""An aborting CTA whose drain runs out reports its own site (no GPU needed: the report stands in the source; a drain that runs
out leaves copies in flight, which no test makes happen). By then another wait has run out and is recorded, so a report that only
takes an empty place would be lost, and tests that look for the drains' sites could not see one."""
import os
import re

import pytest

from split_kv_sparse_gb300 import build as bld

KERNELS = sorted(f for f in os.listdir(bld.CSRC) if f.endswith(".cu"))


def source(name):
    with open(os.path.join(bld.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", KERNELS)
def test_every_drain_that_runs_out_is_reported(name):
    text = source(name)
    report = r"atomicExch\(&a\.status\[1\], W_\w*DRAIN\w*\);"
    drains = len(re.findall(r"\bwait_drain\(", text))
    # (an answer of cluster launch control is waited for with the drains' limit; its role gives up)
    drains -= text.count("ok = __all_sync(0xffffffffu, wait_drain(bar(B_CLC)")
    # several drains may be counted into one flag
    flags = [f for f in re.findall(r"(\w+) = [^;{}]*wait_drain\([^;]*;", text) if f != "ok"]
    for f in set(flags):
        assert re.search(r"if \(!%s\b[^;{}]*\) %s" % (f, report), text), f
    direct = len(re.findall(r"!wait_drain\([^;{}]*\)\s*" + report, text))
    assert direct + len(flags) == drains
    assert "DRAIN" not in "".join(re.findall(r"atomicCAS\(&a\.status\[1\][^;]*;", text))
