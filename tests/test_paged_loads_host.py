"""What the loading warps of the chunk and prompt kernel have started is counted before they can leave their loop (no GPU
needed: the order stands in the source; only limits below a load's latency would show it on a GPU)."""
import os
import re

from split_kv_sparse_gb300 import build as bld


def loader():
    with open(os.path.join(bld.CSRC, "attn_tile.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = text.index("else if (warp == 9 || warp == 11)")
    return text[start:text.index("else if (kF8 && warp >= 12)", start)]


def test_every_started_tile_is_counted_before_the_next_way_out():
    """The end of the role drains the tiles below `done`. A tile counted later than its copy starts would be missed by
    a wait that runs out in between, and its copy could write shared memory that the next CTA has by then."""
    text = loader()
    assert re.search(r"for \(int k = max\(0, done - slots\); k < done; \+\+k\)\s*quiet = wait_drain\(bar\(full \+ k % slots\)",
                     text), "the drain at the end"
    assert text.count("++done") == 1
    first = text.index("mbar_arrive_expect_tx(there")
    last = max(text.index("tma_load_4d(", first), text.index("tma_load_5d(", first))
    assert first < last < text.index("++done"), "counted after the copies were started"
    between = text[first:text.index("++done")]
    for way_out in ("break", "continue", "return", "wait_for", "goto"):
        assert way_out not in between, way_out
