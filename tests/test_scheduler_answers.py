"""The order of reads and refills of the tile scheduler's answers (cluster launch control), checked in the sources.

An answer's slot is refilled through the async proxy once every reader has arrived on its barrier.  Nothing orders a
shared-memory load before a later arrival by itself, so each reader's arrival address has to depend on the value it
read, the scheduler needs a proxy fence between the arrivals and the refill, and it may not leave before the last
answers have been read in the other CTA too.  A reader that breaks this order works, rarely, on a tile that is not its
own, which no run shows reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_block_scaled_gb300", "csrc")
KERNELS = ["gemm_kernel.cuh", "train_kernel.cuh"]


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_every_kernel_with_a_tile_scheduler_is_listed():
    users = [n for n in sorted(os.listdir(CSRC)) if n != "ptx.cuh" and "clc_try_cancel" in code(n)]
    assert users == KERNELS


@pytest.mark.parametrize("name", KERNELS)
def test_arrivals_follow_the_reads(name):
    src = code(name)
    reads = [m.start() for m in re.finditer(r"ptx::clc_read\(", src)]
    assert len(reads) >= 2
    # after each read, the next use of the slot's barrier is through the value read
    for at in reads:
        use = re.search(r"[\w:]*\(?clc_empty\(\w+\)[^;]*;", src[at:]).group(0)
        assert "clc_read_done(clc_empty(" in use, use
    # no arrival on the bare barrier
    assert not re.search(r"arrive\w*\((ptx::map_to_rank\()?clc_empty\(", src)


@pytest.mark.parametrize("name", KERNELS)
def test_the_refill_follows_a_proxy_fence(name):
    src = code(name)
    refill = src.index("ptx::clc_try_cancel")
    wait = src.rindex("clc_empty(slot)", 0, refill)
    assert "fence_proxy_async_smem()" in src[wait:refill]


@pytest.mark.parametrize("name", KERNELS)
def test_the_scheduler_leaves_after_the_last_reads(name):
    src = code(name)
    last = src[src.index("if (!got)", src.index("ptx::clc_try_cancel")):]
    both = re.match(r"if \(!got\) \{\s*for \(int i = 0; i < 2; \+\+i\) \{\s*if \(!wait_bar<[^>]*>\(clc_empty\(slot\)", last)
    one = re.match(r"if \(!got\) \{\s*wait_bar<[^>]*>\(clc_empty\(slot\), ph \^ 1u, ctl\);\s*break;", last)
    assert both or one
    if one:   # of the answer before the last; then nobody may arrive for the last
        arrivals = [m.start() for m in re.finditer(r"clc_read_done\(clc_empty\(", src)]
        assert len(arrivals) >= 3
        for at in arrivals:
            assert re.search(r"if \(got( && lane == 0)?\)", src[at - 120:at + 120])
