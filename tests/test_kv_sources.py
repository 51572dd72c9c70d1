"""What the kernels of the cache's attention must do on ways that no run takes on purpose, read from
their source (no GPU needed): after a wait that gave up the join must not trust a record that this
call has not written."""
import os
import re

import pytest

from integer_quantized_nn_gb300 import build as _build

pytestmark = pytest.mark.cpu


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def test_a_block_that_gives_up_leaves_the_join_nothing():
    """The record says that there is nothing, whatever the block does, until all rows' warps have stored
    an item's parts without a wait that gave up; a barrier is between the two writes."""
    s = source("qnn_kv_attn_rows.cu")
    body = s[s.index("kv_attn_rows_kernel("):]
    none = re.search(r"\n    if \(threadIdx\.x == 0\) attn_record\(a, -1, 0, 0, 0, 0\);\n", body)
    assert none
    wait, sums = body.index("grid_dependency_wait();"), body.index("attn_sums<kThreads>(")
    assert wait < none.start() < sums < body.index("if (warp < kCodeWarp0) {")
    assert "__syncthreads();" in source("qnn_kv_attn.cuh").split("attn_sums(", 1)[1].split("\n}\n")[0]
    assert body.count("attn_record(") == 2
    last = body.index("attn_record(", none.end())
    stored, store = body.index("const bool stored = all_ok();"), body.rindex("slot[ROWS")
    assert store < stored < last
    assert "if (stored && " in body[stored:last]


def test_the_other_kernel_has_no_wait_that_gives_up():
    """It always comes to where it writes its record: one for a block without a share, one for every other."""
    s = source("qnn_kv_attn_few.cu")
    assert "mbar" not in s and s.count("attn_record(") == 2


def test_waits_by_counting_end_within_seconds():
    """2^19 probes of 3.94 us each; the self-test of a wait that runs out times that many nanoseconds."""
    s = source("qnn_ptx.cuh")
    probe, shift = re.search(r"kProbeNs = (\d+), kWaitLimitProbes = 1u << (\d+);", s).groups()
    assert 1e9 <= int(probe) * 2 ** int(shift) <= 4e9
    assert "uint32_t limit = kWaitLimitProbes" in s and "mbar_wait_short(b, 0, status, " in source("qnn_api.cu")


def test_all_lanes_of_the_products_warp_go_the_same_way():
    """Its descriptors are the warp's: what leads to a product or a commit is done by all lanes, and only they by one."""
    s = source("qnn_kv_attn_rows.cu")
    role = s[s.index("} else if (warp == 1) {"):]
    role = role[:role.index("const bool is_v = warp == 3;")]
    assert "lane == 0" not in role and "mbar_arrive" not in role
    for call in re.finditer(r"(?:mma_commit|mma_ts|step)\((?!int)", role):
        before = role[:call.start()]
        block = before[before.rindex("elect_one())"):]
        assert "wait(" not in block and block.count("{") - block.count("}") in (0, 1), block[-300:]
