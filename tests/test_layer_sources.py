"""What the kernels have to keep to and no run can show: the
memory order of what they share, read from their sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_route_layout_gb300", "csrc")


def code(name):
    """The lines of a source file, without comments."""
    with open(os.path.join(CSRC, name)) as f:
        return [line.split("//")[0] for line in f]


def test_accumulators_change_hands_at_cluster_scope():
    """Threads of both CTAs read and free the accumulators that a thread of one has filled:
    every wait on their barriers is at cluster scope with the tensor core's fence behind
    it, every thread's arrival at cluster scope with the fence ahead of it."""
    lines = [line.strip() for line in code("ep_linear_mma.cu")]
    waits = arrivals = 0
    for i, line in enumerate(lines):
        if not re.search(r"bar->acc_(full|empty)", line) or "mbar_init(" in line:
            continue
        if "wait" in line:
            waits += 1
            assert re.search(r"\b(warp_wait_cluster|mbar_wait_soon_cluster|mbar_wait_cluster)\(", line), line
            assert any("tc_fence_after();" in after for after in lines[i + 1:i + 3]), line
        elif "mma_commit(" not in line:        # the tensor core's own arrival
            arrivals += 1
            assert "mbar_signal_at(in_cta(" in line or "mbar_arrive_at(in_cta(" in line, line
            assert "tc_fence_before();" in lines[i - 2:i], line
    assert (waits, arrivals) == (2, 2)


def test_overlapped_kernels_read_by_plain_loads():
    """A kernel that starts under the end of the one before it is alive while that one writes:
    the read-only path, for data that nobody writes meanwhile, is not for it."""
    for name in sorted(os.listdir(CSRC)):
        lines = code(name)
        if not any("begin_overlapped()" in line for line in lines) and name != "ep_linear.cuh":
            continue
        for line in lines:
            assert not re.search(r"__ldg\(|ld_nc|\.nc\.", line), f"{name}: {line.strip()}"


def test_dispatch_reads_the_routing_layout_by_plain_loads():
    """Dispatch kernels start while the routing layout is still being written."""
    written = "mask|local8|local16|chunk_off|chunk_cnt|rank_base|expert_offset"
    for name in ("ep_dispatch.cu", "ep_dispatch_bulk.cu", "ep_dispatch_common.cuh", "ep_split.cu"):
        text = "".join(code(name))
        assert not re.search(rf"(__ldg|ld_nc_v4)\(\s*p\.({written})\b", text), name
        assert re.search(rf"p\.({written})\[", text), name
