"""What the layer operators' kernels have to keep to and no run can show: the
memory order of what they share, read from their sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_route_layout_gb300", "csrc")


def code(name):
    """The lines of a source file, without comments."""
    with open(os.path.join(CSRC, name)) as f:
        return [line.split("//")[0] for line in f]


def test_accumulators_change_hands_at_cluster_scope():
    """Threads read the accumulators that the other CTA's thread filled: no relaxed arrival
    and no wait at the scope of one CTA stands on their barriers."""
    good = ("warp_wait_cluster(", "mbar_wait_soon_cluster(", "mbar_wait_cluster(", "mbar_arrive_at(", "mma_commit(")
    uses = [line.strip() for line in code("ep_linear_mma.cu")
            if re.search(r"bar->acc_(full|empty)", line) and "mbar_init(" not in line]
    assert len(uses) >= 5                      # three arrivals, two waits
    for line in uses:
        assert any(g in line for g in good), line


def test_overlapped_kernels_read_by_plain_loads():
    """A kernel that starts under the end of the one before it is alive while that one writes:
    the read-only path, for data that nobody writes meanwhile, is not for it."""
    for name in sorted(os.listdir(CSRC)):
        lines = code(name)
        if not any("begin_overlapped()" in line for line in lines) and name != "ep_linear.cuh":
            continue
        for line in lines:
            assert not re.search(r"__ldg\(|ld_nc|\.nc\.", line), f"{name}: {line.strip()}"
