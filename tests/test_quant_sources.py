"""What the products of block-quantised operands have to keep to and no run can show: who
meets at the hardware barriers, and the fences there, read from their source."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_route_layout_gb300", "csrc",
                      "ep_qlinear_mma.cu")


def code():
    with open(SOURCE) as f:
        return [line.split("//")[0].strip() for line in f]


def roles():
    """The lines of the MMA warp, the warp that looks for sums, and the epilogue."""
    lines = code()
    at = [next(i for i, line in enumerate(lines) if mark in line)
          for mark in ("} else if (warp == 1) {", "} else if (warp == 2) {", "} else if (warp == 3 &&",
                       "registers_more<")]
    end = next(i for i, line in enumerate(lines) if "tmem_free_own(" in line)
    return lines[at[0]:at[1]], lines[at[1]:at[2]], lines[at[3]:end]


def test_each_barrier_has_a_warp_that_tells_and_warps_that_wait():
    """Accumulators are full (3, 4): one warp tells eight; free (1, 2): eight tell one. The
    two differ in who waits, so that each has 32 threads of one side and 256 of the other."""
    mma, sums, epilogue = roles()
    text = ["\n".join(part) for part in (mma, sums, epilogue)]
    assert [re.findall(r"named_(arrive|sync)\((\d) \+", t) for t in text] == [
        [("sync", "1"), ("sync", "1")], [("arrive", "3")], [("sync", "3"), ("arrive", "1")]]
    assert "kHandover = 32 * (1 + kEpilogueWarps)" in "\n".join(code())


def test_accumulators_change_hands_between_fences():
    """The tensor core's fence is behind every wait for an accumulator and ahead of every
    word that it is full or free."""
    for part in roles():
        for i, line in enumerate(part):
            if "named_arrive(" in line:
                assert "tc_fence_before();" in part[i - 3:i], line
            elif "named_sync(3" in line or "named_sync(1 + (n_acc" in line:
                assert "tc_fence_after();" in part[i + 1:i + 4], line


def test_no_role_leaves_the_hardware_barriers():
    """They have no limit: after a bounded wait that gave up a role goes on through its
    tiles, which it then works out itself, instead of leaving its loop."""
    for part in roles():
        text = "\n".join(part)
        assert "if (!ok) w = qtile_at<" in text
        assert not re.search(r"\b(break|goto)\b|\breturn;", text)    # a lambda returns a value
        assert "for (int i = 0; i < mine; ++i) {" in text
