"""What the norms' backward pass has to keep to and no run can show, read from its source:
a wait for a row that gave up ends the CTA's rows, together and with no copy in flight."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_route_layout_gb300", "csrc", "ep_norm.cu")


def kernel():
    with open(SOURCE) as f:
        lines = [line.split("//")[0].strip() for line in f]
    lines = [line for line in lines if line]
    at = next(i for i, line in enumerate(lines) if "norm_grad_kernel(NormParams p) {" in line)
    end = next(i for i, line in enumerate(lines) if i > at and "norm_sums_kernel(" in line)
    return lines[at:end]


def one(lines, pattern):
    found = [i for i, line in enumerate(lines) if re.search(pattern, line)]
    assert len(found) == 1, (pattern, found)
    return found[0]


LOOP = r"^for \(int64_t row = blockIdx\.x; row < p\.rows; row \+= gridDim\.x\) \{"
LEAVE = r"^if \(leaves\) \{"


def test_the_cta_agrees_on_a_wait_that_gave_up():
    """Any thread's give-up is written ahead of the row's first meeting and read right behind it,
    long ahead of the row's last: no thread sees the next row's."""
    lines = kernel()
    loop = one(lines, LOOP)
    wait = one(lines, r"^if \(!mbar_wait\(&landed\[slot\], phase\)\) gave_up = 1;")
    meeting = one(lines, r"cta_sum\(sum, room\[0\], &gave_up, &leaves\)")
    leave, last = one(lines, LEAVE), one(lines, r"^const int64_t ahead = ")
    assert loop < wait < meeting < leave < last and leave == meeting + 1
    assert lines[last - 1] == "__syncthreads();"
    assert not any(re.search(r"__syncthreads|cta_sums?\(", line) for line in lines[wait:meeting])
    with open(SOURCE) as f:
        text = f.read()
    sums = text[text.index("float cta_sum(float v, float* room"):]
    assert re.search(r"__syncthreads\(\);\s+if \(flag\) \*set = \*flag;", sums[:sums.index("}")])


def test_nothing_is_asked_for_behind_it_and_what_was_lands():
    """Rows are asked for ahead of the loop and at a row's end alone; a CTA that gives up waits for
    the ring's places from this row's on, reports, and leaves."""
    lines = kernel()
    fetches = [i for i, line in enumerate(lines) if re.search(r"\bfetch\(", line)]
    loop, leave, last = one(lines, LOOP), one(lines, LEAVE), one(lines, r"^const int64_t ahead = ")
    assert len(fetches) == 2 and fetches[0] < loop and fetches[1] == last + 1
    depth, end = 0, leave
    while True:
        depth += lines[end].count("{") - lines[end].count("}")
        if depth == 0:
            break
        end += 1
    text = "\n".join(lines[leave:end])
    assert end < last and lines[end - 1] == "return;" and "atomicOr(p.err, kErrNormTimeout);" in text
    assert "i < p.ring_rows && row + (int64_t)i * gridDim.x < p.rows" in text and "mbar_wait(&landed[slot], phase)" in text


def test_the_thread_that_makes_the_barriers_fences_them():
    """The fence that shows barriers to bulk copies is for those its own thread has made."""
    lines = kernel()
    at = one(lines, r"mbar_init\(")
    assert re.search(r"^for \(int i = 0; i < kRingRows; \+\+i\) mbar_init\(&landed\[i\], 1\);", lines[at])
    assert lines[at - 1] == "if (threadIdx.x == 0) {" and lines[at + 1] == "mbar_init_fence();"
