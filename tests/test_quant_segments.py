"""How the quantiser's kernels cut segments into pieces, at the ends of what a config may
have: the source's own arithmetic, run on the host."""
import os
import re
import subprocess

from combine_route_layout_gb300.build import ARCH, CSRC, NVCC_FLAGS, _nvcc

# each line of input: pieces' rows, then the counts of segments; output: their first pieces, and the end
PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include <cstdlib>
#include "ep_segments.cuh"
int main() {
  char line[4096];
  while (fgets(line, sizeof(line), stdin)) {
    char* at = strtok(line, " \n");
    const int per = atoi(at);
    int64_t before = 0;
    while ((at = strtok(nullptr, " \n"))) {
      printf("%lld ", (long long)before);
      const int count = atoi(at);           // as the table keeps it
      before += ep::pieces_of(count, per);
    }
    printf("%lld\n", (long long)before);
  }
}
"""
MOST_ROWS = 2 ** 31 - 1 - 1024


def test_pieces_of_the_largest_segments(tmp_path):
    source, program = tmp_path / "pieces.cu", tmp_path / "pieces"
    source.write_text(PROGRAM)
    r = subprocess.run([_nvcc(), *ARCH, *NVCC_FLAGS, "-I", CSRC, "-o", str(program), str(source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    cases = [(per, counts) for per in (1, 7, 256, 2047, 2048) for counts in
             ([MOST_ROWS], [MOST_ROWS, 5], [0, MOST_ROWS, 0, 1], [MOST_ROWS - 100, 100], [1, 2, 3], [2 ** 31 - 1 - 1023 - 1024, 1023])]
    text = "".join(" ".join(map(str, [per, *counts])) + "\n" for per, counts in cases)
    out = subprocess.run([str(program)], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    for (per, counts), line in zip(cases, out, strict=True):
        want = [0]
        for c in counts:
            want.append(want[-1] + -(-c // per))
        assert [int(v) for v in line.split()] == want, (per, counts)


def test_the_table_is_made_by_that_arithmetic():
    with open(os.path.join(CSRC, "ep_segments.cuh")) as f:
        text = "".join(line.split("//")[0] + "\n" for line in f)
    assert text.count("pieces_of(") == 3                    # the function, the sum over all, each segment's first
    assert len(re.findall(r"\+ per - 1", text)) == 1
    # a loop over pieces steps by the grid, which never has this many CTAs
    assert re.search(r"kMostPieces = INT32_MAX - \(1 << 20\)", text) and "total > kMostPieces" in text
