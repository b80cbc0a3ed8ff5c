"""Index arithmetic of the ragged batches at their largest sizes, compiled for
the host (no GPU needed: the buffers of such a call would fill one)."""
import shutil
import subprocess

import pytest

from quantized_linear_attention_sq_b200.build import CSRC

MAIN = r'''
#include <cstdio>
#include <initializer_list>
#include "sq_spans.cuh"
int main() {
  for (int32_t n : {0, 1, 63, (1 << 27) - 1, 1 << 27, 1 << 30}) std::printf("pieces %d %lld\n", n, (long long)sqr::row_pieces(n));
  for (int32_t b : {0, 1, 16384, 2147483647}) std::printf("blocks %d %lld\n", b, (long long)sqr::most_blocks(1 << 30, b));
  for (int32_t c0 : {-2147483647 - 1, -1, 0, 7, 8, 2147483640, 2147483647}) {
    std::printf("within %d %d\n", c0, (int)sqr::blocks_within(c0, 3, 10));
    std::printf("after %d %d\n", c0, sqr::block_after(9, c0));
  }
}
'''


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("spans")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-I", CSRC,
                    str(at / "main.cpp"), "-o", str(at / "main")], check=True)
    out = subprocess.run([str(at / "main")], check=True, capture_output=True, text=True).stdout
    return [line.split() for line in out.splitlines()]


def test_pieces_of_the_longest_request(lines):
    """A bad slot's o is zeroed whole, whatever its length (2^27 rows are 2^31 pieces)."""
    got = {int(n): int(p) for kind, n, p in (x for x in lines if x[0] == "pieces")}
    assert got == {n: 16 * n for n in (0, 1, 63, 2 ** 27 - 1, 2 ** 27, 2 ** 30)}


def test_blocks_of_the_largest_batch(lines):
    got = {int(b): int(n) for kind, b, n in (x for x in lines if x[0] == "blocks")}
    assert got == {b: 2 ** 24 + b for b in (0, 1, 16384, 2 ** 31 - 1)}


def test_first_blocks_that_no_table_should_hold(lines):
    """A first block near 2^31 must not pass as one inside the workspace."""
    within = {int(c): bool(int(x)) for kind, c, x in (y for y in lines if y[0] == "within")}
    after = {int(c): int(x) for kind, c, x in (y for y in lines if y[0] == "after")}
    assert within == {c: 0 <= c <= 7 for c in within} and len(within) == 7
    assert after == {c: 9 - c if 0 <= c <= 9 else -1 for c in after} and len(after) == 7
