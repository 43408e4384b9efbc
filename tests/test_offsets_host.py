"""The check of packed sequences' offsets at the ends of the 32-bit range (no GPU needed): the
function that every kernel asks, compiled for the host.  A check that forms a length first is shown to
accept offsets that it must not: the difference of two 32-bit offsets does not always fit 32 bits."""
import itertools
import subprocess

import pytest

from state_space_model_05_b200 import build as builder

LOW, HIGH = -(1 << 31), (1 << 31) - 1
TOTAL = 100
VALUES = [LOW, LOW + 1, LOW + 50, LOW + 99, LOW + 100, LOW + 101, -(1 << 30), -101, -100, -1, 0, 1, 50, 99, 100, 101, 1 << 30,
          HIGH - 100, HIGH - 99, HIGH - 1, HIGH]

SOURCE = """
#include <cstdio>
#include "common.cuh"
int main()
{
    int a, b, total;
    while (std::scanf("%d %d %d", &a, &b, &total) == 3) std::printf("%d\\n", (int)ssd::valid_offsets(a, b, total));
}
"""


def wrap(x):
    return (x - LOW) % (1 << 32) + LOW


def length_first(a, b, total):
    """The check with the length formed first, in arithmetic that wraps."""
    n = wrap(b - a)
    return not (a < 0 or n < 0 or wrap(a + n) > total)


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    d = tmp_path_factory.mktemp("offsets")
    (d / "check.cu").write_text(SOURCE)
    subprocess.check_call([builder.nvcc(), *builder.ARCH, "-std=c++17", "-I", builder.INCLUDE, "-I", builder.CSRC,
                           "-o", str(d / "check"), str(d / "check.cu")])

    def run(cases):
        text = "".join(f"{a} {b} {t}\n" for a, b, t in cases)
        out = subprocess.run([str(d / "check")], input=text, capture_output=True, text=True, check=True).stdout
        return [line == "1" for line in out.split()]
    return run


def test_offsets_are_valid_only_in_order_and_in_range(check):
    cases = [(a, b, t) for a, b in itertools.product(VALUES, VALUES) for t in (0, TOTAL, HIGH - 1023)]
    assert check(cases) == [0 <= a <= b <= t for a, b, t in cases]


def test_a_length_formed_first_would_not_do(check):
    """Offsets whose wrapped length passes: the walk over its blocks would leave the buffers."""
    cases = [(a, b, TOTAL) for a, b in itertools.product(VALUES, VALUES)
             if length_first(a, b, TOTAL) and not 0 <= a <= b <= TOTAL]
    assert (100, LOW + 50, TOTAL) in cases and all(a > TOTAL or wrap(b - a) > TOTAL for a, b, _ in cases)
    assert not any(check(cases))


def test_a_table_of_wrapped_lengths_would_not_do(check):
    """Offsets of three sequences whose wrapped lengths are all positive and whose wrapped block counts
    sum to what the table has room for: the last sequence's blocks would lie far before the table."""
    cu, block = [0, 1000, LOW + 999, TOTAL], 128
    lens = [wrap(b - a) for a, b in zip(cu, cu[1:])]
    blocks = [int(wrap(n + block - 1) / block) for n in lens]
    assert min(lens) >= 0 and sum(blocks) <= TOTAL // block + len(lens) and sum(blocks[:2]) < -(1 << 23)
    assert check([(a, b, TOTAL) for a, b in zip(cu, cu[1:])]) == [False, False, False]
