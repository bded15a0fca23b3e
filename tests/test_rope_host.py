"""The append's table of turns a position (CPU only), against 60 digits."""
import subprocess
from decimal import Decimal, getcontext

import pytest

from sparse_mixture_experts_router_gb300 import _build

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "rope_turns.h"
int main(int, char** argv) {
  uint64_t turns[128];
  const int pairs = atoi(argv[2]);
  moe::rope_turns(strtof(argv[1], nullptr), pairs, turns);
  for (int i = 0; i < pairs; ++i) printf("%llu\n", (unsigned long long)turns[i]);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("turns")
    (at / "turns.cu").write_text(SOURCE)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O2", "-std=c++17", "-I", _build.CSRC, str(at / "turns.cu"), "-o", str(at / "turns")],
                   check=True, capture_output=True)
    return str(at / "turns")


def exact(base, pairs):
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    return [Decimal(2) ** 64 * Decimal(base) ** (Decimal(-i) / pairs) / two_pi for i in range(pairs)]


def off(got, want):
    return max(abs(Decimal(g) - w) for g, w in zip(got, want))


# bases that fp32 holds exactly
@pytest.mark.parametrize("base", [1.0, 1.0 + 2.0 ** -20, 1.5, 100.0, 10000.0, 500000.0, 1e6, 2.0 ** 40, 2.0 ** 127])
@pytest.mark.parametrize("pairs", [0, 1, 2, 3, 21, 31, 64, 127, 128])
def test_turns_are_rounded_once(program, base, pairs):
    out = subprocess.run([program, repr(base), str(pairs)], check=True, capture_output=True, text=True, timeout=60).stdout
    got = [int(x) for x in out.split()]
    assert len(got) == pairs
    if pairs:
        assert off(got, exact(base, pairs)) <= Decimal("0.5000001")


def test_a_running_product_of_doubles_is_not():
    """What the bound tells apart: 53 bits, and a rounding more with every pair."""
    f, ratio, got = 2.0 ** 64 / 6.283185307179586476925, 10000.0 ** (-2.0 / 256), []
    for _ in range(128):
        got.append(int(f + 0.5))
        f *= ratio
    assert off(got, exact(10000.0, 128)) > 500
