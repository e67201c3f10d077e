"""How the backward with sinks shares its units out (csrc/sink_units.cuh, plain C++,
compiled here): every unit is taken once."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "flashattention_attention_backward_gb300", "csrc")
SOURCE = """
#include "sink_units.cuh"
extern "C" int unit(int r, int cta, int grid, int passes, int heavy, int ahead) {
  return attn::sinks_unit(r, cta, grid, passes, heavy, ahead);
}
extern "C" int snake(int r, int cta, int grid) { return attn::snake_unit(r, cta, grid); }
"""


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    src, lib = str(d / "units.cpp"), str(d / "units.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared",
                        "-fPIC", "-I", CSRC, src, "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(lib)


def _taken(f, grid, n_units):
    """Units in the order that each CTA takes them, as the kernel's roles do: up to the
    first pass that has none."""
    out = []
    for cta in range(grid):
        r, mine = 0, []
        while f(r, cta) < n_units:
            mine.append(f(r, cta))
            r += 1
        out.append(mine)
    return out


@pytest.mark.parametrize("grid", [1, 2, 3, 7, 16])
def test_every_unit_once(units, grid):
    for n_units in list(range(1, 4 * grid + 3)) + [11 * grid + 5]:
        taken = _taken(lambda r, c: units.snake(r, c, grid), grid, n_units)
        assert sorted(sum(taken, [])) == list(range(n_units))
        for with_sinks in range(0, n_units + 1):
            passes, heavy = divmod(with_sinks, grid)
            for ahead in ([0, 1, 2, 5, 40] if heavy else [0]):
                taken = _taken(lambda r, c: units.unit(r, c, grid, passes, heavy, ahead), grid,
                               n_units)
                at = (n_units, with_sinks, ahead)
                assert sorted(sum(taken, [])) == list(range(n_units)), at
                # those with sinks come first, one more for the first `heavy` CTAs
                for cta, mine in enumerate(taken):
                    count = sum(u < with_sinks for u in mine)
                    assert all(u < with_sinks for u in mine[:count]), at
                    assert count == passes + (cta < heavy), at
