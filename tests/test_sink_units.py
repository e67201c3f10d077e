"""How the backward with sinks shares its units out (csrc/sink_units.cuh, plain C++,
compiled here): every unit is taken once, and clusters are of sizes that can run."""
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
// fit: clusters of 2, 4 and 8 that run at once; *asked counts the questions
extern "C" int cluster(long long with_sinks, long long others, long long most, long long band,
                       long long least, int sms, const int* fit, int* asked, int waves) {
  const attn::SinkUnits units{with_sinks, others, most, band, least};
  auto at_once = [&](int n) {
    ++*asked;
    return fit[n == 2 ? 0 : n == 4 ? 1 : 2];
  };
  return waves ? attn::sinks_cluster_waves(units, sms, at_once)
               : attn::sinks_cluster(units, sms, at_once);
}
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
    u = ctypes.CDLL(lib)
    u.cluster.argtypes = [ctypes.c_longlong] * 5 + [ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                                    ctypes.POINTER(ctypes.c_int), ctypes.c_int]
    return u


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


def _cluster(units, u, sms=152, fit=(76, 36, 15), waves=0):
    asked = ctypes.c_int(0)
    n = units.cluster(*u, sms, (ctypes.c_int * 3)(*fit), ctypes.byref(asked), waves)
    return n, asked.value


FEW = (1, 127, 128, 9, 128)  # units with sinks, others, tiles of one of each, the fewest


@pytest.mark.parametrize("waves", [0, 1])
def test_clusters_that_can_run(units, waves):
    def cluster(u, **kw):
        return _cluster(units, u, waves=waves, **kw)

    # 2 x 32 heads over 8, 4096 keys, window 1024: an SM has 131 tiles, nobody is asked
    assert cluster((16, 496, 128, 36, 128)) == (1, 0)
    assert cluster((320, 320, 10, 10, 10)) == (1, 0)
    assert cluster(FEW)[0] == 8
    # a size that cannot run is not chosen: a smaller one, or none
    assert cluster(FEW, fit=(76, 36, 0))[0] == 4
    assert cluster(FEW, fit=(76, 0, 0))[0] == 2
    assert cluster(FEW, fit=(0, 36, 15))[0] == 1
    # none larger than the fewest tiles of a unit
    assert cluster((1, 5, 40, 2, 3))[0] == 2
    assert cluster((1, 5, 40, 2, 1))[0] == 1
    # nothing but units with sinks
    assert cluster((9, 0, 72, 0, 8))[0] == 8


def test_rounds_of_clusters(units):
    # 16 units: clusters of 8 run 15 at a time, so they would take two rounds
    assert _cluster(units, (16, 624, 1024, 8, 1000))[0] == 4
    assert _cluster(units, (16, 624, 1024, 8, 1000), fit=(76, 36, 16))[0] == 8
