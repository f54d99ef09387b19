"""The plans that cut a symmetric product's tiles into ranges of K, on the CPU: the
kernel's copies run two slabs ahead of its products and know three work items, the
current one and two more, when the address of the next copy is found."""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "dense_gemm_sgemm_amd", "csrc", "tune", "sym_plan.hpp")
SOURCE = """
#include "%s"
extern "C" void plan(int M, int slabs, int batch, int cus, long long* out) {
  const mi355gemm::tune::SymPlan p = mi355gemm::tune::plan_sym(M, slabs, batch, cus);
  const long long v[6] = {p.shape, p.bm, p.whole, p.rest, p.splits, p.per};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    where = tmp_path_factory.mktemp("plan")
    src, lib = str(where / "plan.cpp"), str(where / "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE % HEADER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).plan

    def call(M, slabs, batch, cus=256):
        out = (ctypes.c_longlong * 6)()
        fn(M, slabs, batch, cus, out)
        return dict(zip(("shape", "bm", "whole", "rest", "splits", "per"), out))

    return call


def sizes():
    rng = random.Random(5)
    out = [(4096, 64, 1), (2048, 128, 4), (832, 39, 2), (1024, 64, 6), (128, 2, 1), (1 << 16, 1 << 10, 1)]
    for _ in range(4000):
        M = 64 * rng.randrange(2, 1 + int(2 ** rng.uniform(1, 7)))
        out.append((M, rng.choice([1, 1, 3]) * rng.randrange(M // 64, M // 64 + int(2 ** rng.uniform(0, 9))),
                    int(2 ** rng.uniform(0, 5))))
    return out


def lengths(p, slabs):
    """Slabs of the kinds of work items."""
    out = [slabs] if p["whole"] else []
    if p["rest"]:
        out += [p["per"]] * (p["splits"] > 1) + [slabs - (p["splits"] - 1) * p["per"]]
    return out


def test_work_items_are_whole(plan):
    """Every slab is in one range, tiles are all there, and ranges start a round."""
    for M, slabs, batch in sizes():
        p = plan(M, slabs, batch)
        t = -(-M // p["bm"])
        assert p["shape"] >= 0 and M >= p["bm"] and p["whole"] + p["rest"] == t * (t + 1) // 2 * batch
        assert all(n > 0 for n in lengths(p, slabs)), (M, slabs, batch, p)
        assert p["rest"] == 0 or p["whole"] % 8 == 0


def test_two_work_items_are_three_slabs(plan):
    """Whatever order a workgroup takes its items in, on any number of CUs: the slab
    after next is in one of the two items behind the current one.  So the slab that
    the copies come to at an item's end, three on, is as well."""
    for M, slabs, batch in sizes():
        p = plan(M, slabs, batch)
        assert 2 * min(lengths(p, slabs)) >= 3, (M, slabs, batch, p)
