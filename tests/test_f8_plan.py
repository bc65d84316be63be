"""The sizes of the 8-bit product tests reach every kernel instance, each also with more tiles
than run at once and several K steps a tile: the rules themselves, compiled for the host,
say which instance a size takes."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_f8 as gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """rows of (M, N, K, E, experts, sms) -> rows of (columns, cluster, bn, ctas, runs, tiles)."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is missing")
    exe = str(tmp_path_factory.mktemp("plan") / "f8_plan")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                        "-I", os.path.join(ROOT, "hadamard_rotated_bit_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "c", "f8_plan.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(rows):
        text = "\n".join(" ".join(str(int(v)) for v in row) for row in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def _sizes(test, names):
    """What the test is parametrised with."""
    return next(list(m.args[1]) for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names)


DENSE = _sizes(gpu.test_product_exact, "M,N,K") + _sizes(gpu.test_product_exact_many_tiles, "M,N,K")
ALONG_K = _sizes(gpu.test_product_shared_out_along_k, "M,N,K")
EXPERTS = _sizes(gpu.test_experts_exact, "counts,N,K") + _sizes(gpu.test_experts_exact_many_tiles, "counts,N,K")
LANES = {("lanes", bn, ctas) for bn in (64, 128, 256) for ctas in (1, 2)}


@pytest.mark.parametrize("sms", [148, 152])
def test_every_instance_is_tested(plan, sms):
    sizes = [(M, N, K, 1, False) for M, N, K in DENSE]
    runs = [(M, N, K, 1, False) for M, N, K in ALONG_K]
    experts = [(sum(c), N, K, len(c), True) for c, N, K in EXPERTS]
    taken, wraps = set(), set()
    for size, (columns, cluster, bn, ctas, _, tiles) in zip(sizes + experts, plan([s + (sms,) for s in sizes + experts])):
        name = ("rows", columns, cluster > 1) if columns else ("lanes", bn, ctas)
        taken.add(name)
        # (of the tiles of experts, an upper bound, only those of groups with rows count)
        if size[4]:
            counts, N, K = EXPERTS[experts.index(size)]
            tiles = sum(c > 0 for c in counts) * -(-N // (128 if columns else bn))
        if tiles > (sms if columns else sms // ctas) and size[2] > 128 and cluster == 1:
            wraps.add(name)
    rows = {("rows", c, shared) for c in (16, 32) for shared in (False, True)}
    assert taken == LANES | rows
    assert wraps == LANES | {("rows", 16, False), ("rows", 32, False)}
    assert all(p[4] > 0 for p in plan([s + (sms,) for s in runs]))
