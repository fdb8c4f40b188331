"""The planner of the products grouped by expert (csrc/experts_plan.hpp) in a
host program built with g++: what it plans for any size that the entry points
accept is sound and fits the kernels' 32-bit arguments, and the sizes of
tests/test_gpu_experts_few.py still take the kernels they are there for."""
import os
import random
import shutil
import subprocess

import pytest

from tests import experts_cases as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_orthogonalizing_optimizer_amd", "csrc")
FORWARD, WEIGHT, INPUT = 0, 1, 2
F32, BF16 = 0, 1
INT = (1 << 31) - 1


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("experts") / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c", "experts_plan_check.cpp"), "-o", exe], check=True)

    def f(lines):
        text = "".join(" ".join(map(str, l)) + "\n" for l in lines)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
        assert len(out) == len(lines)
        return [(l.split()[0],) + tuple(map(int, l.split()[1:])) for l in out]
    return f


def sizes(n, seed):
    rng = random.Random(seed)
    spread = lambda hi: min(1 << hi, int(2 ** rng.uniform(0, hi + 0.2)))
    for _ in range(n):
        dtype = rng.choice((F32, BF16))
        direct = int(dtype == BF16 and rng.random() < 0.5)
        unit = 8 if direct else 1
        yield (rng.choice((FORWARD, WEIGHT, INPUT)), spread(30), spread(16), -(-spread(21) // unit) * unit,
               -(-spread(21) // unit) * unit, dtype, direct)


LIMITS = [(p, r, e, o, i, d, 0) for p in range(3) for r in (1, 1 << 24, 1 << 30) for e in (1, 1 << 16)
          for o in (1, 1 << 15, 1 << 21) for i in (1, 1 << 15, 1 << 21) for d in (F32, BF16)]


def test_plans_fit_the_kernels(ask):
    """Over sizes from one to the limits, of the products that are not refused
    for their tiles: grids below 2^32 threads, rows of a unit that a kernel can
    add to an expert's rows in 32 bits, and units and their parts that the
    workspace has room for."""
    asked = list(sizes(20000, 1)) + LIMITS
    seen = {}
    for q, (kernel, tile, splits, tiles, joined, chunk, cap, nbytes, _, _) in zip(asked, ask(asked)):
        which, rows, experts, out, in_, dtype, direct = q
        if max(tiles * splits, joined * (tile * tile // 2048)) > 1 << 22:
            continue  # refused
        seen[which, kernel] = seen.get((which, kernel), 0) + 1
        assert 0 < tiles and 1 <= splits <= 32, q
        if kernel == "few":
            assert which == FORWARD and nbytes == 0 and -(-out // 16) * min(experts, rows) <= 1 << 22, q
            continue
        ocols = out if which == FORWARD else in_
        per = -(-out // tile) * -(-ocols // tile) if which == WEIGHT else -(-ocols // tile)
        if which == WEIGHT:
            # a kernel's count + chunk - 1
            assert 0 < chunk and rows + chunk - 1 <= INT, q
            assert chunk % (64 if dtype == BF16 else 32) == 0, q
            assert tiles == (experts + rows // chunk) * per, q
            # an expert in k > 1 units has more than (k - 1) chunk rows: 2 (rows // chunk) parts at most
            parts = 2 * (rows // chunk) * per
            if kernel == "big":
                # experts in parts have a unit of the head each
                assert rows // chunk <= 512 and experts + rows // chunk <= 2048, q
            else:
                assert joined == rows // chunk * per and splits == 1, q
            assert nbytes >= parts * tile * tile * 4, q
        else:
            assert tiles == (rows // tile + min(experts, rows)) * per, q
            assert joined == (tiles if splits > 1 else 0), q
            assert nbytes >= joined * splits * tile * tile * 4, q
        if kernel == "big":
            assert tile == 256 and direct and experts <= 2048, q
            # a list has an eighth of the tiles, the last 16 in 2 parts or the last 8 in 4
            assert cap >= -(-tiles // 8) + 24, q
        else:
            assert tile == 128, q
    assert len(seen) == 7, seen


def test_few_row_cases_take_their_kernels(ask):
    """Whole 16-byte pieces or not: the cases run both."""
    for direct in (0, 1):
        cases = [c for c in C.FEW if not direct or (c[4] == BF16 and c[3] % 8 == 0)]
        for c, p in zip(cases, ask([(FORWARD, *c[:5], direct) for c in cases])):
            assert p[0] == "few" and p[8:] == c[5], (c, direct, p)


def test_every_few_row_kernel_has_a_case():
    have = {(c[4],) + c[5] for c in C.FEW}
    assert have == {(d, t, w) for d in (F32, BF16) for t in (1, 2, 4) for w in (0, 1)}
    two = [c for c in C.FEW if c[5][0] == 2]
    for dtype, piece in ((F32, 4), (BF16, 8)):
        mine = [c for c in two if c[4] == dtype]
        # the second group of channels whole, cut and outside; rows shorter than a piece
        assert {(0 if c[2] % 32 == 0 else 1 if c[2] % 32 > 16 else 2) for c in mine} == {0, 1, 2}
        assert any(c[3] < piece for c in mine)
        # an expert with several rounds of two tiles, one with 17 to 32 rows, one with up to 16
        for c in mine:
            counts = C.counts(c)
            assert sum(counts) == c[0] and len(counts) == c[1]
        assert any(max(C.counts(c)) > 64 for c in mine)
        assert any(any(17 <= n <= 32 for n in C.counts(c)) and any(0 < n <= 16 for n in C.counts(c)) for c in mine)


def test_large_cases_take_the_large_tiles(ask):
    for c, p in zip(C.LARGE, ask([(*c, BF16, 1) for c in C.LARGE])):
        assert p[0] == "big", (c, p)
