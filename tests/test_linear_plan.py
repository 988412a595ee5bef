"""Which tile takes a product of the linear layer, on the CPU: the plan is compiled alone with g++. Every tile that
is built is one that some size reaches, and the sizes of linear_shapes reach all of them."""

import os
import shutil
import subprocess

import pytest

from linear_shapes import CANDIDATES, STAND_IN, TILES, TOO_MANY_TILES, product

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = tmp_path_factory.mktemp("plan") / "plan_driver"
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                            os.path.join(ROOT, "zero_partition_plan_amd", "csrc"),
                            os.path.join(ROOT, "tests", "plan", "plan_driver.cpp"), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    return str(exe)


def ask(driver, questions):
    """(shape, splits, k of a split, fits, shape that runs) of each (rows, columns, k, direct)."""
    text = "".join("%d %d %d %d\n" % q for q in questions)
    run = subprocess.run([driver], input=text, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0
    return [tuple(int(v) for v in line.split()) for line in run.stdout.splitlines()]


def test_built_tiles_are_the_planned_ones(driver):
    rows = [[int(v) for v in line.split()] for line in
            subprocess.run([driver, "shapes"], capture_output=True, text=True, timeout=60).stdout.splitlines()]
    assert [r[0] for r in rows] == [*CANDIDATES, STAND_IN]
    for r in rows:
        assert r[1:5] == r[5:9], r                     # held, rows, columns, groups
        assert r[9] == (r[0] == STAND_IN)


def test_every_tile_is_reached_and_by_the_listed_sizes(driver):
    keys = list(TILES)
    for more in (0, 1):                                # n odd, and even beside it
        got = ask(driver, [(*product(o, m, k, n + more), 1) for (o, _, _), (m, k, n) in TILES.items()])
        for key, (shape, splits, k_split, fits, runs) in zip(keys, got):
            assert (shape, splits > 1) == key[1:] and fits and runs == shape, (key, shape, splits)
            assert k_split % 64 == 0
    for order in ("fwd", "dx", "dw"):
        assert {s for o, s, _ in keys if o == order} == set(CANDIDATES)


def test_held_operands_take_tiles_that_hold_them(driver):
    sizes = [product(o, m, k, n + 1) for (o, _, _), (m, k, n) in TILES.items()]
    for (o, shape, _), with_, without in zip(TILES, ask(driver, [(*s, 1) for s in sizes]), ask(driver, [(*s, 0) for s in sizes])):
        assert without[:3] == with_[:3]                # the workspace does not depend on it
        assert without[4] == (STAND_IN if shape in (0, 5, 6) else shape)


def test_too_many_small_tiles_take_the_stand_in(driver):
    m, k, n = TOO_MANY_TILES
    shape, splits, _, fits, runs = ask(driver, [(m, n, k, 1)])[0]
    assert shape != STAND_IN and splits == 1 and fits and runs == STAND_IN
    assert ask(driver, [(1 << 27, 1 << 27, 8, 1)])[0][3] == 0


def test_splits_cover_k(driver):
    """Every step of k belongs to one split, none of them empty, whatever the size."""
    import random
    rng = random.Random(5)
    sizes = [tuple(int(2 ** rng.uniform(0, 17)) for _ in range(2)) + (int(2 ** rng.uniform(0, 20)),) for _ in range(5000)]
    sizes += [(7, 9, 0), (1, 1, 1), (1 << 27, 1, 1), (1, 1, 1 << 27)]
    for (m, n, k), (shape, splits, k_split, _, _) in zip(sizes, ask(driver, [(*s, 1) for s in sizes])):
        assert splits * k_split >= k > (splits - 1) * k_split or (k == 0 and splits == 1), (m, n, k, splits, k_split)
