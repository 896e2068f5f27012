"""The score-shaped attention's planner and walk, replayed on the CPU: what a
launch would read lies inside its tensors and what it stages inside its
buffers. A stray read whose value is unused shows in no result."""
import os
import random
import subprocess

import pytest

from neighborhood_attention_video_gb300 import build as na_build

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "scored_plan", "walk.cpp")
EXE = os.path.join(HERE, "scored_plan", "_build", "walk")


@pytest.fixture(scope="module")
def walk():
    os.makedirs(os.path.dirname(EXE), exist_ok=True)
    res = subprocess.run([na_build.nvcc(), "-O2", "-std=c++17", "-I", na_build.CSRC, "-I", na_build.INCLUDE, SRC, "-o", EXE],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr

    def run(problems):
        lines = [" ".join(map(str, (*shape, *kernel, docs, mode))) for shape, kernel, docs, mode in problems]
        out = subprocess.run([EXE], input="\n".join(lines), capture_output=True, text=True, timeout=600)
        assert out.returncode == 0, out.stderr
        return list(zip(problems, out.stdout.splitlines(), strict=True))

    return run


# a brick whose frames run past the last one, in chunks of more than 96 columns
SHAPES = [
    ((1, 8, 64, 33, 8, 64), (3, 7, 33)),
    ((1, 16, 32, 48, 8, 64), (3, 7, 7)),
    ((2, 6, 13, 21, 4, 32), (3, 5, 7)),
    ((1, 20, 80, 110, 4, 64), (7, 13, 35)),
    ((1, 16, 64, 64, 8, 64), (3, 7, 7)),
    ((1, 8, 48, 64, 16, 128), (3, 7, 7)),
    ((1, 13, 20, 21, 8, 64), (11, 11, 11)),
    ((1, 2, 40, 40, 1, 128), (1, 31, 33)),
    ((1, 1, 2, 700, 1, 32), (1, 1, 501)),
    ((3, 1, 1, 1, 1, 16), (1, 1, 1)),
    ((2, 7, 19, 23, 2, 64), (1, 1, 1)),
    ((1, 9, 20, 40, 2, 32), (3, 1, 1)),
]


@pytest.mark.parametrize("mode", [0, 1, 2], ids=["forward", "dq", "dkv"])
def test_listed_walks_stay_inside(walk, mode):
    for problem, line in walk([(s, k, d, mode) for s, k in SHAPES for d in range(4)]):
        assert line.startswith("ok "), (problem, line)


def test_random_walks_stay_inside(walk):
    rng = random.Random(3)
    problems = []
    while len(problems) < 600:
        dims = [min(n, int(2 ** rng.uniform(0, b))) for n, b in ((40, 5.4), (120, 7), (300, 8.3))]
        kernel = tuple(2 * rng.randrange((min(n, m) + 1) // 2) + 1 for n, m in zip(dims, (21, 61, 151)))
        shape = (rng.choice((1, 2, 3)), *dims, rng.randint(1, 4), rng.choice((16, 32, 64, 128)))
        if dims[0] * dims[1] * dims[2] <= 100000:
            problems.append((shape, kernel, rng.randrange(4), rng.randrange(3)))
    for problem, line in walk(problems):
        assert line.startswith("ok "), (problem, line)


def test_large_windows_are_planned_or_refused(walk):
    """Windows of a frame up to the whole grid of 2^31 positions: a plan whose shared
    memory fits, or none. Up to 2^14 keys there always is one."""
    rng = random.Random(2)
    problems = [((1, 1, n, m, 1, hd), (1, a, b), d, mode)
                for n, m, a, b in ((600, 600, 511, 511), (300, 300, 299, 299), (400, 400, 255, 255),
                                   (40001, 40001, 30001, 30001), (4, 2000000, 1, 1999999), (65537, 65537, 65535, 65535),
                                   (1, 2 ** 31 - 1, 1, 2 ** 31 - 1), (2 ** 31 - 1, 1, 2 ** 31 - 1, 1))
                for hd in (16, 128) for d in (0, 1) for mode in (0, 1, 2)]
    problems += [((1, 2 ** 31 - 1, 1, 1, 1, 16), (2 ** 31 - 1, 1, 1), 0, mode) for mode in (0, 1, 2)]
    problems += [((2 ** 30, 1, 1, 1, 4, 16), (1, 1, 1), 0, mode) for mode in (0, 1, 2)]
    small = len(problems)
    while len(problems) < 300:
        area = 2 ** rng.uniform(10, 17.5)
        kh = min(int(2 ** rng.uniform(0, 17.5)), int(area)) | 1
        kw = max(1, int(area / kh)) | 1
        grid = (kh + rng.choice((0, 1, 7, kh)), kw + rng.choice((0, 1, 7, kw)))
        if grid[0] * grid[1] <= 60000:
            problems.append(((1, 1, *grid, 1, rng.choice((16, 32, 64, 128))), (1, kh, kw), rng.randrange(2), rng.randrange(3)))
    lines = walk(problems)
    for i, ((shape, kernel, docs, mode), line) in enumerate(lines):
        assert line == "unplanned" or line.startswith("ok "), ((shape, kernel, docs, mode), line)
        if i >= small and kernel[1] * kernel[2] <= 2 ** 14:
            assert line.startswith("ok "), ((shape, kernel, docs, mode), line)
    assert {x.split()[0] for _, x in lines} == {"ok", "unplanned"}
