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
]


@pytest.mark.parametrize("mode", [0, 1, 2], ids=["forward", "dq", "dkv"])
def test_listed_walks_stay_inside(walk, mode):
    for problem, line in walk([(s, k, d, mode) for s, k in SHAPES for d in (0, 1)]):
        assert line.startswith("ok "), (problem, line)


def test_random_walks_stay_inside(walk):
    rng = random.Random(3)
    problems = []
    while len(problems) < 600:
        dims = [min(n, int(2 ** rng.uniform(0, b))) for n, b in ((40, 5.4), (120, 7), (300, 8.3))]
        kernel = tuple(2 * rng.randrange((min(n, m) + 1) // 2) + 1 for n, m in zip(dims, (21, 61, 151)))
        shape = (rng.choice((1, 2, 3)), *dims, rng.randint(1, 4), rng.choice((16, 32, 64, 128)))
        if dims[0] * dims[1] * dims[2] <= 100000:
            problems.append((shape, kernel, rng.randrange(2), rng.randrange(3)))
    for problem, line in walk(problems):
        assert line.startswith("ok "), (problem, line)
