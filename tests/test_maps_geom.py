"""Host replay of the map operators' geometry (CPU); see map_geom_check.cpp for what is checked."""
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

SHAPES = [(32, 96, 56, 56), (32, 192, 28, 28), (64, 96, 56, 56), (128, 768, 7, 7), (64, 384, 14, 14), (13, 101, 23, 19),
          (1, 1, 1, 1), (1, 3, 1, 1), (8, 300, 32, 32), (1, 8, 16400, 16400), (5, 1, 1 << 15, 1 << 15), (1, 33000, 1, 2),
          (4, 1 << 20, 1, 1), (1, 1 << 24, 1, 1), (131072, 1024, 1, 1), (1, 9000, 1, 8), (2, 2, 4096, 4096)]


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("geom") / "map_geom_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-o", exe, os.path.join(HERE, "map_geom_check.cpp")], check=True)
    return exe


def run(checker, shape):
    r = subprocess.run([checker, *map(str, shape)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "OK", (shape, r.stdout + r.stderr)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(checker, shape):
    run(checker, shape)


def test_sweep_shapes(checker):
    for C in (64, 128, 256, 512):
        for H in (32, 64, 128, 256):
            run(checker, (max(1, round(2 ** 28 / (4 * C * H * H))), C, H, H))


def test_every_width(checker):
    for C in [*range(1, 140), *range(140, 1100, 13), *range(1100, 20000, 977)]:
        for H, W in ((1, 1), (7, 7), (14, 14), (5, 30), (32, 32)):
            run(checker, (40, C, H, W))


def test_random_shapes(checker):
    rng = random.Random(5)
    for _ in range(300):
        C = int(round(2 ** rng.uniform(0, 14)))
        H, W = (int(round(2 ** rng.uniform(0, 8))) for _ in range(2))
        run(checker, (int(round(2 ** rng.uniform(0, 12))), C, H, W))
