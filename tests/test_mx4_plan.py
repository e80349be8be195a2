"""The 4-bit product's host logic under AddressSanitizer and UBSan (CPU only).

tests/c/mx4_plan.cpp includes the library's own csrc/mx4_plan.h and is compiled
with g++ and -fsanitize=address,undefined -fno-sanitize-recover=all."""

import os
import shutil
import subprocess

import pytest

from tests.mx4_routes import ROUTES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_step_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "mx4_plan")
    # host-only build with g++ (no device code involved)
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fno-omit-frame-pointer",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "c", "mx4_plan.cpp"), os.path.join(CSRC, "common.cpp"),
                    "-o", out], check=True, timeout=300)
    return out


def run(exe, *args, text=None):
    p = subprocess.run([exe, *args], input=text, capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stderr[-4000:]
    return p.stdout


def test_random_plans_hold_their_bounds(exe):
    """Sizes up to 2^30: parts are whole pairs of steps, none empty, and cover the
    contraction; partial sums fit the workspace; cuts lie on multiples of 256;
    every launch is a possible one."""
    assert run(exe, "plan", "991", "200000").split() == ["200000", "0"]


def test_every_way_is_in_the_gpu_tests(exe):
    got = run(exe, "route", text="".join("%d %d %d %d\n" % r[:4] for r in ROUTES)).splitlines()
    wrong = [(r, g) for r, g in zip(ROUTES, got) if r[4] != g]
    assert not wrong, wrong
    ways = " ".join(r[4] for r in ROUTES)
    for way in ("few 1", "few 2", "few 3", "few 4", "64x4/1", "64x4/4", "64x4/16", "64x2/1", "128/1", "256/1", "columns", "rows"):
        assert way in ways
