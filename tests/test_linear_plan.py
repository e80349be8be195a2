"""The linear layer's host logic under AddressSanitizer and UBSan (CPU only).

tests/c/linear_plan.cpp includes the library's own csrc/linear_plan.h (checks
of matrices and overlaps, and by which launches a product is computed) and is
compiled with g++ and -fsanitize=address,undefined -fno-sanitize-recover=all,
so that any signed overflow or access out of bounds ends it.
"""

import os
import shutil
import subprocess

import pytest

from tests.linear_routes import KINDS, ROUTES, program_case

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_step_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "linear_plan")
    # host-only build with g++ (no device code involved)
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fno-omit-frame-pointer",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "c", "linear_plan.cpp"), os.path.join(CSRC, "common.cpp"),
                    "-o", out], check=True, timeout=300)
    return out


def run(exe, *args, text=None):
    p = subprocess.run([exe, *args], input=text, capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stderr[-4000:]
    return p.stdout


def test_overlap_matches_brute_force(exe):
    """No overlap is missed; matrices of one row stride, and single rows, are refused only for one."""
    assert run(exe, "overlap", "12345", "200000").split() == ["200000", "0", "0"]


def test_random_plans_hold_their_bounds(exe):
    """Sizes up to 2^30 and workspaces up to twice what a call uses: partial sums
    and operands laid out anew fit, the parts cover the contraction, cuts and
    pieces lie on multiples of 256, and every launch is a possible one."""
    assert run(exe, "plan", "777", "200000").split() == ["200000", "0"]


def routes(exe, products, workspace=64 << 20):
    """The launches of aligned products (call, output rows, columns, contraction)."""
    lines = "".join(f"{c} 0 {m} {n} {k} 1 1 {workspace}\n" for c, m, n, k in products)
    return run(exe, "route", text=lines).splitlines()


def test_small_outputs_over_long_contractions_are_not_split_too_far(exe):
    """One thread adds an output's parts one after the other, so many parts of a
    small output cost more than they save: (33, 64, 11008) in 86 parts of
    128-tiles took 15.1 us, in 20 of 64-tiles 10.7."""
    small = [("forward", 33, 64, 11008), ("grad_input", 1, 64, 11008), ("grad_input", 16, 64, 11008),
             ("grad_weight", 64, 64, 8192), ("grad_weight", 16, 96, 19917), ("forward", 144, 32, 9456)]
    for p, r in zip(small, routes(exe, small)):
        tile, parts = r.removeprefix("direct ").split("/")
        assert tile == "64" and int(parts) <= 40, (p, r)
    # where a few parts are enough, or where each part is long, the split stays
    assert routes(exe, [("grad_input", 7, 16, 1888), ("grad_weight", 64, 64, 1 << 20)]) == ["direct 128/15", "direct 64/256"]


def test_every_way_is_in_the_gpu_tests(exe):
    """tests/linear_routes.py: each product takes the way it stands for, and every
    kernel form is among them."""
    got = run(exe, "route", text="".join(program_case(*r[:8]) for r in ROUTES)).splitlines()
    wrong = [(r, g) for r, g in zip(ROUTES, got) if r[8] != g]
    assert not wrong, wrong
    seen = {(r[0], r[1], w.split("/")[0], "split" if w.split("/")[1] != "1" else "whole", r[8].split()[0])
            for r in ROUTES if not r[8].startswith("few") for w in r[8].split() if "/" in w}
    for call, wt in KINDS:
        for tile, parts, how in (("256", "whole", "direct"), ("128", "whole", "direct"), ("128", "split", "direct"),
                                 ("64", "whole", "direct"), ("64", "split", "direct"),
                                 ("128", "whole", "staged"), ("128", "split", "staged")):
            assert (call, wt, tile, parts, how) in seen, (call, wt, tile, parts, how)
    few = {(r[1], r[6], r[8]) for r in ROUTES if r[8].startswith("few")}
    assert few >= {(wt, 1, f"few {t}x{f}") for wt in ("bf16", "e4m3") for t in (1, 2) for f in (1, 2, 3, 4)}
    assert few >= {(wt, 0, f"few 1x{f}") for wt in ("bf16", "e4m3") for f in (1, 2, 3, 4)}
