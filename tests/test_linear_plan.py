"""The plan of a linear map's tiles, on the host: whatever the number of SMs, the grid's units
take each item once."""
import os
import subprocess

import pytest

from train_oracle import SHARED_ROUNDS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("c") / "plan_walk")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Wno-unused-function", "-O2",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "zero_partitioned_mixed_adam_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "plan_walk.cpp"), "-o", exe], check=True)
    return exe


def test_every_item_is_taken_once(walk):
    sms = ["152", "160", "148", "142", "132", "76", "75", "19", "2"]
    r = subprocess.run([walk, "3000", *sms], capture_output=True, text=True, timeout=300, check=True)
    got = dict(line.split() for line in r.stdout.splitlines())
    assert int(got.pop("turns")) > 100      # the drawn sizes do reach the shared rounds
    assert got == {n: "0" for n in sms}


def test_the_shapes_of_shared_rounds_have_them(walk):
    """The sizes that the GPU tests name so: dw's early tiles go round more than once."""
    for shape in SHARED_ROUNDS:
        r = subprocess.run([walk, "turns", *map(str, shape)], capture_output=True, text=True, check=True)
        assert int(r.stdout) >= 2, shape
