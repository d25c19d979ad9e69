"""Which vectors the embedding gradient reads of rows at any address, on the host: all of a row's
elements, and nothing outside of the matrix."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("c") / "row_reads_walk")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-O2", "-I",
                    os.path.join(ROOT, "zero_partitioned_mixed_adam_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "row_reads_walk.cpp"), "-o", exe], check=True)

    def run(*args):
        r = subprocess.run([exe, *args], capture_output=True, text=True, check=True)
        return {k: int(v) for k, v in (line.split() for line in r.stdout.splitlines())}
    return run


def test_rows_are_read_whole_and_nothing_else(walk):
    got = walk()
    assert got["vectors"] > 10000 and got["cut"] > 100
    assert got["wrong"] == 0 and got["outside"] == 0
    # of the rows that are read without a look at each vector none has one that is not whole
    assert got["unsafe"] == 0 and got["most"] == 9


def test_whole_vectors_alone_would_read_outside(walk):
    """What the walk is for: with every vector read whole it counts reads outside."""
    got = walk("whole")
    assert got["wrong"] == 0 and got["outside"] > 0
