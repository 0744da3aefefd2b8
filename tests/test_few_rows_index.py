"""Where the kernel for few rows loads the scales and zeros of 4-bit weights and
the rows of X: its index arithmetic (csrc/few_rows_index.hpp) walked on the host,
lane by lane.  No load reaches behind the tensor, whatever its number of blocks,
and every group is loaded by the lane that hands it round; the copy of X takes
every chunk once, and of empty rows none, without dividing by their number."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("few_rows") / "few_rows_index")
    # (unoptimised: a division whose result nobody uses is made, and traps where it divides by zero)
    subprocess.run(["g++", "-O0", "-std=c++17", "-Wall", "-Werror", os.path.join(HERE, "few_rows_index.cpp"), "-o", exe],
                   check=True)
    return lambda *a: subprocess.run([exe, *map(str, a)], check=True, capture_output=True, text=True).stdout.split()


@pytest.mark.parametrize("N,K,group,reach", [
    (512, 128, 32, 8), (64, 160, 32, 6), (4, 192, 64, 2), (40, 1408, 64, 4), (9728, 896, 128, 2), (4096, 4224, 128, 2),
    (512, 256, 32, 0), (64, 4096, 64, 0), (4096, 4096, 128, 0), (33, 768, 256, 0)])
def test_no_scale_behind_the_tensor(walk, N, K, group, reach):
    """`reach`: the bytes that the lanes of a run's missing second block would
    read behind the last row, were they not kept from it."""
    free, past, right = map(int, walk(N, K, group))
    assert (free, past, right) == (reach, 0, 1)


def test_sizes_with_and_without_a_last_half_run(walk):
    out = walk("all")
    fields = dict(zip(out[0::2], map(int, out[1::2])))
    assert fields["sizes"] == 9 * (144 + 72 + 36 + 18)
    assert fields["reached"] > 0          # the sweep has sizes where it matters
    assert fields["past"] == 0 and fields["wrong"] == 0


@pytest.mark.parametrize("threads", [64, 256, 512])
@pytest.mark.parametrize("K", [0, 8, 128, 136, 4096, 14336])
def test_rows_of_x_are_copied_once(walk, K, threads):
    for rows in (1, 2, 4):
        least, most, besides = map(int, walk("copy", K, rows, threads))
        assert (least, most, besides) == ((1, 1, 0) if K else (0, 0, 0))
