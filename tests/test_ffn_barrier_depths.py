"""The models of test_ffn_barrier_protocols.py at every ring depth that the feed-forward kernels have, as their sources
state them.  (Pairs work alone: the models' form of two pairs that share copies has no kernel.)"""
import pathlib
import re

import pytest

from test_barrier_protocols import check
from test_ffn_barrier_protocols import few, pairs

CSRC = pathlib.Path(__file__).resolve().parents[1] / "sparse_backward_gemm_gb300" / "csrc"


def depths(name):
    """The numbers that a constant kStages may take."""
    line = re.search(r"constexpr int kStages = ([^;]*);", (CSRC / name).read_text()).group(1)
    return sorted({int(v) for v in re.findall(r"[?:] (\d+)", line)})


PAIR, FEW = depths("ffn_tc.cu"), depths("ffn_few.cu")


def test_the_depths_are_found():
    assert PAIR == [6, 7] and FEW == [3, 4, 5]


@pytest.mark.parametrize("stages", PAIR)
@pytest.mark.parametrize("segments", [[1], [3], [5, 5], [6, 6], [7, 1, 9], [2, 2, 2, 2], [13, 3], [1, 1, 1]])
def test_pairs(stages, segments):
    assert not any(check(pairs(segments, stages, 1)))


@pytest.mark.parametrize("stages", FEW)
@pytest.mark.parametrize("slices", [1, 2, 3, 4, 5, 6, 7, 9, 10, 11, 16, 23])
def test_few(slices, stages):
    assert not any(check(few(slices, stages)))


def test_the_model_needs_the_stage_handed_back():
    """A producer that ran a slice ahead of the empty barrier would be seen."""
    roles, arrivers = pairs([13], 6, 1)
    for c in range(2):
        roles[f"prod{c}"] = [op for op in roles[f"prod{c}"] if op[0] != "wait"]
    dead, missed, overrun = check((roles, arrivers))
    assert missed or overrun
