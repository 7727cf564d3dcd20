"""No copy of the library is multicast to a cluster's shared memories: each CTA loads what lands in its own.

The library is loaded by every rank of a run on several GPUs, where such loads are not used.  The one instruction that
may name the cluster is the tensor cores' commit, a barrier arrival at both CTAs of a pair."""
import pathlib
import re

import pytest

SOURCES = sorted(p for p in pathlib.Path(__file__).resolve().parents[1].joinpath("sparse_backward_gemm_gb300", "csrc").iterdir()
                 if p.suffix in (".cu", ".cuh", ".h"))
LITERALS = re.compile(r'"(?:[^"\\]|\\.)*"(?:\s*"(?:[^"\\]|\\.)*")*')


def instructions(text):
    """The instructions of all string literals, adjacent ones joined as the compiler does."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in LITERALS.finditer(text):
        yield from "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(0))).split(";")


def test_the_parser_joins_literals():
    found = list(instructions('asm("cp.async.bulk.tensor.2d"\n   ".multicast::cluster [%0];" :: "r"(x)); // "a;b"'))
    assert found == ["cp.async.bulk.tensor.2d.multicast::cluster [%0]", "", "r"]


@pytest.mark.parametrize("path", SOURCES, ids=lambda p: p.name)
def test_no_multicast_copy(path):
    for i in instructions(path.read_text()):
        if "multicast" in i:
            assert "tcgen05.commit" in i and "bulk" not in i, i
