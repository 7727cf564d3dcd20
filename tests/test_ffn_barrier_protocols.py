"""Models of the barrier protocols of the feed-forward kernels (sparse_backward_gemm_gb300/csrc/ffn_tc.cu, ffn_few.cu),
checked on the CPU as in test_barrier_protocols.py: no deadlock, no missed phase, no early arrival."""
import pytest

from test_barrier_protocols import check, ring


def pairs(segments, stages, np):
    """np pairs of CTAs that work through the same pieces (k-slices each) in step.  A pair's even CTA has the full
    barriers; every producer's copies of a slice are counted on those of the CTAs that they reach: with two pairs, on
    both.  Both pairs' MMAs hand a stage back to every CTA."""
    roles, arrivers = {}, {}
    ctas, leaders = range(2 * np), [2 * p for p in range(np)]
    reach = {c: leaders if np == 2 else [0] for c in ctas}
    for s in range(stages):
        for ld in leaders:
            arrivers[(("full", ld), s)] = [f"prod{c}" for c in ctas if ld in reach[c]]
        for c in ctas:
            arrivers[(("empty", c), s)] = [f"mma{ld}" for ld in leaders]
    for ld in leaders:
        for a in range(2):
            arrivers[(("tempty", ld), a)] = [f"epi{ld}", f"epi{ld + 1}"]
    total = sum(segments)
    for c in ctas:
        ops = []
        for i in range(total):
            if i >= stages:
                ops.append(("wait", ring(("empty", c), i - stages, stages)))
            ops += [("arrive", ring(("full", ld), i, stages)) for ld in reach[c]]
        for i in range(max(total - stages, 0), total):        # a CTA leaves when its stages are handed back
            ops.append(("wait", ring(("empty", c), i, stages)))
        roles[f"prod{c}"] = ops
        roles[f"epi{c}"] = [op for g in range(len(segments))
                            for op in (("wait", ring(("tfull", c - c % 2), g, 2)), ("arrive", ring(("tempty", c - c % 2), g, 2)))]
    for ld in leaders:
        ops, i = [], 0
        for g, n in enumerate(segments):
            if g >= 2:
                ops.append(("wait", ring(("tempty", ld), g - 2, 2)))
            for _ in range(n):
                ops.append(("wait", ring(("full", ld), i, stages)))
                ops += [("arrive", ring(("empty", c), i, stages)) for c in ctas]
                i += 1
            ops.append(("sig", ring(("tfull", ld), g, 2)))
        roles[f"mma{ld}"] = ops
    return roles, arrivers


@pytest.mark.parametrize("np", [1, 2])
@pytest.mark.parametrize("stages", [5, 7])
@pytest.mark.parametrize("segments", [[1], [3], [5, 5], [7, 1, 9], [2, 2, 2, 2], [12, 3], [1, 1, 1]])
def test_pairs(np, stages, segments):
    dead, missed, overrun = check(pairs(segments, stages, np))
    assert not dead and not missed and not overrun


def test_the_model_needs_both_pairs_to_hand_back():
    """With the empty barriers counting one pair's MMAs alone, a copy could run into a slice the other still reads."""
    roles, arrivers = pairs([12], 5, 2)
    for k in list(arrivers):
        if k[0][0] == "empty":
            arrivers[k] = ["mma0"]
    roles["mma2"] = [op for op in roles["mma2"] if not (op[0] == "arrive" and op[1][0][0][0] == "empty")]
    assert check((roles, arrivers))[2]


def few(slices, stages):
    """ffn_few.cu: the first ring-full of weights, then its tokens, then a slice at a time."""
    first = min(slices, stages)
    prod = [("arrive", ring("full", i, stages)) for i in range(first)]
    for i in range(slices):
        if i >= first:
            prod += [("wait", ring("empty", i - stages, stages)), ("arrive", ring("full", i, stages))]
    mma = []
    for i in range(slices):
        mma += [("wait", ring("full", i, stages)), ("sig", ring("empty", i, stages))]
    mma.append(("sig", ("done", 0)))
    return dict(prod=prod, mma=mma, epi=[("wait", ("done", 0))]), {("full", s): ["prod"] for s in range(stages)}


@pytest.mark.parametrize("slices", [1, 2, 4, 5, 6, 10, 11, 16, 23])
@pytest.mark.parametrize("stages", [4, 5])
def test_few(slices, stages):
    dead, missed, overrun = check(few(slices, stages))
    assert not dead and not missed and not overrun
