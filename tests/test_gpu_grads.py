"""Norm of gradients and clipping on the GPU against the float64 oracle.

The norm: squares are added 16 at a time in f32 (a sum off by at most 18 2^-24, its root by half that) and in f64 from
there; the sum is rounded to f32 (half of 2^-24 in the root), the root and its product with scale once more: 11.5 2^-24
in all.  The coefficient: three more roundings; a value one more."""
import math

import numpy as np
import pytest
import torch

from oracle import grads as og

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
NORM = 11.5 * 2.0 ** -24
COEF = NORM + 3 * 2.0 ** -24
KIND = {"l2": cl.GRAD_NORM_L2, "max": cl.GRAD_NORM_MAX}
BF, F32 = torch.bfloat16, torch.float32
GUARD = 3.0


def make(sizes, types, lead, seed, std=1.0):
    """Tensors that lie `lead` values behind each other in flat buffers filled with a mark, normal values of differing
    spread in them."""
    g = torch.Generator(device=gu.DEV).manual_seed(seed)
    flats, out = [], []
    for dt in (F32, BF):
        total = sum(n + lead for n, t in zip(sizes, types) if t == dt) + lead
        flats.append(torch.full((max(1, total),), GUARD, dtype=dt, device=gu.DEV))
    at = [lead, lead]
    for i, (n, t) in enumerate(zip(sizes, types)):
        k = int(t == BF)
        v = flats[k][at[k]: at[k] + n]
        v.copy_(torch.randn(n, generator=g, device=gu.DEV) * std * 10.0 ** (-(i % 4)))
        out.append(v)
        at[k] += n + lead
    return flats, out


def call(ts, kind="l2", scale=1.0, max_norm=None, norms=True, fill=0xFF):
    lst = cl.grad_list(ts)
    norm, coef = (torch.full((1,), 7.0, device=gu.DEV) for _ in range(2))
    each = torch.full((max(1, len(ts)),), 7.0, device=gu.DEV) if norms else None
    ws = torch.full((cl.collider_grad_norm_workspace_size(lst, len(ts)),), fill, dtype=torch.uint8, device=gu.DEV)
    if max_norm is None:
        cl.collider_grad_norm(lst, len(ts), KIND[kind], scale, norm, each, ws)
    else:
        cl.collider_grad_clip(lst, len(ts), KIND[kind], scale, max_norm, norm, each, coef, ws)
    cl.collider_check()
    return float(norm), each[: len(ts)].cpu().double().numpy() if norms else None, float(coef)


def near(a, b, rel):
    return (math.isnan(a) and math.isnan(b)) or a == b or abs(a - b) <= rel * abs(b)


def check(sizes, types, lead, kind, scale, max_norm, seed=1, std=1.0):
    flats, ts = make(sizes, types, lead, seed, std)
    before = [t.clone() for t in ts]
    host = [gu.host(t) for t in ts]
    want, want_each = og.norm(host, kind, scale)
    rel = NORM if kind == "l2" else 2 * 2.0 ** -24
    norm, each, _ = call(ts, kind, scale)
    assert near(norm, want, rel), (norm, want)
    assert all(near(a, b, rel) for a, b in zip(each, want_each))
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    norm2, each2, coef = call(ts, kind, scale, max_norm)
    assert norm2 == norm and np.array_equal(each, each2)
    assert near(coef, og.coefficient(want, max_norm, scale), COEF)
    f = np.float32(coef)
    for t, b in zip(ts, before):
        w = (b.float() * float(f)).to(t.dtype)             # in f32, rounded once: exactly this
        assert torch.equal(t, w)
    for flat in flats:                                     # the marks between the tensors stand
        inside = torch.zeros(flat.shape, dtype=torch.bool, device=gu.DEV)
        for t in ts:
            if t.dtype == flat.dtype and t.numel():
                inside[t.storage_offset(): t.storage_offset() + t.numel()] = True
        assert bool((flat[~inside] == GUARD).all())


SHAPES = [[1], [5], [0], [0, 3, 0, 0, 17, 0], [1, 1, 1, 1, 1, 1, 1], [2047, 2048, 2049, 8191, 8192, 8193, 16384, 16385],
          [100003, 7, 256, 70000], [1 << 20, 0, 3, (1 << 20) + 1], [5000017], [33] * 40, [4096] * 700 + [1] * 9]


@pytest.mark.parametrize("sizes", SHAPES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("types", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("lead", [0, 1, 3])
def test_norm_and_clip(sizes, types, lead):
    t = [BF if types == "bf16" or (types == "mixed" and i % 2) else F32 for i in range(len(sizes))]
    check(sizes, t, lead, "l2", 1.0, 0.25)
    check(sizes, t, lead, "max", 0.5, 0.1, seed=2)
    check(sizes, t, lead, "l2", 0.125, 1e9, seed=3)        # not clipped, only scaled


def test_more_tensors_than_a_launch_takes():
    sizes = [1 + (i * 37) % 300 for i in range(2500)]
    check(sizes, [F32 if i % 3 else BF for i in range(2500)], 1, "l2", 1.0, 0.5)
    check(sizes, [F32] * 2500, 0, "max", 1.0, 0.5)


def test_not_clipped_is_left_alone():
    _, ts = make([1000, 77], [F32, BF], 1, 4)
    ts[0][3] = float(np.float32(1e-40))                    # (a value that a multiplication might flush)
    before = [t.clone() for t in ts]
    for limit in (1e6, math.inf):
        _, _, coef = call(ts, "l2", 1.0, limit)
        assert coef == 1.0 and all(torch.equal(a, b) for a, b in zip(ts, before))
    _, _, coef = call(ts, "l2", 1.0, 0.0)
    assert coef == 0.0 and not any(t.any() for t in ts)


@pytest.mark.parametrize("std", [1e-43, 1e-30, 1e-22, 1e-16, 1e17, 1e19, 1e25, 1e35])
def test_values_whose_squares_leave_f32(std):
    for dt in (F32, BF):
        g = torch.Generator(device=gu.DEV).manual_seed(5)
        t = (torch.randn(70001, generator=g, device=gu.DEV, dtype=torch.float64) * std).to(dt)
        t[:: 3] *= 1e-4
        want, _ = og.norm([gu.host(t)], "l2")
        norm, _, _ = call([t], "l2")
        assert near(norm, want, NORM) or abs(norm - want) <= 2.0 ** -149, (norm, want)


def test_norms_that_do_not_fit():
    t = torch.full((1000,), 3e38, device=gu.DEV)
    for kind, limit in (("l2", 1.0),):
        norm, each, coef = call([t], kind, 1.0, limit)
        assert norm == math.inf and coef == 0.0 and bool((t == torch.tensor(3e38, device=gu.DEV)).all())
    norm, _, _ = call([t], "l2", 1e-3)                     # scaled, it fits
    assert near(norm, og.norm([gu.host(t)], "l2", 1e-3)[0], NORM + 2.0 ** -24)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dt", [F32, BF])
def test_not_finite(bad, kind, dt):
    for at in (0, 12345, 40001):
        ts = [torch.ones(100, device=gu.DEV), torch.ones(40002, device=gu.DEV, dtype=dt), torch.ones(9, device=gu.DEV)]
        ts[1][at] = bad
        before = [t.clone() for t in ts]
        norm, each, coef = call(ts, kind, 1.0, 0.5)
        assert coef == 0.0 and (math.isnan(norm) if math.isnan(bad) else norm == math.inf)
        want = [10.0, math.nan if math.isnan(bad) else math.inf, 3.0] if kind == "l2" else [1.0, each[1], 1.0]
        assert all(near(a, b, NORM) for a, b in zip(each, want)) and not math.isfinite(each[1])
        assert all(torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0)) for a, b in zip(ts, before))
    both = [torch.tensor([math.inf, math.nan], device=gu.DEV)]
    assert math.isnan(call(both, kind)[0])


def test_empty_list_and_left_out_outputs():
    norm, _, coef = call([], "l2", 1.0, 1.0)
    assert norm == 0.0 and coef == 1.0
    t = torch.ones(100, device=gu.DEV)
    lst = cl.grad_list([t])
    ws = torch.empty(cl.collider_grad_norm_workspace_size(lst, 1), dtype=torch.uint8, device=gu.DEV)
    cl.collider_grad_norm(lst, 1, cl.GRAD_NORM_L2, 1.0, None, None, ws)
    cl.collider_grad_clip(lst, 1, cl.GRAD_NORM_L2, 1.0, 5.0, None, None, None, ws)
    cl.collider_check()
    assert near(float(t[0]), 5.0 / (10.0 + 1e-6), COEF)


def test_a_gradient_listed_twice_counts_twice():
    t = torch.ones(4096, device=gu.DEV)
    assert near(call([t, t], "l2")[0], math.sqrt(8192.0), NORM)


def test_clipping_again_and_replayed():
    """Bit for bit the same from run to run, whatever the workspace held; a replayed graph reads the gradients anew."""
    _, ts = make([300000, 17, 90001], [F32, BF, F32], 1, 6)
    before = [t.clone() for t in ts]
    results = []
    for fill in (0, 0xFF):
        for t, b in zip(ts, before):
            t.copy_(b)
        results.append((call(ts, "l2", 1.0, 0.3, fill=fill), [t.clone() for t in ts]))
    (n0, e0, c0), out0 = results[0]
    (n1, e1, c1), out1 = results[1]
    assert (n0, c0) == (n1, c1) and np.array_equal(e0, e1) and all(torch.equal(a, b) for a, b in zip(out0, out1))
    lst = cl.grad_list(ts)
    norm, coef = torch.empty(1, device=gu.DEV), torch.empty(1, device=gu.DEV)
    ws = torch.empty(cl.collider_grad_norm_workspace_size(lst, 3), dtype=torch.uint8, device=gu.DEV)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        cl.collider_grad_clip(lst, 3, cl.GRAD_NORM_L2, 1.0, 0.3, norm, None, coef, ws)
    for k in (1.0, 2.0):
        for t, b in zip(ts, before):
            t.copy_(b * k)
        g.replay()
        torch.cuda.synchronize()
        want, _ = og.norm([gu.host(b * k) for b in before], "l2")
        assert near(float(norm), want, NORM)
    for t, b in zip(ts, before):
        t.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    assert float(norm) == n0 and all(torch.equal(a, b) for a, b in zip(ts, out0))


def test_offsets_beyond_32_bits():
    """A gradient of 2.2e9 values and one behind it."""
    n = (1 << 31) + 100003
    t = torch.zeros(n, dtype=BF, device=gu.DEV)
    t[0], t[n - 1], t[1 << 31] = 3.0, 4.0, 12.0
    u = torch.full((5,), 2.0, device=gu.DEV)
    norm, each, coef = call([t, u], "l2", 1.0, 6.5)
    assert near(each[0], 13.0, NORM) and near(norm, math.sqrt(169 + 20), NORM)
    for at, v in ((0, 3.0), (n - 1, 4.0), (1 << 31, 12.0)):
        assert float(t[at]) == float(torch.tensor(v * np.float32(coef)).to(BF))
    assert int(t.count_nonzero()) == 3
