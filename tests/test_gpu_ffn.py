"""Gated feed-forward block on the GPU against the float64 oracle, element by element.

Every bound counts roundings: H is half a step of bf16 (s of up to 32 tokens is kept as two bf16 values, H of H); a sum of K products in f32 is off by at most K 2^-23 of the sum
of their magnitudes (E of that sum below); the activation and its slope by 2^-18 (1 + |g|) of the magnitudes that meet
there (one exponential and one reciprocal, of arguments that f32 rounds)."""
import threading

import numpy as np
import pytest
import torch

from oracle import ffn as off
import workloads

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
ACT = {"silu": cl.GLU_SILU, "gelu_tanh": cl.GLU_GELU_TANH}
H = 2.0 ** -8
BF = torch.bfloat16


def E(k):
    return k * 2.0 ** -23


def inputs(M, D, F, seed, spread=1.0):
    r = np.random.default_rng(seed)
    b = workloads.bf16_representable
    v = dict(x=r.normal(size=(M, D)) * spread, w_up=r.normal(size=(D, 2 * F)) * D ** -0.5,
             w_down=r.normal(size=(F, D)) * F ** -0.5, dy=r.normal(size=(M, D)), up=r.normal(size=(M, 2 * F)) * 2.0 * spread)
    return {k: b(a.astype(np.float32)).astype(np.float64) for k, a in v.items()}


def forward_bounds(v, kind):
    o = off.forward(v["x"], v["w_up"], v["w_down"], kind)
    D, F = v["x"].shape[1], v["w_down"].shape[0]
    e_up = E(D) * (np.abs(v["x"]) @ np.abs(v["w_up"]))
    g, u = np.split(np.abs(o["up"]), 2, axis=1)
    eg, eu = np.split(e_up, 2, axis=1)
    ds = 1.2 * eg * (u + eu) + g * eu + 2.0 ** -18 * (1 + g) * g * u      # |a'| < 1.2, |a| <= |g|
    ds = ds + (H if len(v["x"]) > 32 else H * H) * (np.abs(o["s"]) + ds)
    wd = np.abs(v["w_down"])
    ey = ds @ wd + E(F) * ((np.abs(o["s"]) + ds) @ wd)
    return o, dict(up=H * (np.abs(o["up"]) + e_up) + e_up, y=H * (np.abs(o["y"]) + ey) + ey)


def backward_bounds(v, kind, keep, half):
    """half: half a step of the weight gradients' type."""
    o = off.backward(v["x"], v["up"], v["dy"], v["w_up"], v["w_down"], kind, keep)
    m = np.ones((len(v["x"]), 1), bool) if keep is None else np.asarray(keep, bool)[:, None]
    x, up, dy = (np.abs(np.where(m, v[k], 0.0)) for k in ("x", "up", "dy"))
    D, F, n = x.shape[1], v["w_down"].shape[0], max(1, int(m.sum()))
    g, u = np.split(up, 2, axis=1)
    wd, wu = np.abs(v["w_down"]), np.abs(v["w_up"])
    mag = dy @ wd.T
    rel = E(D) + 2.0 ** -18 * (1 + g)
    e_dup = np.concatenate((mag * u * 1.2 * rel, mag * g * rel), axis=1)
    e_dup = e_dup + H * (np.abs(o["dup"]) + e_dup)
    e_s = 2.0 ** -18 * (1 + g) * g * u
    e_s = e_s + H * (np.abs(o["s"]) + e_s)
    dup, s = np.abs(o["dup"]) + e_dup, np.abs(o["s"]) + e_s
    ex = e_dup @ wu.T + E(2 * F) * (dup @ wu.T)
    eu = x.T @ e_dup + E(n) * (x.T @ dup)
    ed = e_s.T @ dy + E(n) * (s.T @ dy)
    return o, dict(dx=ex + H * (np.abs(o["dx"]) + ex), dw_up=eu + half * (np.abs(o["dw_up"]) + eu),
                   dw_down=ed + half * (np.abs(o["dw_down"]) + ed))


def within(got, want, bound, what):
    got = gu.host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = np.max(np.abs(got - want) / (bound + 1e-30)) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of its bound"


def strided(rows, cols, pad, fill=7.0, dtype=BF):
    t = torch.full((rows, cols + pad), fill, dtype=dtype, device=gu.DEV)
    return t, t[:, :cols]


def put(v, pad=0, rows=None, fill=float("nan")):
    """v as bf16 rows with `pad` more elements each (and `rows` in all), the rest filled."""
    t, view = strided(rows or v.shape[0], v.shape[1], pad, fill)
    view[: v.shape[0]].copy_(gu.bf16(v))
    return t


def desc(M, D, F, kind, grad=cl.BF16, **ld):
    return cl.FfnDesc(M=M, D=D, F=F, act=ACT[kind], grad_dtype=grad, **ld)


GUARDS = []


def workspace(size):
    """Filled with NaNs, should anything be read before it is written; the bytes behind it are looked at after the call."""
    t = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device=gu.DEV)
    t[size:] = 0xAB
    GUARDS.append(t[size:])
    return t[:size]


def check_guards():
    assert all(bool((g == 0xAB).all()) for g in GUARDS)
    GUARDS.clear()


def run_forward(v, kind, pads=(0, 0, 0), want_up=True, stream=None):
    M, D = v["x"].shape
    F = v["w_down"].shape[0]
    d = desc(M, D, F, kind, x_ld=D + pads[0] if pads[0] else 0, up_ld=2 * F + pads[1] if pads[1] else 0,
             y_ld=D + pads[2] if pads[2] else 0)
    x, wu, wd = put(v["x"], pads[0]), gu.bf16(v["w_up"]), gu.bf16(v["w_down"])
    (ut, up), (yt, y) = strided(M, 2 * F, pads[1]), strided(M, D, pads[2])
    ws = workspace(cl.collider_ffn_fwd_workspace_size(d))
    cl.collider_ffn_fwd(d, x, wu, wd, ut if want_up else None, yt, ws, stream=stream)
    cl.collider_check()
    check_guards()
    assert bool((ut[:, 2 * F:] == 7).all()) and bool((yt[:, D:] == 7).all())
    return up, y


SIZES = [(1, 8, 8), (1, 256, 1024), (3, 1024, 2048), (17, 520, 648), (32, 64, 64), (64, 2048, 264), (65, 264, 520), (40, 520, 1032), (100, 1032, 2056), (2, 64, 136), (5, 200, 72), (16, 512, 264), (33, 1536, 96), (127, 72, 136), (128, 128, 256),
         (129, 256, 384), (192, 256, 384), (300, 200, 1000), (513, 64, 8), (700, 8, 640), (200, 256, 8192), (1025, 384, 1096),
         (1300, 512, 2048), (2300, 1024, 2816)]


@pytest.mark.parametrize("M,D,F", SIZES)
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_forward(M, D, F, kind):
    v = inputs(M, D, F, M + D + F)
    o, b = forward_bounds(v, kind)
    up, y = run_forward(v, kind)
    within(up, o["up"], b["up"], "up")
    within(y, o["y"], b["y"], "y")
    up2, y2 = run_forward(v, kind, (8, 24, 16))          # strided: the same bits
    assert torch.equal(up2, up) and torch.equal(y2, y)
    none, y3 = run_forward(v, kind, want_up=False)       # not kept: left as it was
    assert torch.equal(y3, y) and bool((none == 7).all())


def test_forward_wide_values():
    """Gates of up to some hundreds, where the activation is 0 or the gate itself."""
    for kind in ("silu", "gelu_tanh"):
        v = inputs(70, 96, 200, 3, spread=60.0)
        o, b = forward_bounds(v, kind)
        up, y = run_forward(v, kind)
        within(up, o["up"], b["up"], "up")
        within(y, o["y"], b["y"], "y")


def test_forward_keeps_infinities_in_their_rows():
    v = inputs(300, 64, 128, 5)
    want = [gu.host(t) for t in run_forward(v, "silu")]
    v["x"][17, 3], v["x"][200, 5] = np.inf, np.nan
    got = [gu.host(t) for t in run_forward(v, "silu")]
    rest = np.setdiff1d(np.arange(300), [17, 200])
    for g, w in zip(got, want):
        assert np.array_equal(g[rest], w[rest]) and not np.isfinite(g[[17, 200]]).any(axis=1).all()
        assert np.isnan(g[200]).all()


def test_forward_of_few_tokens_keeps_infinities():
    """An s that bf16 takes for infinity gives y what one infinity gives, in its row alone."""
    v = inputs(5, 64, 128, 6)
    v["x"][:], v["w_up"][:] = 1.0, 0.0
    v["w_up"][0, :2], v["w_up"][0, 128:130] = 2.0 ** 60, 1.0
    v["x"][2, 0] = 2.0 ** 34                               # s = 2^94 * 2^34 = 2^128 there, at columns 0 and 1
    v["w_down"][0], v["w_down"][1] = 1.0, 0.5
    up, y = run_forward(v, "silu")
    y = gu.host(y)
    assert (y[2] == np.inf).all()
    assert np.array_equal(y[[0, 1, 3, 4]], np.full((4, 64), 1.5 * 2.0 ** 60))


def index(M, f, seed):
    """A keep-mask and its index; f None: all tokens, without an index."""
    if f is None:
        return None, None, None
    keep = np.random.default_rng(seed).random(M) >= f
    if f == 0.99:
        keep[:] = False
        keep[M // 2] = True
    rows = np.flatnonzero(keep)
    idx = np.full(M, 1 << 30)                            # never read behind the kept ones
    idx[: rows.size] = rows
    return keep, gu.i32(idx), gu.i32([rows.size])


def run_backward(v, kind, keep, idx, nk, saved=0, dyr=0, dxr=0, grad=cl.BF16, pads=(0, 0, 0), want="xud", stream=None):
    M, D = v["x"].shape
    F = v["w_down"].shape[0]
    d = desc(M, D, F, kind, grad, x_ld=D + pads[0] if pads[0] else 0, up_ld=2 * F + pads[1] if pads[1] else 0,
             y_ld=D + pads[2] if pads[2] else 0)
    mask = np.ones(M, bool) if keep is None else keep
    n = int(mask.sum())

    def rows(k, form, pad):
        a = v[k].copy()
        if form == cl.ROWS_COMPACT:
            return put(a[mask], pad, rows=max(1, n))     # room for the kept rows alone
        a[~mask] = np.nan                                # filtered rows are never used
        return put(a, pad)
    x, up, dy = rows("x", saved, pads[0]), rows("up", saved, pads[1]), rows("dy", dyr, pads[2])
    gdt = BF if grad == cl.BF16 else torch.float32
    dx, dxv = strided(M, D, pads[0])
    dwu, dwd = (torch.full(s, 7.0, dtype=gdt, device=gu.DEV) for s in ((D, 2 * F), (F, D)))
    ws = workspace(cl.collider_ffn_bwd_workspace_size(d))
    cl.collider_ffn_bwd(d, gu.bf16(v["w_up"]) if "x" in want else None, gu.bf16(v["w_down"]), x if "u" in want else None, up,
                        saved, dy, dyr, idx, nk, dx if "x" in want else None, dxr, dwu if "u" in want else None,
                        dwd if "d" in want else None, ws, stream=stream)
    cl.collider_check()
    check_guards()
    assert bool((dx[:, D:] == 7).all())
    if dxr == cl.ROWS_COMPACT and keep is not None and "x" in want:
        end = min(M, -(-n // 128) * 128)
        assert not dxv[n:end].any() and bool((dxv[end:] == 7).all())
    return dxv, dwu, dwd


def check_backward(v, kind, keep, got, dxr=0, grad=cl.BF16, want="xud"):
    o, b = backward_bounds(v, kind, keep, H if grad == cl.BF16 else 2.0 ** -24)
    dx, dwu, dwd = got
    if "x" in want:
        if dxr == cl.ROWS_COMPACT and keep is not None:
            within(dx[: int(keep.sum())], o["dx"][keep], b["dx"][keep], "dx")
        else:
            within(dx, o["dx"], b["dx"], "dx")
            assert keep is None or not dx[torch.from_numpy(~keep).to(gu.DEV)].any()
    for name, t in (("dw_up", dwu), ("dw_down", dwd)):
        if name[3] in want:
            within(t, o[name], b[name], name)
        else:
            assert bool((t == 7).all())


@pytest.mark.parametrize("M,D,F", SIZES)
@pytest.mark.parametrize("f", [None, 0.0, 0.4, 0.99, 1.0])
def test_backward(M, D, F, f):
    kind = "silu" if (M + F) % 16 else "gelu_tanh"
    v = inputs(M, D, F, M + D)
    keep, idx, nk = index(M, f, M)
    got = run_backward(v, kind, keep, idx, nk)
    check_backward(v, kind, keep, got)
    again = run_backward(v, kind, keep, idx, nk, pads=(8, 16, 24))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("grad", [cl.BF16, cl.F32])
@pytest.mark.parametrize("saved,dyr,dxr", [(0, 1, 0), (1, 0, 1), (1, 1, 1), (0, 0, 1), (1, 1, 0)])
@pytest.mark.parametrize("M,f", [(290, 0.4), (130, 0.99), (257, None), (140, 1.0)])
def test_backward_rows(kind, grad, saved, dyr, dxr, M, f):
    v = inputs(M, 136, 264, 11)
    keep, idx, nk = index(M, f, 7)
    check_backward(v, kind, keep, run_backward(v, kind, keep, idx, nk, saved, dyr, dxr, grad), dxr, grad)


@pytest.mark.parametrize("want", ["x", "u", "d", "xu", "ud", "xd", ""])
@pytest.mark.parametrize("f", [None, 0.3])
def test_backward_of_some(want, f):
    v = inputs(200, 64, 256, 12)
    keep, idx, nk = index(200, f, 3)
    check_backward(v, "silu", keep, run_backward(v, "silu", keep, idx, nk, want=want), want=want)


def test_backward_wide_values():
    for kind in ("silu", "gelu_tanh"):
        v = inputs(150, 96, 200, 13, spread=40.0)
        check_backward(v, kind, None, run_backward(v, kind, None, None, None))


def test_kept_index_outside_the_tokens():
    """Reported; its row counts as zeros, the others' gradients are what they are without it."""
    v = inputs(200, 64, 128, 14)
    keep, idx, nk = index(200, 0.4, 5)
    n = int(keep.sum())
    rows = np.flatnonzero(keep)
    for bad in (200, -1, 1 << 30):
        bidx = idx.clone()
        bidx[n - 1] = bad
        with pytest.raises(cl.ColliderError) as e:
            run_backward(v, "silu", keep, bidx, nk)
        assert e.value.status == cl.ERR_INVALID_ARG
    # (the call's outputs, once the report is taken)
    k2 = keep.copy()
    k2[rows[-1]] = False
    M, D, F = 200, 64, 128
    d = desc(M, D, F, "silu")
    dx = torch.full((M, D), 7.0, dtype=BF, device=gu.DEV)
    dwu, dwd = torch.empty(D, 2 * F, dtype=BF, device=gu.DEV), torch.empty(F, D, dtype=BF, device=gu.DEV)
    t = {k: gu.bf16(a) for k, a in v.items()}
    cl.collider_ffn_bwd(d, t["w_up"], t["w_down"], t["x"], t["up"], 0, t["dy"], 0, bidx, nk, dx, 0, dwu, dwd,
                        workspace(cl.collider_ffn_bwd_workspace_size(d)))
    with pytest.raises(cl.ColliderError):
        cl.collider_check()
    check_backward(v, "silu", k2, (dx, dwu, dwd))


def step(v, kind, B, T, keep):
    """Forward and backward of one block's MLP as a training step calls them, and the buffers."""
    M, D, F = B * T, v["x"].shape[1], v["w_down"].shape[0]
    d = desc(M, D, F, kind, cl.F32)
    t = {k: gu.bf16(v[k]) for k in ("x", "w_up", "w_down", "dy")}
    t.update(up=torch.empty(M, 2 * F, dtype=BF, device=gu.DEV), y=torch.empty(M, D, dtype=BF, device=gu.DEV),
             dx=torch.empty(M, D, dtype=BF, device=gu.DEV), dwu=torch.empty(D, 2 * F, device=gu.DEV),
             dwd=torch.empty(F, D, device=gu.DEV), norm=torch.empty(1, device=gu.DEV), coef=torch.empty(1, device=gu.DEV))
    t["idx"], _, t["nk"] = gu.compact(keep.reshape(B, T))
    t["list"] = cl.grad_list([t["dwu"], t["dwd"]])
    ws = [workspace(n) for n in (cl.collider_ffn_fwd_workspace_size(d), cl.collider_ffn_bwd_workspace_size(d),
                                 cl.collider_grad_norm_workspace_size(t["list"], 2))]

    def run():
        cl.collider_ffn_fwd(d, t["x"], t["w_up"], t["w_down"], t["up"], t["y"], ws[0])
        cl.collider_ffn_bwd(d, t["w_up"], t["w_down"], t["x"], t["up"], 0, t["dy"], 0, t["idx"], t["nk"], t["dx"], 0,
                            t["dwu"], t["dwd"], ws[1])
        cl.collider_grad_clip(t["list"], 2, cl.GRAD_NORM_L2, 1.0, 0.5, t["norm"], None, t["coef"], ws[2])
    return t, run


def test_a_training_step():
    """Forward, filtered backward, clipping: against the oracle, then captured and replayed on new inputs."""
    B, T, D, F = 2, 150, 128, 320
    keep = np.random.default_rng(8).random(B * T) >= 0.4
    v = inputs(B * T, D, F, 15)
    t, run = step(v, "silu", B, T, keep)
    outs = ("y", "up", "dx", "dwu", "dwd", "norm", "coef")

    def check(v):
        cl.collider_check()
        assert all(bool((g == 0xAB).all()) for g in GUARDS)
        o, b = forward_bounds(v, "silu")
        within(t["y"], o["y"], b["y"], "y")
        v = dict(v, up=gu.host(t["up"]))
        o, b = backward_bounds(v, "silu", keep, 2.0 ** -24)
        within(t["dx"], o["dx"], b["dx"], "dx")
        norm, coef = float(t["norm"]), float(t["coef"])
        want = np.sqrt((o["dw_up"] ** 2).sum() + (o["dw_down"] ** 2).sum())
        slack = np.sqrt((b["dw_up"] ** 2).sum() + (b["dw_down"] ** 2).sum()) + 1e-6 * want
        assert abs(norm - want) <= slack and abs(coef - 0.5 / (norm + 1e-6)) <= 1e-6 * coef
        for name, k in (("dw_up", "dwu"), ("dw_down", "dwd")):
            within(gu.host(t[k]) / coef, o[name], b[name] + 2.0 ** -22 * np.abs(o[name]), name)
    run()
    check(v)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            run()
    v2 = inputs(B * T, D, F, 16)
    for k in ("x", "w_up", "w_down", "dy"):
        t[k].copy_(gu.bf16(v2[k]))
    g.replay()
    torch.cuda.synchronize()
    check(v2)
    first = {k: t[k].clone() for k in outs}
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], t[k]) for k in outs)
    run()
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], t[k]) for k in outs)


def test_two_streams_and_two_threads():
    """Calls at once, each with its own buffers and stream, give what they give alone."""
    B, T, D, F = 1, 260, 192, 512
    keep = np.random.default_rng(9).random(T) >= 0.3
    jobs = [step(inputs(T, D, F, 20 + i), "gelu_tanh", B, T, keep) for i in range(2)]
    outs = ("y", "up", "dx", "dwu", "dwd", "norm", "coef")
    want = []
    for t, run in jobs:
        run()
        cl.collider_check()
        want.append({k: t[k].clone() for k in outs})
    errors = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    jobs[i][1]()
                cl.collider_check()
        except Exception as e:   # noqa: BLE001 (reported below)
            errors.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(2):
        assert all(torch.equal(want[i][k], jobs[i][0][k]) for k in outs)


def test_offsets_beyond_32_bits():
    """up holds 2.2e9 values: the rows at its end against the oracle."""
    M, D, F = 270001, 64, 4096
    r = torch.Generator(device=gu.DEV).manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=r, device=gu.DEV)  # noqa: E731
    t = dict(x=n(M, D).to(BF), w_up=(n(D, 2 * F) * D ** -0.5).to(BF), w_down=(n(F, D) * F ** -0.5).to(BF), dy=n(M, D).to(BF))
    up, y = torch.full((M, 2 * F), 7.0, dtype=BF, device=gu.DEV), torch.full((M, D), 7.0, dtype=BF, device=gu.DEV)
    d = desc(M, D, F, "silu")
    cl.collider_ffn_fwd(d, t["x"], t["w_up"], t["w_down"], up, y, torch.empty(cl.collider_ffn_fwd_workspace_size(d),
                                                                              dtype=torch.uint8, device=gu.DEV))
    cl.collider_check()
    at = np.r_[0:3, 131070:131074, M - 140: M]
    v = {k: gu.host(a if k[0] == "w" else a[at]) for k, a in t.items()}
    o, b = forward_bounds(v, "silu")
    within(up[at], o["up"], b["up"], "up")
    within(y[at], o["y"], b["y"], "y")
    # backward: two kept rows of every three behind the first half, so that rows move
    rows = torch.arange(M // 2, M, device=gu.DEV)
    rows = rows[rows % 3 != 0]
    idx = torch.zeros(M, dtype=torch.int32, device=gu.DEV)
    idx[: rows.numel()] = rows.to(torch.int32)
    nk = torch.tensor([rows.numel()], dtype=torch.int32, device=gu.DEV)
    dx = torch.full((M, D), 7.0, dtype=BF, device=gu.DEV)
    ws = torch.empty(cl.collider_ffn_bwd_workspace_size(d), dtype=torch.uint8, device=gu.DEV)
    cl.collider_ffn_bwd(d, t["w_up"], t["w_down"], None, up, 0, t["dy"], 0, idx, nk, dx, 0, None, None, ws)
    cl.collider_check()
    v["up"] = gu.host(up[at])
    keep = (at >= M // 2) & (at % 3 != 0)
    o, b = backward_bounds(v, "silu", keep, H)
    within(dx[at], o["dx"], b["dx"], "dx")
    assert not dx[: M // 2].any()
