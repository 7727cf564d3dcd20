"""The residual join on the GPU (norms after and before a branch, gate, residual scale), forward and backward,
against the float64 oracle; and a sandwich-normed branch run through the operators together."""
import numpy as np
import pytest
import torch

from oracle import ckpt as ock
from oracle import join as oj
import workloads

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
FMT = {"e4m3": cl.CKPT_E4M3, "int8": cl.CKPT_INT8}
EPS = 1e-5
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}    # half a step, relative


class Case:
    def __init__(self, B, T, D, dtype="bf16", ln=False, gate=0, res=False, post=True, pre=True, branch=True, alpha=1.0,
                 f=0.4, pad=0, seed=0):
        self.B, self.T, self.D, self.M = B, T, D, B * T
        self.dtype, self.ln, self.alpha, self.branch, self.pad = dtype, ln, alpha, branch, pad
        rng = np.random.default_rng(seed + 1000 * B + 10 * T + D)
        r = (lambda v: workloads.bf16_representable(v).astype(np.float64)) if dtype == "bf16" else \
            (lambda v: np.asarray(v, np.float32).astype(np.float64))
        self.store = r
        n = lambda *s: rng.normal(size=s)  # noqa: E731
        wide = np.where(rng.random(D) < 0.03, 10.0, 1.0)
        self.x, self.y = r(n(self.M, D) * wide), (r(0.3 * n(self.M, D) * wide + 0.1) if branch else None)
        self.p = dict(post_w=r(1 + 0.1 * n(D)) if post else None, post_b=r(0.1 * n(D)) if post and ln else None,
                      gate=r(0.3 + 0.1 * n(gate, D)) if gate else None, res_w=r(1 + 0.1 * n(D)) if res else None,
                      pre_w=r(1 + 0.1 * n(D)) if pre else None, pre_b=r(0.1 * n(D)) if pre and ln else None)
        self.da, self.dh = r(n(self.M, D)) if pre else None, r(n(self.M, D))
        self.keep = (rng.random((B, T)) >= f).astype(np.uint8)
        self.post, self.pre = post, pre
        self.desc = cl.ResidualNormDesc(dtype=cl.BF16 if dtype == "bf16" else cl.F32, B=B, T=T, D=D,
                                        norm=cl.NORM_LAYER if ln else cl.NORM_RMS, post=int(post), pre=int(pre), eps=EPS,
                                        res_scale=alpha, gate_rows=gate)
        if pad:
            self.desc.x_ld = D + pad
            self.desc.y_ld = self.desc.h_ld = self.desc.a_ld = D + 2 * pad
        self.tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.params = cl.residual_norm_params(**{k: self.up(v) for k, v in self.p.items()})

    def up(self, v):
        return None if v is None else (gu.bf16(v) if self.dtype == "bf16" else gu.f32(v))

    def rows(self, which, v=None, fill=7.0):
        """A [M, D] view with the case's row stride."""
        ld = getattr(self.desc, which + "_ld") or self.D
        t = torch.full((self.M, ld), fill, dtype=self.tdt, device=gu.DEV)
        if v is not None:
            t[:, : self.D] = self.up(v)
        return t

    def forward(self):
        x, y = self.rows("x", self.x), self.rows("y", self.y) if self.branch else None
        o = dict(h=self.rows("h") if self.branch else None, a=self.rows("a") if self.pre else None)
        for k, there in (("rstd_y", self.post), ("rstd_h", self.pre), ("mean_y", self.post and self.ln),
                         ("mean_h", self.pre and self.ln)):
            o[k] = torch.full((self.M,), 7.0, device=gu.DEV) if there else None
        cl.collider_residual_norm_fwd(self.desc, self.params, x, y, cl.residual_norm_out(**o))
        cl.collider_check()
        return o

    # f32 work before the rounding: a row sum is a tree of at most 64 additions (per thread 16, lanes 5, warps 16,
    # and slack), so a statistic is within 2^-17 relative of its magnitudes; each product and sum after it adds 2^-24
    def check_forward(self, o):
        D, p, e, half = self.D, self.p, 2.0 ** -17, HALF[self.dtype]
        ref = oj.join_forward(self.x, self.y, p, self.B, self.T, self.alpha, self.ln, EPS)
        h = self.x
        if self.branch:
            lam = self.alpha * (1.0 if p["res_w"] is None else p["res_w"])
            g = np.abs(oj.gate_rows(p["gate"], self.B, self.T, D))
            hat = np.abs(self.y)
            if self.post:
                m, r = ref["mean_y"], ref["rstd_y"]
                self.check_stats(o, "y", self.y, m, r)
                hat = (np.abs(self.y - m[:, None]) * r[:, None] + 1) * np.abs(p["post_w"])
                if p["post_b"] is not None:
                    hat = hat + np.abs(p["post_b"])
            mag = np.abs(lam * self.x) + g * hat
            h = gu.host(o["h"][:, :D])
            assert np.all(np.abs(h - ref["h"]) <= half * (np.abs(ref["h"]) + e * mag) + e * mag)
            assert bool((o["h"][:, D:] == 7).all())
        if self.pre:
            m, r = oj.stats(h, self.ln, EPS)            # of h as it is stored
            self.check_stats(o, "h", h, m, r)
            want = oj.norm(h, m, r, p["pre_w"], p["pre_b"])
            mag = (np.abs(h - m[:, None]) * r[:, None] + 1) * np.abs(p["pre_w"])
            if p["pre_b"] is not None:
                mag = mag + np.abs(p["pre_b"])
            a = gu.host(o["a"][:, :D])
            assert np.all(np.abs(a - want) <= half * (np.abs(want) + e * mag) + e * mag)
            assert bool((o["a"][:, D:] == 7).all())

    def check_stats(self, o, k, v, m, r):
        assert np.all(np.abs(gu.host(o["rstd_" + k]) - r) <= 2.0 ** -17 * r)
        if self.ln:
            assert np.all(np.abs(gu.host(o["mean_" + k]) - m) <= 2.0 ** -17 * np.mean(np.abs(v), axis=1))

    def saved(self, form):
        """What the backward reads: h and statistics of the oracle's forward, y and h as rows or decoded checkpoints."""
        ref = oj.join_forward(self.x, self.y, self.p, self.B, self.T, self.alpha, self.ln, EPS, store=self.store)
        f32 = lambda v: np.asarray(v, np.float32).astype(np.float64)  # noqa: E731
        st = {k: f32(ref[k]) if k in ref else np.zeros(self.M) for k in ("mean_y", "rstd_y", "mean_h", "rstd_h")}
        y, h = self.y, ref["h"] if self.branch else self.x
        cks = {}
        if form != "rows":
            for k, v in (("y", y), ("h", h)):
                if v is not None:
                    cks[k] = ock.pack(v, form)
            y = None if y is None else ock.unpack(*cks["y"], form)
            h = ock.unpack(*cks["h"], form)
        return y, h, st, cks

    def backward(self, form="rows", saved_rows=0, in_rows=0, out_rows=0, dense=False, dh=True, skip=(), alias=False,
                 ws=None, data=None):
        y, h, st, cks = data or self.saved(form)
        M, D = self.M, self.D
        keep = np.ones_like(self.keep) if dense else self.keep
        km = np.flatnonzero(keep.reshape(-1))
        idx = np.full(M, -1)
        idx[: km.size] = km
        cu = np.concatenate([[0], np.cumsum(keep.sum(1))])
        index = (None, None, None) if dense else (gu.i32(idx), gu.i32(cu), gu.i32([km.size]))
        lay = lambda v, r: v if v is None or r == 0 else np.concatenate([v[km], np.full((M - km.size, v.shape[1]), 99)])  # noqa: E731
        sv = {}
        if self.p["res_w"] is not None:
            sv["x"] = self.rows("x", lay(self.x, saved_rows))
        for k, v, there in (("y", y, self.branch), ("h", h, self.pre)):
            if not there:
                continue
            if form == "rows":
                sv[k] = self.rows(k, lay(v, saved_rows))
            else:
                c, e = (torch.from_numpy(np.ascontiguousarray(lay(t.astype(np.int64), saved_rows)).astype(np.uint8)).to(
                    gu.DEV) for t in cks[k])
                sv[k + "_ckpt"] = cl.ckpt(FMT[form], c, e)
        for k, there in (("rstd_y", self.post), ("mean_y", self.post and self.ln), ("rstd_h", self.pre),
                         ("mean_h", self.pre and self.ln)):
            if there:
                sv[k] = gu.f32(st[k])
        G = dict(dx=self.rows("x"), dy=self.rows("y") if self.branch else None)
        for k, w in (("dpost_w", "post_w"), ("dpost_b", "post_b"), ("dgate", "gate"), ("dres_w", "res_w"),
                     ("dpre_w", "pre_w"), ("dpre_b", "pre_b")):
            there = self.p[w] is not None and k not in skip
            G[k] = torch.full(self.p[w].shape, 7.0, device=gu.DEV) if there else None
        gdh = self.rows("h", lay(self.dh, in_rows)) if dh else None
        if alias:
            G["dx"] = gdh
        if ws is None:
            ws = torch.empty(cl.collider_residual_norm_bwd_workspace_size(self.desc), dtype=torch.uint8,
                             device=gu.DEV).fill_(255)
        cl.collider_residual_norm_bwd(self.desc, self.params, cl.residual_norm_saved(**sv), saved_rows,
                                      self.rows("a", lay(self.da, in_rows)) if self.pre else None, gdh, in_rows, *index,
                                      cl.residual_norm_grads(**G), out_rows, ws)
        cl.collider_check()
        ref, mag = oj.join_backward(self.x if self.p["res_w"] is not None else None, y, h, st, self.da,
                                    self.dh if dh else None, self.p, self.B, self.T, keep, self.alpha, self.ln)
        return G, ref, mag, km

    def check_backward(self, **kw):
        out_rows = kw.get("out_rows", 0)
        G, ref, mag, km = self.backward(**kw)
        n, D, e, half = km.size, self.D, 2.0 ** -17, HALF[self.dtype]
        for k in ("dx", "dy"):
            if G[k] is None:
                continue
            got, want, m = gu.host(G[k][:, :D]), ref[k], mag[k]
            if out_rows == 1:
                pad = min(-(-n // 128) * 128, self.M)
                assert np.all(got[n:pad] == 0), k
                if not kw.get("alias"):
                    assert np.all(got[pad:] == 7), k
                got, want, m = got[:n], want[km], m[km]
            if not kw.get("alias"):
                assert bool((G[k][:, D:] == 7).all()), k
            assert np.all(np.abs(got - want) <= half * (np.abs(want) + e * m) + e * m), k
        # sums over n rows: 2^-17 of each term (a row's own error), and n + 64 additions
        for k in ("dpost_w", "dpost_b", "dgate", "dres_w", "dpre_w", "dpre_b"):
            if G[k] is not None:
                assert np.all(np.abs(gu.host(G[k]) - ref[k]) <= (e + (n + 64) * 2.0 ** -24) * mag[k]), k
        return G


SHAPES = [(1, 1, 8), (1, 1, 2048), (2, 3, 64), (3, 37, 264), (2, 130, 1000), (4, 65, 1536), (1, 300, 4096), (1, 9, 4104),
          (2, 5, 8192)]


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ln", [False, True])
def test_forward(B, T, D, dtype, ln):
    c = Case(B, T, D, dtype, ln, gate=B, res=True, alpha=0.5, pad=8)
    c.check_forward(c.forward())


@pytest.mark.parametrize("kw", [dict(gate=0), dict(gate=1), dict(post=False), dict(post=False, gate=2), dict(pre=False),
                                dict(pre=False, post=False, gate=1), dict(branch=False, post=False), dict(res=True),
                                dict(alpha=-2.0, gate=2)])
@pytest.mark.parametrize("ln", [False, True])
def test_forward_parts(kw, ln):
    c = Case(2, 21, 192, ln=ln, **kw)
    c.check_forward(c.forward())


def test_forward_in_place_and_degenerate_rows():
    c = Case(2, 70, 512, gate=1)
    c.y[3] = 0.0                                # a row whose norm is all epsilon
    c.x[5] = c.y[5] = 0.0
    o = c.forward()
    c.check_forward(o)
    assert np.all(gu.host(o["a"][5]) == 0) and abs(float(o["rstd_y"][3]) - EPS ** -0.5) < 1e-3 * EPS ** -0.5
    for which in ("x", "y"):                    # h in the place of x, and of y
        x, y = c.rows("x", c.x), c.rows("y", c.y)
        h = x if which == "x" else y
        a, ry, rh = c.rows("a"), torch.empty(c.M, device=gu.DEV), torch.empty(c.M, device=gu.DEV)
        cl.collider_residual_norm_fwd(c.desc, c.params, x, y, cl.residual_norm_out(h=h, a=a, rstd_y=ry, rstd_h=rh))
        assert torch.equal(h, o["h"]) and torch.equal(a, o["a"])
    c.y[7, 100] = np.nan                        # stays in its row
    o2 = c.forward()
    bad = torch.isnan(o2["h"]).any(1)
    assert bad[7] and int(bad.sum()) == 1 and torch.equal(o2["a"][8:], o["a"][8:])


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("dtype,ln", [("bf16", False), ("bf16", True), ("f32", False), ("f32", True)])
def test_backward(B, T, D, dtype, ln):
    Case(B, T, D, dtype, ln, gate=B, res=True, alpha=0.5, pad=8).check_backward()


@pytest.mark.parametrize("form", ["e4m3", "int8"])
@pytest.mark.parametrize("saved_rows", [0, 1])
@pytest.mark.parametrize("B,T,D,dtype,ln", [(1, 1, 32, "bf16", False), (3, 50, 96, "bf16", True), (2, 77, 2048, "bf16", False),
                                            (2, 33, 1536, "f32", True), (1, 40, 4128, "bf16", False)])
def test_backward_from_checkpoints(form, saved_rows, B, T, D, dtype, ln):
    Case(B, T, D, dtype, ln, gate=B, res=True).check_backward(form=form, saved_rows=saved_rows)


@pytest.mark.parametrize("saved_rows,in_rows,out_rows", [(0, 0, 1), (0, 1, 0), (1, 0, 0), (1, 1, 1)])
def test_backward_row_layouts(saved_rows, in_rows, out_rows):
    Case(3, 111, 320, gate=3, res=True).check_backward(saved_rows=saved_rows, in_rows=in_rows, out_rows=out_rows)


@pytest.mark.parametrize("kw", [dict(gate=0), dict(gate=1), dict(post=False), dict(post=False, gate=2), dict(pre=False),
                                dict(pre=False, post=False, gate=1), dict(branch=False, post=False), dict(res=True),
                                dict(alpha=-2.0, gate=2)])
@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("dense", [False, True])
def test_backward_parts(kw, ln, dense):
    c = Case(2, 150, 192, ln=ln, **kw)
    c.check_backward(dense=dense)
    if c.pre:
        c.check_backward(dense=dense, dh=False)


@pytest.mark.parametrize("B,T,D", [(70, 3, 64), (5, 200, 128), (300, 1, 256)])
def test_gates_of_many_sequences(B, T, D):
    """Sequences shorter than a block's share of rows, some of them without a kept token."""
    c = Case(B, T, D, "f32", gate=B, f=0.5)
    c.keep[1::3] = 0
    c.check_backward()
    c.keep[:] = 0
    c.keep[B // 2, 0] = 1
    c.check_backward()


def test_gates_of_more_sequences_than_a_grid_is_high():
    c = Case(70001, 1, 8, "f32", gate=70001, f=0.3)
    c.check_forward(c.forward())
    c.check_backward()


def test_nothing_kept():
    c = Case(2, 200, 256, gate=2, res=True)
    c.keep[:] = 0
    for out_rows in (0, 1):
        G, _, _, _ = c.backward(out_rows=out_rows)
        for k in ("dpost_w", "dgate", "dres_w", "dpre_w"):
            assert bool((G[k] == 0).all())
        for k in ("dx", "dy"):
            assert bool((G[k] == (0 if out_rows == 0 else 7)).all())


def test_unwanted_gradients_and_dx_in_the_place_of_dh():
    c = Case(2, 90, 448, gate=2, res=True)
    full = c.check_backward()
    part = c.check_backward(skip=("dpost_w", "dres_w", "dgate"))
    none = c.check_backward(skip=("dpost_w", "dres_w", "dgate", "dpre_w"))
    for k in ("dx", "dy", "dpre_w"):
        assert torch.equal(part[k], full[k]) and (k == "dpre_w" or torch.equal(none[k], full[k]))
    c.check_backward(alias=True)
    c.check_backward(alias=True, in_rows=1, out_rows=1)


def test_filtered_rows_reach_nothing():
    """NaN in every filtered row of what the backward reads."""
    c = Case(2, 120, 256, gate=2, res=True)
    clean = c.check_backward()
    y, h, st, _ = c.saved("rows")
    gone = c.keep.reshape(-1) == 0
    for v in (c.x, y, h, c.da, c.dh, *st.values()):
        v[gone] = np.nan
    G, _, _, _ = c.backward(data=(y, h, st, {}))
    for k in G:
        assert G[k] is None or torch.equal(G[k], clean[k]), k


def test_bad_index_is_skipped_and_reported():
    c = Case(1, 40, 64, gate=1)
    y, h, st, _ = c.saved("rows")
    idx = np.arange(40)
    idx[11] = 4000
    G = dict(dx=c.rows("x"), dy=c.rows("y"))
    ws = torch.empty(cl.collider_residual_norm_bwd_workspace_size(c.desc), dtype=torch.uint8, device=gu.DEV)
    sv = cl.residual_norm_saved(y=c.rows("y", y), h=c.rows("h", h), rstd_y=gu.f32(st["rstd_y"]), rstd_h=gu.f32(st["rstd_h"]))
    cl.collider_residual_norm_bwd(c.desc, c.params, sv, 0, c.rows("a", c.da), c.rows("h", c.dh), 0, gu.i32(idx),
                                  gu.i32([0, 40]), gu.i32([40]), cl.residual_norm_grads(**G), 0, ws)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_check()
    assert e.value.status == cl.ERR_INVALID_ARG
    assert bool((G["dx"][11] == 7).all()) and bool(torch.isfinite(G["dx"]).all())


def test_bit_identical_on_another_stream():
    c = Case(3, 257, 768, gate=3, res=True, f=0.3)
    data = c.saved("e4m3")
    first = c.check_backward(form="e4m3", data=data)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again, _, _, _ = c.backward(form="e4m3", data=data)
    side.synchronize()
    for k, v in first.items():
        assert v is None or torch.equal(v, again[k]), k


def test_offsets_beyond_32_bits():
    """Rows 2^28 elements apart: the last row of nine lies beyond 2^32 bytes.  All tensors are columns of one buffer."""
    D, ld = 64, 1 << 28
    c = Case(3, 3, D, gate=3, res=True, f=0.3)
    want_f, want_b = c.forward(), c.check_backward()
    big = torch.empty(c.M * ld, dtype=torch.bfloat16, device=gu.DEV).view(c.M, ld)
    names = ["x", "y", "h", "a", "da", "dh", "dx", "dy"]
    t = {k: big[:, i * D:(i + 1) * D] for i, k in enumerate(names)}
    d = cl.ResidualNormDesc.from_buffer_copy(c.desc)
    d.x_ld = d.y_ld = d.h_ld = d.a_ld = ld
    for k, v in (("x", c.x), ("y", c.y), ("da", c.da), ("dh", c.dh)):
        t[k].copy_(c.up(v))
    ry, rh = torch.empty(c.M, device=gu.DEV), torch.empty(c.M, device=gu.DEV)
    cl.collider_residual_norm_fwd(d, c.params, t["x"], t["y"], cl.residual_norm_out(h=t["h"], a=t["a"], rstd_y=ry, rstd_h=rh))
    assert torch.equal(t["h"], want_f["h"]) and torch.equal(t["a"], want_f["a"]) and torch.equal(rh, want_f["rstd_h"])
    y, h, st, _ = c.saved("rows")
    t["h"].copy_(c.up(h))
    km = np.flatnonzero(c.keep.reshape(-1))
    idx = np.full(c.M, -1)
    idx[: km.size] = km
    G = {k: torch.empty_like(want_b[k]) for k in ("dpost_w", "dgate", "dres_w", "dpre_w")}
    ws = torch.empty(cl.collider_residual_norm_bwd_workspace_size(d), dtype=torch.uint8, device=gu.DEV)
    sv = cl.residual_norm_saved(x=t["x"], y=t["y"], h=t["h"], rstd_y=gu.f32(st["rstd_y"]), rstd_h=gu.f32(st["rstd_h"]))
    cl.collider_residual_norm_bwd(d, c.params, sv, 0, t["da"], t["dh"], 0, gu.i32(idx),
                                  gu.i32(np.concatenate([[0], np.cumsum(c.keep.sum(1))])), gu.i32([km.size]),
                                  cl.residual_norm_grads(dx=t["dx"], dy=t["dy"], **G), 0, ws)
    cl.collider_check()
    for k in ("dx", "dy"):
        assert torch.equal(t[k], want_b[k]), k
    for k in G:
        assert torch.equal(G[k], want_b[k]), k


@pytest.mark.parametrize("ln", [False, True])
def test_many_rows(ln):
    """A sequence of 300001 tokens: column sums of some 180000 rows."""
    c = Case(1, 300001, 8, "f32", ln, gate=1, res=True)
    c.check_forward(c.forward())
    c.check_backward()


# --------------------------------------------------------------------------
# a sandwich-normed branch: pre norm, linear branch, join; the checkpoints of its forward; its backward
# --------------------------------------------------------------------------
class Branch:
    """x -> a = norm(x) -> y = a W -> (h, a2) = join(x, y); a, y and h kept in 8 bits, the kept rows only."""

    def __init__(self, B=2, T=200, D=256, fmt="e4m3", seed=0):
        self.B, self.T, self.D, self.M, self.fmt = B, T, D, B * T, fmt
        rng = np.random.default_rng(seed)
        g = lambda *s, std=1.0, mean=0.0: workloads.bf16_representable(mean + std * rng.normal(size=s))  # noqa: E731
        self.host = dict(x=g(self.M, D), w=g(D, D, std=0.05), w0=g(D, std=0.1, mean=1), post_w=g(D, std=0.1, mean=1),
                         pre_w=g(D, std=0.1, mean=1), gate=g(1, D, std=0.1, mean=0.4), da2=g(self.M, D), dh=g(self.M, D))
        self.t = {k: gu.bf16(v) for k, v in self.host.items()}
        self.keep = workloads.gumbel_keep_mask(B, T, 0.4, seed=7)
        self.idx, self.cu, self.nk = gu.compact(self.keep)
        mk = dict(dtype=cl.BF16, B=B, T=T, D=D, norm=cl.NORM_RMS, eps=EPS, res_scale=1.0)
        self.d0 = cl.ResidualNormDesc(post=0, pre=1, gate_rows=0, **mk)
        self.d1 = cl.ResidualNormDesc(post=1, pre=1, gate_rows=1, **mk)
        self.p0 = cl.residual_norm_params(pre_w=self.t["w0"])
        self.p1 = cl.residual_norm_params(post_w=self.t["post_w"], gate=self.t["gate"], pre_w=self.t["pre_w"])
        e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=gu.DEV)  # noqa: E731
        M = self.M
        self.b = {k: e(M, D) for k in ("a", "y", "h", "a2", "dx_res", "dy", "da", "dx")}
        self.b.update({k: e(M, dt=torch.float32) for k in ("r0", "ry", "rh")})
        self.b.update({k: e(D, dt=torch.float32) for k in ("dpost_w", "dpre_w", "dw0")})
        self.b.update(dgate=e(1, D, dt=torch.float32), dw=e(D, D, dt=torch.float32))
        self.ck = {k: cl.ckpt(FMT[fmt], e(M, D, dt=torch.uint8), e(M, D // 32, dt=torch.uint8)) for k in ("x", "a", "y", "h")}
        self.ws = e(max(cl.collider_residual_norm_bwd_workspace_size(self.d1),
                        cl.collider_linear_ckpt_workspace_size(M, D, D)), dt=torch.uint8)

    def step(self):
        b, t, M, D, C = self.b, self.t, self.M, self.D, cl.ROWS_COMPACT
        cl.collider_residual_norm_fwd(self.d0, self.p0, t["x"], None, cl.residual_norm_out(a=b["a"], rstd_h=b["r0"]))
        torch.matmul(b["a"], t["w"], out=b["y"])
        cl.collider_residual_norm_fwd(self.d1, self.p1, t["x"], b["y"],
                                      cl.residual_norm_out(h=b["h"], a=b["a2"], rstd_y=b["ry"], rstd_h=b["rh"]))
        for k, v in (("x", t["x"]), ("a", b["a"]), ("y", b["y"]), ("h", b["h"])):
            cl.collider_ckpt_pack(cl.BF16, v, D, M, D, self.idx, self.nk, self.ck[k])
        index = (self.idx, self.cu, self.nk)
        cl.collider_residual_norm_bwd(
            self.d1, self.p1, cl.residual_norm_saved(y_ckpt=self.ck["y"], h_ckpt=self.ck["h"], rstd_y=b["ry"], rstd_h=b["rh"]),
            C, t["da2"], t["dh"], 0, *index,
            cl.residual_norm_grads(dx=b["dx_res"], dy=b["dy"], dpost_w=b["dpost_w"], dgate=b["dgate"], dpre_w=b["dpre_w"]), C,
            self.ws)
        cl.collider_linear_bwd_ckpt(M, D, D, self.ck["a"], C, t["w"], b["dy"], C, self.idx, self.nk, b["da"], C, b["dw"], None,
                                    self.ws)
        cl.collider_residual_norm_bwd(
            self.d0, self.p0, cl.residual_norm_saved(h_ckpt=self.ck["x"], rstd_h=b["r0"]), C, b["da"], b["dx_res"], C, *index,
            cl.residual_norm_grads(dx=b["dx"], dpre_w=b["dw0"]), 0, self.ws)

    OUT = ("dx", "dw", "dw0", "dpost_w", "dgate", "dpre_w")

    def reference(self):
        """The same chain in float64, from the GPU's saved values."""
        h, fmt, km = self.host, self.fmt, np.flatnonzero(self.keep.reshape(-1))
        deq = {}
        for k, src in (("x", self.t["x"]), ("a", self.b["a"]), ("y", self.b["y"]), ("h", self.b["h"])):
            deq[k] = ock.unpack(*ock.pack(gu.host(src), fmt), fmt)
        z = np.zeros(self.M)
        f64 = {k: np.asarray(v, np.float64) for k, v in h.items()}
        p1 = dict(post_w=f64["post_w"], post_b=None, gate=f64["gate"], res_w=None, pre_w=f64["pre_w"], pre_b=None)
        st = dict(mean_y=z, mean_h=z, rstd_y=gu.host(self.b["ry"]), rstd_h=gu.host(self.b["rh"]))
        g1, _ = oj.join_backward(None, deq["y"], deq["h"], st, f64["da2"], f64["dh"], p1, self.B, self.T, self.keep, 1.0, False)
        dw = deq["a"][km].T @ g1["dy"][km]
        da = g1["dy"] @ f64["w"].T
        p0 = dict(post_w=None, post_b=None, gate=None, res_w=None, pre_w=f64["w0"], pre_b=None)
        g0, _ = oj.join_backward(None, None, deq["x"], dict(mean_h=z, rstd_h=gu.host(self.b["r0"])), da, g1["dx"], p0, self.B,
                                 self.T, self.keep, 1.0, False)
        return dict(dx=g0["dx"], dw=dw, dw0=g0["dpre_w"], dpost_w=g1["dpost_w"], dgate=g1["dgate"], dpre_w=g1["dpre_w"])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_branch_through_the_operators(fmt):
    br = Branch(fmt=fmt)
    br.step()
    cl.collider_check()
    ref = br.reference()
    for k in br.OUT:   # at most three bf16 roundings (2^-8 each) on the way: within 2e-2 of the largest value
        assert gu.rel_err(gu.host(br.b[k]), ref[k]) <= 2e-2, k


def test_a_branch_in_graphs_that_share_a_workspace():
    """Two captured branches with one workspace, replayed in turn with new inputs, give what eager calls give."""
    one, two = Branch(seed=1), Branch(seed=2)
    two.ws = one.ws
    want = []
    for br in (one, two):
        br.step()                      # (the first call on a device allocates: before any capture)
        torch.cuda.synchronize()
        want.append({k: br.b[k].clone() for k in br.OUT})
    graphs = []
    for br in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            br.step()
        graphs.append(g)
    for _ in range(2):
        for br in (one, two):
            for k in br.OUT:
                br.b[k].fill_(9)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        cl.collider_check()
        for br, w in zip((one, two), want):
            for k in br.OUT:
                assert torch.equal(br.b[k], w[k]), k
    one.t["dh"].zero_()                # new inputs in the captured buffers
    graphs[0].replay()
    torch.cuda.synchronize()
    got = {k: one.b[k].clone() for k in one.OUT}
    one.step()
    torch.cuda.synchronize()
    for k in one.OUT:
        assert torch.equal(one.b[k], got[k]), k
