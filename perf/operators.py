"""What is measured of the checkpoint and residual-norm operators of libcollider.

Five operators of a filtered training step (every call below works on the kept
tokens of B sequences of T tokens, token t of sequence b being row b*T + t):

  join_fwd  the residual join: h = alpha*x + gate * post(y) and a = pre(h), the
            norm after a block's branch, its gate, the residual scale and the
            norm before the next branch
  join_bwd  its backward on the kept rows, the saved y and h in bf16 / f32 or as
            8-bit checkpoints
  pack      rows of activations -> 8-bit checkpoint (one code a value, one
            power-of-two exponent for each 32 values of a row)
  unpack    8-bit checkpoint -> rows
  linear    backward of a linear layer whose input was saved in 8 bits
"""
import math

import torch

own = False

DEV = "cuda:0"
GROUP = 32           # values that share an exponent
E_MIN = -120         # the smallest exponent a group is given
LIMIT = {"e4m3": 448.0, "int8": 127.0}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _join(name, op, B, T, D, **kw):
    c = dict(name=name, op=op, B=B, T=T, D=D, dtype="bf16", norm="rms", gate="channel", res="none", alpha=1.0,
             f=0.0, saved="same")
    c.update(kw)
    return c


def listed():
    return [
        # one token of a 2048-wide block: nothing but latency
        _join("join_fwd token", "join_fwd", 1, 1, 2048),
        # the forward of a TinyLlama-shaped block's join, batch 4 x 2048
        _join("join_fwd 4x2048x2048", "join_fwd", 4, 2048, 2048),
        # LayerNorms in f32, a gate row for each sequence, ragged length
        _join("join_fwd ln f32 3x333x1536", "join_fwd", 3, 333, 1536, dtype="f32", norm="ln", gate="sequence",
              alpha=0.5),
        # a short f32 sequence with a learned residual scale, 40% filtered
        _join("join_bwd ln f32 1x128x256", "join_bwd", 1, 128, 256, dtype="f32", norm="ln", res="channel", f=0.4),
        # the backward of the TinyLlama-shaped join, 40% filtered
        _join("join_bwd 4x2048x2048", "join_bwd", 4, 2048, 2048, f=0.4),
        # Qwen2.5-shaped, y and h from 8-bit checkpoints, a gate row a sequence
        _join("join_bwd e4m3 2x4096x1536", "join_bwd", 2, 4096, 1536, f=0.4, saved="e4m3", gate="sequence"),
        # a small checkpoint of every row
        dict(name="pack int8 1x128x256", op="pack", B=1, T=128, N=256, dtype="bf16", fmt="int8", f=0.0),
        # the MLP's [gate | up] activations of a TinyLlama-shaped block, the kept rows only
        dict(name="pack e4m3 4x2048x11264", op="pack", B=4, T=2048, N=11264, dtype="bf16", fmt="e4m3", f=0.4),
        # a kept-rows checkpoint spread over its full rows, ragged length
        dict(name="unpack int8 3x1001x1536", op="unpack", B=3, T=1001, N=1536, dtype="bf16", fmt="int8", f=0.2,
             src="compact", dst="full"),
        # the kept rows of the [gate | up] checkpoint, for the backward's GEMMs
        dict(name="unpack e4m3 4x2048x11264", op="unpack", B=4, T=2048, N=11264, dtype="bf16", fmt="e4m3", f=0.4,
             src="full", dst="compact"),
        # the smallest linear layer of the repository's workloads
        dict(name="linear e4m3 128x256x256", op="linear", B=1, T=128, K=256, N=256, fmt="e4m3", f=0.4, bias=True,
             src="full"),
        # the MLP down-projection of a TinyLlama-shaped block, 40% filtered
        dict(name="linear e4m3 8192x5632x2048", op="linear", B=4, T=2048, K=5632, N=2048, fmt="e4m3", f=0.4,
             bias=False, src="full"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["join_fwd", "join_bwd", "pack", "unpack", "linear"])
    f = rng.choice([0.0, 0.2, 0.4, 0.6])
    B = rng.randint(1, 4)
    T = _log(rng, 1, 2048)
    if op in ("join_fwd", "join_bwd"):
        saved = rng.choice(["same", "e4m3", "int8"]) if op == "join_bwd" else "same"
        D = 32 * _log(rng, 2, 64) if saved != "same" else 8 * _log(rng, 8, 256)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            T = max(1, T // 2)
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, norm=rng.choice(["rms", "ln"]),
                    gate=rng.choice(["none", "channel", "sequence"]), res=rng.choice(["none", "channel"]),
                    alpha=rng.choice([1.0, 0.5, 1.25]), f=f if op == "join_bwd" else 0.0, saved=saved)
    if op in ("pack", "unpack"):
        c = dict(op=op, B=B, T=T, N=32 * _log(rng, 2, 350), dtype=rng.choice(["bf16", "bf16", "f32"]),
                 fmt=rng.choice(["e4m3", "int8"]), f=f)
        if c["dtype"] == "f32":
            c["T"] = max(1, T // 2)
        if op == "unpack":
            c.update(src=rng.choice(["full", "compact"]), dst=rng.choice(["full", "compact"]))
        return c
    return dict(op=op, B=B, T=T, K=32 * _log(rng, 2, 128), N=8 * _log(rng, 8, 256), fmt=rng.choice(["e4m3", "int8"]),
                f=f, bias=rng.choice([True, False]), src=rng.choice(["full", "compact"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _kept(case):
    """Kept tokens of each sequence."""
    return case["T"] - int(math.floor(case["f"] * case["T"] + 1e-9))


def _index(case, g):
    """The ascending index list of the kept rows (every sequence drops its floor(f*T) lowest scores)."""
    B, T, k = case["B"], case["T"], _kept(case)
    score = torch.rand(B, T, generator=g, device=DEV)
    rows = score.topk(k, dim=1).indices.sort(dim=1).values + torch.arange(B, device=DEV)[:, None] * T
    return rows.reshape(-1)


def _activations(shape, g, dt, std=1.0):
    """Normal values with a few wide channels, as residual streams have."""
    v = torch.randn(shape, generator=g, device=DEV) * std
    wide = torch.rand(shape[-1], generator=g, device=DEV) < 0.01
    return (v * torch.where(wide, 12.0, 1.0)).to(dt)


def _saved8(s, key, v, fmt, rows=None):
    """Checkpoint of v (of its rows `rows` alone, in a buffer with room for all of them)."""
    code, exps = _pack(v if rows is None else v[rows], fmt)
    if rows is not None:
        full = torch.zeros(v.shape, dtype=torch.uint8, device=DEV)
        fexp = torch.zeros(v.shape[0], v.shape[1] // GROUP, dtype=torch.uint8, device=DEV)
        full[: code.shape[0]], fexp[: code.shape[0]] = code, exps
        code, exps = full, fexp
    s[key], s[key + "_exps"] = code, exps


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    B, T, op = case["B"], case["T"], case["op"]
    M = B * T
    rows = _index(case, g)
    s = dict(case=dict(case), M=M, n=rows.numel(), rows=rows, idx=torch.zeros(M, dtype=torch.int32, device=DEV),
             nk=torch.tensor([rows.numel()], dtype=torch.int32, device=DEV))
    s["idx"][: rows.numel()] = rows.to(torch.int32)
    s["cu"] = (torch.arange(B + 1, device=DEV) * _kept(case)).to(torch.int32)
    new = lambda *shape, dt=torch.float32: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
    if op in ("join_fwd", "join_bwd"):
        dt, D = _dtype(case), case["D"]
        par = lambda n, mean, std: (torch.randn(n, D, generator=g, device=DEV) * std + mean).to(dt)  # noqa: E731
        s["x"] = _activations((M, D), g, dt)
        s["y"] = _activations((M, D), g, dt, 0.3)
        s["post_w"], s["pre_w"] = par(1, 1.0, 0.1)[0], par(1, 1.0, 0.1)[0]
        s["gate"] = None if case["gate"] == "none" else par(1 if case["gate"] == "channel" else B, 0.3, 0.1)
        s["res_w"] = par(1, 1.0, 0.1)[0] if case["res"] == "channel" else None
        ln = case["norm"] == "ln"
        s["post_b"], s["pre_b"] = (par(1, 0.0, 0.1)[0], par(1, 0.0, 0.1)[0]) if ln else (None, None)
        stats = ("mean_y", "rstd_y", "mean_h", "rstd_h") if ln else ("rstd_y", "rstd_h")
        if op == "join_fwd":
            s["h"], s["a"] = new(M, D, dt=dt), new(M, D, dt=dt)
            s.update({k: new(M) for k in stats})
            return s
        s.update(_join_fwd(s))
        s["da"] = (torch.randn(M, D, generator=g, device=DEV) * 0.05).to(dt)
        s["dh"] = (torch.randn(M, D, generator=g, device=DEV) * 0.05).to(dt)
        del s["a"]
        if case["saved"] != "same":
            _saved8(s, "y", s["y"].float(), case["saved"])
            _saved8(s, "h", s["h"].float(), case["saved"])
        s["dx"], s["dy"] = new(M, D, dt=dt), new(M, D, dt=dt)
        s["dpost_w"], s["dpre_w"] = new(D), new(D)
        s["dgate"] = None if s["gate"] is None else new(*s["gate"].shape)
        s["dres_w"] = None if s["res_w"] is None else new(D)
        s["dpost_b"], s["dpre_b"] = (new(D), new(D)) if ln else (None, None)
        return s
    if op == "pack":
        s["v"] = _activations((M, case["N"]), g, _dtype(case))
        s["code"] = new(M, case["N"], dt=torch.uint8)
        s["exps"] = new(M, case["N"] // GROUP, dt=torch.uint8)
        return s
    if op == "unpack":
        v = _activations((M, case["N"]), g, _dtype(case)).float()
        _saved8(s, "code", v, case["fmt"], rows if case["src"] == "compact" else None)
        s["out"] = new(M, case["N"], dt=_dtype(case))
        return s
    K, N, bf = case["K"], case["N"], torch.bfloat16
    x = _activations((M, K), g, bf).float()
    _saved8(s, "x", x, case["fmt"], rows if case["src"] == "compact" else None)
    s["w"] = (torch.randn(K, N, generator=g, device=DEV) * 0.02).to(bf)
    s["dy"] = torch.randn(M, N, generator=g, device=DEV).to(bf)
    s["dx"], s["dw"] = new(M, K, dt=bf), new(K, N)
    s["db"] = new(N) if case["bias"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _pack(v, fmt):
    """Codes and exponent bytes of [rows, N] values: a group's exponent is the smallest e >= E_MIN with
    |v| <= LIMIT * 2^e over its 32 values, a code is the nearest 8-bit value to v * 2^-e (ties to even), the
    byte is e + 127; a group that holds a NaN or an infinity has byte 255 and codes 0."""
    n, N = v.shape
    g = v.float().reshape(n, N // GROUP, GROUP)
    big = g.abs().amax(-1)
    fine = torch.isfinite(big)
    m, e = torch.frexp(torch.where(fine, big, 0.0))
    top, bits = (0.875, 9) if fmt == "e4m3" else (127 / 128, 7)
    e = (e - bits + (m > top).int()).clamp_min(E_MIN)
    e = torch.where(big > 0, e, E_MIN)
    q = torch.where(fine[..., None], g * torch.exp2(-e.float())[..., None], 0.0)
    code = q.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else q.round().to(torch.int8).view(torch.uint8)
    return code.reshape(n, N), torch.where(fine, e + 127, 255).to(torch.uint8)


def _unpack(code, exps, fmt):
    """The f32 values of a checkpoint."""
    v = code.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()
    scale = torch.where(exps == 255, math.nan, torch.exp2(exps.float() - 127))
    return v * scale.repeat_interleave(GROUP, dim=1)


def _f(v):
    return None if v is None else v.float()


def _stats(v, ln, eps):
    if ln:
        mean = v.mean(-1)
        return mean, 1.0 / torch.sqrt((v - mean[:, None]).square().mean(-1) + eps)
    return None, 1.0 / torch.sqrt(v.square().mean(-1) + eps)


EPS = 1e-5


def _hat(v, mean, rstd):
    return (v if mean is None else v - mean[:, None]) * rstd[:, None]


def _affine(v, w, b):
    return v * w if b is None else v * w + b


def _gate_rows(s, rows):
    """The gate of each of `rows` (tokens), or 1."""
    g = _f(s["gate"])
    return 1.0 if g is None else g[0] if g.shape[0] == 1 else g[rows // s["case"]["T"]]


def _join_fwd(s):
    c, dt = s["case"], s["x"].dtype
    ln = c["norm"] == "ln"
    x, y = s["x"].float(), s["y"].float()
    mean_y, rstd_y = _stats(y, ln, EPS)
    p = _affine(_hat(y, mean_y, rstd_y), _f(s["post_w"]), _f(s["post_b"]))
    res = x * c["alpha"] if s["res_w"] is None else x * c["alpha"] * _f(s["res_w"])
    h = (res + _gate_rows(s, torch.arange(s["M"], device=DEV)) * p).to(dt)
    mean_h, rstd_h = _stats(h.float(), ln, EPS)   # of h as it is stored
    a = _affine(_hat(h.float(), mean_h, rstd_h), _f(s["pre_w"]), _f(s["pre_b"])).to(dt)
    out = dict(h=h, a=a, rstd_y=rstd_y, rstd_h=rstd_h)
    if ln:
        out.update(mean_y=mean_y, mean_h=mean_h)
    return out


def _norm_bwd(d, hat, rstd, ln):
    """Gradient of a norm's input from that of its normalised output."""
    g = d - hat * (d * hat).mean(-1, keepdim=True)
    return (g - d.mean(-1, keepdim=True) if ln else g) * rstd[:, None]


def _join_bwd(s):
    c, rows, dt = s["case"], s["rows"], s["dx"].dtype
    ln = c["norm"] == "ln"
    pick = lambda v: None if v is None else v[rows].float()  # noqa: E731
    if c["saved"] == "same":
        y, h = pick(s["y"]), pick(s["h"])
    else:
        y = _unpack(s["y"][rows], s["y_exps"][rows], c["saved"])
        h = _unpack(s["h"][rows], s["h_exps"][rows], c["saved"])
    yh, hh = (_hat(v, pick(s.get("mean_" + k)), pick(s["rstd_" + k])) for v, k in ((y, "y"), (h, "h")))
    da = pick(s["da"])
    dh = pick(s["dh"]) + _norm_bwd(da * _f(s["pre_w"]), hh, pick(s["rstd_h"]), ln)
    u = _gate_rows(s, rows) * dh
    out = {k: torch.zeros_like(s["dx"]) for k in ("dx", "dy")}
    dx = dh * c["alpha"]
    out["dx"][rows] = (dx if s["res_w"] is None else dx * _f(s["res_w"])).to(dt)
    out["dy"][rows] = _norm_bwd(u * _f(s["post_w"]), yh, pick(s["rstd_y"]), ln).to(dt)
    out["dpre_w"], out["dpost_w"] = (da * hh).sum(0), (u * yh).sum(0)
    if ln:
        out["dpre_b"], out["dpost_b"] = da.sum(0), u.sum(0)
    if s["gate"] is not None:
        dg = dh * _affine(yh, _f(s["post_w"]), _f(s["post_b"]))
        out["dgate"] = dg.reshape(s["gate"].shape[0], -1, c["D"]).sum(1)   # every sequence keeps as many tokens
    if s["res_w"] is not None:
        out["dres_w"] = (dh * pick(s["x"]) * c["alpha"]).sum(0)
    return out


def _codes(code, exps, fmt):
    """A checkpoint as numbers: its codes as the 8-bit values they are, and its exponent bytes."""
    return dict(code=code.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8), exps=exps)


def _linear(s):
    c, rows = s["case"], s["rows"]
    at = rows if c["src"] == "full" else slice(0, s["n"])
    x, dy = _unpack(s["x"][at], s["x_exps"][at], c["fmt"]), s["dy"][rows].float()
    dx = torch.zeros_like(s["dx"])
    dx[rows] = (dy @ s["w"].float().T).to(dx.dtype)
    out = dict(dx=dx, dw=x.T @ dy)
    if c["bias"]:
        out["db"] = dy.sum(0)
    return out


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "join_fwd":
        return _join_fwd(s)
    if op == "join_bwd":
        return _join_bwd(s)
    if op == "pack":
        return _codes(*_pack(s["v"][s["rows"]], c["fmt"]), c["fmt"])
    if op == "unpack":
        at = s["rows"] if c["src"] == "full" else slice(0, s["n"])
        v = _unpack(s["code"][at], s["code_exps"][at], c["fmt"]).to(s["out"].dtype)
        if c["dst"] == "compact":
            return v
        out = torch.zeros_like(s["out"])
        out[s["rows"]] = v
        return out
    return _linear(s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _plan(s, cl):
    """The descriptors and workspaces a program keeps beside its buffers."""
    c, op = s["case"], s["case"]["op"]
    ckpt = lambda k, fmt: cl.ckpt(fmt, s[k], s[k + "_exps"])  # noqa: E731
    p = {}
    need = 0
    if op in ("join_fwd", "join_bwd"):
        gate = s["gate"]
        p["desc"] = cl.ResidualNormDesc(
            dtype=cl.F32 if c["dtype"] == "f32" else cl.BF16, B=c["B"], T=c["T"], D=c["D"],
            norm=cl.NORM_LAYER if c["norm"] == "ln" else cl.NORM_RMS, post=1, pre=1, eps=EPS, res_scale=c["alpha"],
            gate_rows=0 if gate is None else gate.shape[0])
        p["params"] = cl.residual_norm_params(**{k: s[k] for k in ("post_w", "post_b", "gate", "res_w", "pre_w",
                                                                  "pre_b")})
        if op == "join_bwd":
            eight = c["saved"] != "same"
            fmt = cl.CKPT_INT8 if c["saved"] == "int8" else cl.CKPT_E4M3
            p["saved"] = cl.residual_norm_saved(
                x=s["x"] if s["res_w"] is not None else None, y=None if eight else s["y"], h=None if eight else s["h"],
                y_ckpt=ckpt("y", fmt) if eight else None, h_ckpt=ckpt("h", fmt) if eight else None,
                mean_y=s.get("mean_y"), rstd_y=s["rstd_y"], mean_h=s.get("mean_h"), rstd_h=s["rstd_h"])
            p["grads"] = cl.residual_norm_grads(**{k: s[k] for k in ("dx", "dy", "dpost_w", "dpost_b", "dgate", "dres_w",
                                                                    "dpre_w", "dpre_b")})
            need = cl.collider_residual_norm_bwd_workspace_size(p["desc"])
        else:
            p["out"] = cl.residual_norm_out(**{k: s.get(k) for k in ("h", "a", "mean_y", "rstd_y", "mean_h", "rstd_h")})
    elif op == "pack":
        p["ckpt"] = cl.ckpt(cl.CKPT_INT8 if c["fmt"] == "int8" else cl.CKPT_E4M3, s["code"], s["exps"])
    elif op == "unpack":
        p["ckpt"] = ckpt("code", cl.CKPT_INT8 if c["fmt"] == "int8" else cl.CKPT_E4M3)
    else:
        p["ckpt"] = ckpt("x", cl.CKPT_INT8 if c["fmt"] == "int8" else cl.CKPT_E4M3)
        need = cl.collider_linear_ckpt_workspace_size(s["M"], c["K"], c["N"])
    p["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    return p


def _own(s):
    import sparse_backward_gemm_gb300 as cl
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s, cl)
    c, op, M, n = s["case"], s["case"]["op"], s["M"], s["n"]
    if op == "join_fwd":
        cl.collider_residual_norm_fwd(p["desc"], p["params"], s["x"], s["y"], p["out"])
        return {k: s[k] for k in ("h", "a", "rstd_y", "rstd_h", "mean_y", "mean_h") if s.get(k) is not None}
    if op == "join_bwd":
        idx, cu, nk = (s["idx"], s["cu"], s["nk"]) if c["f"] else (None, None, None)
        cl.collider_residual_norm_bwd(p["desc"], p["params"], p["saved"], cl.ROWS_FULL, s["da"], s["dh"], cl.ROWS_FULL,
                                      idx, cu, nk, p["grads"], cl.ROWS_FULL, p["ws"])
        return {k: s[k] for k in ("dx", "dy", "dpre_w", "dpost_w", "dpre_b", "dpost_b", "dgate", "dres_w")
                if s[k] is not None}
    idx, nk = (s["idx"], s["nk"]) if c["f"] else (None, None)
    dt = cl.F32 if c.get("dtype") == "f32" else cl.BF16
    side = lambda k: cl.ROWS_FULL if c[k] == "full" else cl.ROWS_COMPACT  # noqa: E731
    if op == "pack":
        cl.collider_ckpt_pack(dt, s["v"], c["N"], M, c["N"], idx, nk, p["ckpt"])
        return _codes(s["code"][:n], s["exps"][:n], c["fmt"])
    if op == "unpack":
        cl.collider_ckpt_unpack(dt, p["ckpt"], side("src"), M, c["N"], idx, nk, s["out"], c["N"], side("dst"))
        return s["out"] if c["dst"] == "full" else s["out"][:n]
    cl.collider_linear_bwd_ckpt(M, c["K"], c["N"], p["ckpt"], side("src"), s["w"], s["dy"], cl.ROWS_FULL, s["idx"], s["nk"],
                              s["dx"], cl.ROWS_FULL, s["dw"], s["db"], p["ws"])
    return {k: s[k] for k in ("dx", "dw", "db") if s[k] is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    op, M, n = case["op"], case["B"] * case["T"], case["B"] * _kept(case)
    e = 4 if case.get("dtype") == "f32" else 2
    if op in ("join_fwd", "join_bwd"):
        D = case["D"]
        stats = 16 if case["norm"] == "ln" else 8
        vecs = (2 + (1 if case["res"] == "channel" else 0) + (2 if case["norm"] == "ln" else 0)
                + {"none": 0, "channel": 1, "sequence": case["B"]}[case["gate"]])
        if op == "join_fwd":
            return dict(bytes=M * (4 * D * e + stats) + vecs * D * e, flops=20 * M * D)
        src = e if case["saved"] == "same" else 1 + 1 / GROUP
        x = e if case["res"] == "channel" else 0
        return dict(bytes=n * (D * (2 * e + 2 * src + x) + stats + 4) + 2 * M * D * e + vecs * D * (e + 4),
                    flops=35 * n * D)
    if op == "pack":
        return dict(bytes=n * case["N"] * (e + 1 + 1 / GROUP) + 4 * n, flops=4 * n * case["N"])
    if op == "unpack":
        out = M if case["dst"] == "full" else n
        return dict(bytes=n * case["N"] * (1 + 1 / GROUP) + out * case["N"] * e + 4 * n, flops=2 * n * case["N"])
    K, N = case["K"], case["N"]
    return dict(bytes=n * K * (1 + 1 / GROUP) + n * N * 2 + K * N * 2 + M * K * 2 + K * N * 4, flops=4 * n * K * N)


def _two64(e):
    """2^e in 64 bits for whole e within +-256, from a table of exact powers."""
    return torch.tensor([2.0 ** k for k in range(-256, 257)], dtype=torch.float64, device=DEV)[e.long() + 256]


def _values64(code, exps, fmt):
    """A checkpoint's values in 64 bits, from the bits of its codes."""
    c = code.to(torch.int64)
    if fmt == "int8":
        v = torch.where(c >= 128, c - 256, c).double()
    else:
        field, frac = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(field == 0, frac * 2.0 ** -9, (8 + frac) * _two64(field - 10))
        v = torch.where(c >= 128, -mag, mag)
    n, N = code.shape
    e = _two64(exps.long() - 127)
    e = torch.where(exps == 255, math.nan, e)
    return (v.reshape(n, N // GROUP, GROUP) * e[:, :, None]).reshape(n, N)


def _exact_pack(s):
    c = s["case"]
    v = s["v"][s["rows"]].double()
    n, N = v.shape
    g = v.reshape(n, -1, GROUP)
    m, e = torch.frexp(g.abs().amax(-1) / LIMIT[c["fmt"]])   # the ratio is m * 2^e, m in [0.5, 1)
    e = torch.where(m > 0.5, e, e - 1).clamp_min(E_MIN)
    q = g / _two64(e)[..., None]
    if c["fmt"] == "e4m3":
        step = _two64(torch.frexp(q).exponent.clamp(-5, 9) - 4)   # of a binade of 8 codes
        q = torch.round(q / step) * step
    else:
        q = torch.round(q)
    return dict(code=q.reshape(n, N), exps=e.double() + 127)


def _exact_join(s):
    c = s["case"]
    ln, T, D = c["norm"] == "ln", c["T"], c["D"]
    d = lambda k: None if s.get(k) is None else s[k].double()  # noqa: E731
    one = torch.ones((), dtype=torch.float64, device=DEV)
    lam = c["alpha"] * (one if s["res_w"] is None else d("res_w"))
    if c["op"] == "join_fwd":
        def norm(v, w, b):
            mu = v.sum(1, keepdim=True) / D if ln else torch.zeros(v.shape[0], 1, dtype=torch.float64, device=DEV)
            r = (((v - mu) ** 2).sum(1, keepdim=True) / D + EPS) ** -0.5
            return (v - mu) * r * w + (b if b is not None else 0.0), mu[:, 0], r[:, 0]
        p, my, ry = norm(d("y"), d("post_w"), d("post_b"))
        gate = d("gate")
        if gate is not None:
            p = (p.reshape(gate.shape[0], -1, D) * gate[:, None]).reshape(-1, D)
        h = lam * d("x") + p
        a, mh, rh = norm(h.to(s["x"].dtype).double(), d("pre_w"), d("pre_b"))
        out = dict(h=h, a=a, rstd_y=ry, rstd_h=rh)
        if ln:
            out.update(mean_y=my, mean_h=mh)
        return out
    rows = s["rows"]
    if c["saved"] == "same":
        y, h = d("y")[rows], d("h")[rows]
    else:
        y = _values64(s["y"], s["y_exps"], c["saved"])[rows]
        h = _values64(s["h"], s["h_exps"], c["saved"])[rows]
    zero = torch.zeros(s["M"], dtype=torch.float64, device=DEV)
    my, mh = (d("mean_y"), d("mean_h")) if ln else (zero, zero)
    ry, rh = d("rstd_y")[rows, None], d("rstd_h")[rows, None]
    yh, hh = (y - my[rows, None]) * ry, (h - mh[rows, None]) * rh

    def back(t, hat, r):
        # (I - hat hat^T / D [- 1 1^T / D]) t, times the reciprocal deviation
        out = t - hat * torch.einsum("rd,rd->r", t, hat)[:, None] / D
        if ln:
            out = out - t.sum(1, keepdim=True) / D
        return r * out
    da, dh = d("da")[rows], d("dh")[rows]
    dh = dh + back(da * d("pre_w"), hh, rh)
    B = c["B"]
    gate = d("gate")
    grow = torch.ones(B, D, dtype=torch.float64, device=DEV) if gate is None else gate.expand(B, D)
    by = lambda v: v.reshape(B, -1, D)  # noqa: E731
    u = (by(dh) * grow[:, None]).reshape(-1, D)
    full = lambda v: torch.zeros(s["M"], D, dtype=torch.float64, device=DEV).index_copy(0, rows, v)  # noqa: E731
    out = dict(dx=full(dh * lam), dy=full(back(u * d("post_w"), yh, ry)), dpre_w=torch.einsum("rd,rd->d", da, hh),
               dpost_w=torch.einsum("rd,rd->d", u, yh))
    if ln:
        out.update(dpre_b=da.sum(0), dpost_b=u.sum(0))
    if gate is not None:
        branch = yh * d("post_w") + (d("post_b") if ln else 0.0)
        dg = torch.einsum("brd,brd->bd", by(dh), by(branch))
        out["dgate"] = dg if gate.shape[0] > 1 or B == 1 else dg.sum(0, keepdim=True)
    if s["res_w"] is not None:
        out["dres_w"] = c["alpha"] * torch.einsum("rd,rd->d", dh, d("x")[rows])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("join_fwd", "join_bwd"):
        return _exact_join(s)
    if op == "pack":
        return _exact_pack(s)
    n, rows = s["n"], s["rows"]
    if op == "unpack":
        v = _values64(s["code"], s["code_exps"], c["fmt"])
        v = v[rows] if c["src"] == "full" else v[:n]
        if c["dst"] == "compact":
            return v
        return torch.zeros(s["M"], c["N"], dtype=torch.float64, device=DEV).index_copy(0, rows, v)
    x = _values64(s["x"], s["x_exps"], c["fmt"])
    x = x[rows] if c["src"] == "full" else x[:n]
    dy = s["dy"].double()[rows]
    dx = torch.einsum("rn,kn->rk", dy, s["w"].double())
    out = dict(dx=torch.zeros(s["M"], c["K"], dtype=torch.float64, device=DEV).index_copy(0, rows, dx),
               dw=torch.einsum("rk,rn->kn", x, dy))
    if c["bias"]:
        out["db"] = dy.sum(0)
    return out
