"""What is measured of the gated feed-forward block and of gradient clipping.

Four operators of a training step (M = B*T tokens, token t of sequence b being
row b*T + t):

  ffn_fwd    the gated feed-forward block: [g | u] = x W_up, s = act(g) * u,
             y = s W_down, with [g | u] saved for the backward
  ffn_bwd    its backward on the kept tokens: the gradients of x, W_up and W_down
  grad_norm  the norm of a list of gradients, and each one's own
  grad_clip  the same, and the gradients scaled in place so that the norm is at
             most max_norm
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6   # of the clipping coefficient's denominator


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _ffn(name, op, B, T, D, F, act="silu", f=0.0, src="full", dst="full"):
    """src: the rows x, [g | u] and dy are given as; dst: the rows dx is wanted as."""
    c = dict(name=name, op=op, B=B, T=T, D=D, F=F, act=act)
    if op == "ffn_bwd":
        c.update(f=f, src=src, dst=dst)
    return c


def _grads(name, op, L, D, F, kv, V, dtype="f32", kind="l2", gap=0, scale=1.0):
    """The gradients of L blocks (V: and of the embedding, final norm and head); gap: values between two tensors
    of the buffer that holds them."""
    return dict(name=name, op=op, L=L, D=D, F=F, kv=kv, V=V, dtype=dtype, kind=kind, gap=gap, scale=scale)


def listed():
    return [
        # one token through a TinyLlama-shaped block's MLP: the weights are read once, nothing else counts
        _ffn("ffn_fwd token", "ffn_fwd", 1, 1, 2048, 5632),
        # a short sequence through the smallest block of the repository's tests: latency
        _ffn("ffn_fwd 192x256x384", "ffn_fwd", 2, 96, 256, 384, act="gelu_tanh"),
        # the MLP of a TinyLlama-shaped block, batch 4 x 2048
        _ffn("ffn_fwd 8192x2048x5632", "ffn_fwd", 4, 2048, 2048, 5632),
        # Qwen2.5-shaped, ragged length
        _ffn("ffn_fwd 3003x1536x8960", "ffn_fwd", 3, 1001, 1536, 8960),
        # the smallest block's backward, 40% filtered: latency
        _ffn("ffn_bwd 192x256x384", "ffn_bwd", 2, 96, 256, 384, act="gelu_tanh", f=0.4),
        # the TinyLlama-shaped MLP's backward, 40% filtered
        _ffn("ffn_bwd 8192x2048x5632", "ffn_bwd", 4, 2048, 2048, 5632, f=0.4),
        # the same MLP unfiltered at half the batch
        _ffn("ffn_bwd dense 4096x2048x5632", "ffn_bwd", 2, 2048, 2048, 5632),
        # Qwen2.5-shaped, ragged length, rows that a filtered block hands on compact, 20% filtered
        _ffn("ffn_bwd compact 3003x1536x8960", "ffn_bwd", 3, 1001, 1536, 8960, f=0.2, src="compact", dst="compact"),
        # the gradients of one small block: latency
        _grads("grad_norm small block", "grad_norm", 1, 256, 384, 128, 0, scale=0.25),
        # the gradients of one TinyLlama-shaped block
        _grads("grad_clip block", "grad_clip", 1, 2048, 5632, 256, 0),
        # the gradients of the whole 22-block stack with its embedding and head: 1.1 G values in 135 tensors
        _grads("grad_clip stack", "grad_clip", 22, 2048, 5632, 256, 32000),
        # a Qwen2.5-shaped block's gradients in bf16 at odd addresses, the largest value as the norm
        _grads("grad_clip max bf16", "grad_clip", 1, 1536, 8960, 256, 0, dtype="bf16", kind="max", gap=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_bwd", "ffn_bwd", "grad_norm", "grad_clip"])
    if op in ("ffn_fwd", "ffn_bwd"):
        c = dict(op=op, B=rng.randint(1, 4), T=_log(rng, 1, 2048), D=8 * _log(rng, 8, 256), F=8 * _log(rng, 16, 704),
                 act=rng.choice(["silu", "gelu_tanh"]))
        if op == "ffn_bwd":
            rows = rng.choice(["full", "full", "compact"])
            c.update(f=rng.choice([0.0, 0.2, 0.4, 0.6]), src=rows, dst=rng.choice(["full", rows]))
        return c
    D = 8 * _log(rng, 8, 256)
    return dict(op=op, L=_log(rng, 1, 22), D=D, F=8 * _log(rng, 16, 704), kv=64 * rng.randint(1, 4),
                V=rng.choice([0, _log(rng, 500, 32000)]), dtype=rng.choice(["f32", "f32", "bf16", "mixed"]),
                kind=rng.choice(["l2", "l2", "max"]), gap=rng.choice([0, 0, 1, 3]),
                scale=rng.choice([1.0, 0.125]) if op == "grad_norm" else 1.0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _kept(case):
    """Kept tokens of each sequence."""
    return case["T"] - int(math.floor(case.get("f", 0.0) * case["T"] + 1e-9))


def _index(case, g):
    """The ascending index list of the kept rows (every sequence drops its floor(f*T) lowest scores)."""
    B, T, k = case["B"], case["T"], _kept(case)
    score = torch.rand(B, T, generator=g, device=DEV)
    rows = score.topk(k, dim=1).indices.sort(dim=1).values + torch.arange(B, device=DEV)[:, None] * T
    return rows.reshape(-1)


def _normed(shape, g):
    """Rows as a block's norm hands them on: normal values with a few wide channels."""
    v = torch.randn(shape, generator=g, device=DEV)
    wide = torch.rand(shape[-1], generator=g, device=DEV) < 0.01
    return (v * torch.where(wide, 3.0, 1.0)).to(torch.bfloat16)


def _sizes(case):
    """Values of each gradient, in the order of the parameters."""
    D, F, kv, V = case["D"], case["F"], case["kv"], case["V"]
    block = [D, D * (D + 2 * kv), D * D, D, 2 * D * F, F * D]
    return ([V * D] if V else []) + block * case["L"] + ([D, D * V] if V else [])


def _prepare_ffn(case, g):
    M, D, F, bf = case["B"] * case["T"], case["D"], case["F"], torch.bfloat16
    rows = _index(case, g)
    new = lambda *shape: torch.empty(shape, dtype=bf, device=DEV)  # noqa: E731
    s = dict(case=dict(case), M=M, n=rows.numel(), rows=rows)
    s["x"] = _normed((M, D), g)
    s["w_up"] = (torch.randn(D, 2 * F, generator=g, device=DEV) * D ** -0.5).to(bf)
    s["w_down"] = (torch.randn(F, D, generator=g, device=DEV) * F ** -0.5).to(bf)
    if case["op"] == "ffn_fwd":
        s["up"], s["y"] = new(M, 2 * F), new(M, D)
        return s
    s["up"] = s["x"] @ s["w_up"]
    s["dy"] = (torch.randn(M, D, generator=g, device=DEV) * 0.05).to(bf)
    if case["src"] == "compact":
        s.update({k: s[k][rows] for k in ("x", "up", "dy")})
    s["dx"] = new(M, D)
    s["dw_up"], s["dw_down"] = new(D, 2 * F), new(F, D)
    s["idx"] = torch.zeros(M, dtype=torch.int32, device=DEV)
    s["idx"][: rows.numel()] = rows.to(torch.int32)
    s["nk"] = torch.tensor([rows.numel()], dtype=torch.int32, device=DEV)
    return s


def _prepare_grads(case, g):
    """Every tensor is a part of a flat buffer of its type; the values of different tensors differ in size by up to a hundred."""
    sizes, s = _sizes(case), dict(case=dict(case))
    types = [torch.bfloat16 if case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 2) else torch.float32
             for i in range(len(sizes))]
    s["flat"], s["grads"] = {}, [None] * len(sizes)
    for dt, key in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        mine = [i for i, t in enumerate(types) if t == dt]
        if not mine:
            continue
        flat = torch.randn(sum(sizes[i] + case["gap"] for i in mine), generator=g, device=DEV, dtype=dt)
        at = case["gap"]
        for i in mine:
            s["grads"][i] = flat[at: at + sizes[i]]
            s["grads"][i] *= 10.0 ** (-2 - 2 * ((i * 7) % 11) / 10)
            at += sizes[i] + case["gap"]
        s["flat"][key] = flat
    s["norm"], s["coef"] = (torch.empty(1, device=DEV) for _ in range(2))
    s["norms"] = torch.empty(len(sizes), device=DEV)
    s["max_norm"] = 1.0 if case["kind"] == "l2" else 0.01
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    return _prepare_ffn(case, g) if case["op"].startswith("ffn") else _prepare_grads(case, g)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
C1, C3 = math.sqrt(2 / math.pi), 0.044715


def _act(g, act):
    """The activation of the gate and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    t = torch.tanh(C1 * (g + C3 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * C1 * (1 + 3 * C3 * g * g)


def _ffn_fwd(s):
    F, dt = s["case"]["F"], s["x"].dtype
    up = s["x"].float() @ s["w_up"].float()
    y = (_act(up[:, :F], s["case"]["act"])[0] * up[:, F:]) @ s["w_down"].float()
    return dict(up=up.to(dt), y=y.to(dt))


def _ffn_bwd(s):
    c, F, dt = s["case"], s["case"]["F"], s["x"].dtype
    pick = lambda k: (s[k][s["rows"]] if c["src"] == "full" else s[k]).float()  # noqa: E731
    x, up, dy = pick("x"), pick("up"), pick("dy")
    a, da = _act(up[:, :F], c["act"])
    ds = dy @ s["w_down"].float().T
    dup = torch.cat((ds * up[:, F:] * da, ds * a), 1)
    dx = (dup @ s["w_up"].float().T).to(dt)
    if c["dst"] == "full":
        dx = torch.zeros(s["M"], c["D"], dtype=dt, device=DEV).index_copy_(0, s["rows"], dx)
    return dict(dx=dx, dw_up=(x.T @ dup).to(dt), dw_down=((a * up[:, F:]).T @ dy).to(dt))


def _grad_norm(s):
    c = s["case"]
    if c["kind"] == "max":
        norms = torch.stack([g.abs().amax().float() for g in s["grads"]]) * c["scale"]
        return norms, norms.amax(0, keepdim=True)
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    return (squares.sqrt() * c["scale"]).float(), (squares.sum(0, keepdim=True).sqrt() * c["scale"]).float()


def _grad_clip(s):
    norms, norm = _grad_norm(s)
    coef = s["case"]["scale"] * torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    for g in s["grads"]:
        g.copy_(g.float() * coef)
    return dict(s["flat"], norm=norm, norms=norms, coef=coef)


def _plain(s):
    op = s["case"]["op"]
    if op == "grad_norm":
        norms, norm = _grad_norm(s)
        return dict(norm=norm, norms=norms)
    return {"ffn_fwd": _ffn_fwd, "ffn_bwd": _ffn_bwd, "grad_clip": _grad_clip}[op](s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _plan(s, cl):
    """The descriptors, lists and workspaces a program keeps beside its buffers."""
    c, op, p = s["case"], s["case"]["op"], {}
    if op.startswith("ffn"):
        p["desc"] = cl.FfnDesc(M=s["M"], D=c["D"], F=c["F"], act=cl.GLU_SILU if c["act"] == "silu" else cl.GLU_GELU_TANH,
                               grad_dtype=cl.BF16)
        size = cl.collider_ffn_fwd_workspace_size if op == "ffn_fwd" else cl.collider_ffn_bwd_workspace_size
        need = size(p["desc"])
    else:
        p["list"] = cl.grad_list(s["grads"])
        p["kind"] = cl.GRAD_NORM_MAX if c["kind"] == "max" else cl.GRAD_NORM_L2
        need = cl.collider_grad_norm_workspace_size(p["list"], len(s["grads"]))
    p["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    return p


def _own(s):
    import sparse_backward_gemm_gb300 as cl
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s, cl)
    c, op = s["case"], s["case"]["op"]
    if op == "ffn_fwd":
        cl.collider_ffn_fwd(p["desc"], s["x"], s["w_up"], s["w_down"], s["up"], s["y"], p["ws"])
        return dict(up=s["up"], y=s["y"])
    if op == "ffn_bwd":
        rows = lambda k: cl.ROWS_FULL if c[k] == "full" else cl.ROWS_COMPACT  # noqa: E731
        idx, nk = (s["idx"], s["nk"]) if c["f"] else (None, None)
        cl.collider_ffn_bwd(p["desc"], s["w_up"], s["w_down"], s["x"], s["up"], rows("src"), s["dy"], rows("src"), idx, nk,
                            s["dx"], rows("dst"), s["dw_up"], s["dw_down"], p["ws"])
        return dict(dx=s["dx"] if c["dst"] == "full" else s["dx"][: s["n"]], dw_up=s["dw_up"], dw_down=s["dw_down"])
    if op == "grad_norm":
        cl.collider_grad_norm(p["list"], len(s["grads"]), p["kind"], c["scale"], s["norm"], s["norms"], p["ws"])
        return dict(norm=s["norm"], norms=s["norms"])
    cl.collider_grad_clip(p["list"], len(s["grads"]), p["kind"], c["scale"], s["max_norm"], s["norm"], s["norms"], s["coef"],
                          p["ws"])
    return dict(s["flat"], norm=s["norm"], norms=s["norms"], coef=s["coef"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op.startswith("ffn"):
        M, D, F = case["B"] * case["T"], case["D"], case["F"]
        if op == "ffn_fwd":
            return dict(bytes=2 * (2 * M * D + 2 * M * F + 3 * D * F), flops=6 * M * D * F)
        n = case["B"] * _kept(case)
        out = M if case["dst"] == "full" else n
        return dict(bytes=2 * (2 * n * D + 2 * n * F + out * D + 6 * D * F), flops=12 * n * D * F)
    sizes = _sizes(case)
    width = [2 if case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 2) else 4 for i in range(len(sizes))]
    b = sum(n * w for n, w in zip(sizes, width))
    return dict(bytes=b * (2 if op == "grad_clip" else 1), flops=sum(sizes) * (3 if op == "grad_clip" else 2))


def _act64(g, act):
    """The activation and its derivative in 64 bits, from their definitions."""
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * torch.sigmoid(-g)
    z = C1 * (g + C3 * g ** 3)
    phi = torch.sigmoid(2 * z)   # (1 + tanh z) / 2
    return g * phi, phi + g * 2 * phi * torch.sigmoid(-2 * z) * C1 * (1 + 3 * C3 * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda k: s[k].double()  # noqa: E731
    if case["op"] == "ffn_fwd":
        up = torch.einsum("md,df->mf", d("x"), d("w_up"))
        g, u = up.chunk(2, dim=1)
        return dict(up=up, y=torch.einsum("mf,fd->md", _act64(g, case["act"])[0] * u, d("w_down")))
    if case["op"] == "ffn_bwd":
        x, up, dy = d("x"), d("up"), d("dy")
        if case["src"] == "full":
            x, up, dy = x[s["rows"]], up[s["rows"]], dy[s["rows"]]
        g, u = up.chunk(2, dim=1)
        a, slope = _act64(g, case["act"])
        ds = torch.einsum("md,fd->mf", dy, d("w_down"))
        dg, du = ds * u * slope, ds * a
        wg, wu = d("w_up").chunk(2, dim=1)
        dx = torch.einsum("mf,df->md", dg, wg) + torch.einsum("mf,df->md", du, wu)
        if case["dst"] == "full":
            full = torch.zeros(s["M"], case["D"], dtype=torch.float64, device=DEV)
            full[s["rows"]] = dx
            dx = full
        dw_up = torch.cat((torch.einsum("md,mf->df", x, dg), torch.einsum("md,mf->df", x, du)), 1)
        return dict(dx=dx, dw_up=dw_up, dw_down=torch.einsum("mf,md->fd", a * u, dy))
    order = 2 if case["kind"] == "l2" else math.inf
    norms = torch.stack([torch.linalg.vector_norm(g.double(), order) for g in s["grads"]]) * case["scale"]
    norm = torch.linalg.vector_norm(norms, order).reshape(1)
    if case["op"] == "grad_norm":
        return dict(norm=norm, norms=norms)
    coef = case["scale"] * min(1.0, s["max_norm"] / (norm.item() + EPS))
    out = dict(norm=norm, norms=norms, coef=torch.full((1,), coef, dtype=torch.float64, device=DEV))
    for key, flat in s["flat"].items():
        factor = torch.ones_like(flat)
        for t in s["grads"]:
            if t.dtype == flat.dtype:
                at = t.storage_offset()
                factor[at: at + t.numel()] = 0
        out[key] = flat.double() * torch.where(factor == 0, coef, 1.0)
    return out
