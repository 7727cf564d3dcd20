"""8-bit activation checkpoints on the GPU: pack and unpack bit for bit against the float64 oracle, and the
linear backward from a checkpoint."""
import numpy as np
import pytest
import torch

from oracle import ckpt as ock
import workloads

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
FMT = {"e4m3": cl.CKPT_E4M3, "int8": cl.CKPT_INT8}
DT = {"bf16": (cl.BF16, torch.bfloat16), "f32": (cl.F32, torch.float32)}


def values(rows, N, dtype, seed):
    """Rows over the whole range of exponents, with zero groups, ties, limits, infinities and NaNs among them."""
    rng = np.random.default_rng(seed)
    v = rng.normal(size=(rows, N)) * np.exp(rng.uniform(-20, 20, size=(rows, 1)))
    v[rng.random((rows, N)) < 0.02] = 0.0
    v *= np.where(rng.random(N) < 0.05, 30.0, 1.0)
    if rows > 7:
        v[1] = -0.0
        v[2, :32] = np.linspace(-448, 448, 32)
        v[3, :32] = np.arange(32) * 4 - 63.5
        v[4, 1], v[5, N - 1], v[6, N // 2] = np.nan, np.inf, -np.inf
        v[7, :] = np.where(np.arange(N) % 32 == 0, 3.0e38, 1e-38)
    v = v.astype(np.float32)
    return workloads.bf16_representable(v) if dtype == "bf16" else v


def index(M, f, seed):
    rng = np.random.default_rng(seed)
    keep = rng.random(M) >= f
    rows = np.flatnonzero(keep)
    idx = np.full(M, -1)
    idx[: rows.size] = rows
    return rows, gu.i32(idx), gu.i32([rows.size])


def dev(v, dtype):
    return torch.from_numpy(np.ascontiguousarray(v)).to(gu.DEV).to(DT[dtype][1])


def strided(rows, cols, dtype, pad, fill=0):
    """A [rows, cols] view with `pad` more elements a row, filled with a mark."""
    t = torch.full((rows, cols + pad), fill, dtype=dtype, device=gu.DEV)
    return t, t[:, :cols]


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


SIZES = [(1, 32), (1, 1056), (8, 96), (130, 64), (257, 2048), (37, 11264), (300, 1536)]


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_pack_and_unpack(M, N, dtype, fmt):
    v = values(M, N, dtype, M + N)
    cdt, tdt = DT[dtype]
    src, sv = strided(M, N, tdt, 8)
    sv.copy_(dev(v, dtype))
    ct, code = strided(M + 1, N, torch.uint8, 16, 0xAB)
    et, exps = strided(M + 1, N // 32, torch.uint8, 3, 0xCD)
    q = cl.ckpt(FMT[fmt], code, exps)
    want_c, want_e = ock.pack(v, fmt)
    # every row, then the kept rows; rows and columns beyond are left as they were
    for f in (None, 0.45):
        ct.fill_(0xAB)
        et.fill_(0xCD)
        rows, idx, nk = (np.arange(M), None, None) if f is None else index(M, f, M)
        cl.collider_ckpt_pack(cdt, src, src.stride(0), M, N, idx, nk, q)
        cl.collider_check()
        n = rows.size
        assert np.array_equal(code[:n].cpu().numpy(), want_c[rows])
        assert np.array_equal(exps[:n].cpu().numpy(), want_e[rows])
        assert bool((ct[n:] == 0xAB).all()) and bool((ct[:, N:] == 0xAB).all())
        assert bool((et[n:] == 0xCD).all()) and bool((et[:, N // 32:] == 0xCD).all())
        # back: COMPACT and FULL
        val = ock.unpack(want_c, want_e, fmt)[rows]
        for drows in (cl.ROWS_COMPACT, cl.ROWS_FULL):
            dt, dst = strided(M, N, tdt, 16, 7.0)
            cl.collider_ckpt_unpack(cdt, q, cl.ROWS_COMPACT, M, N, idx, nk, dst, dt.stride(0), drows)
            cl.collider_check()
            got = gu.host(dst)
            if drows == cl.ROWS_FULL:
                full = np.zeros((M, N))
                full[rows] = val
                assert same(got, full)
            else:
                pad = min(-(-n // 128) * 128, M)
                assert same(got[:n], val) and np.all(got[n:pad] == 0) and np.all(got[pad:] == 7)
            assert bool((dt[:, N:] == 7).all())
    # a checkpoint of FULL rows, its kept rows
    cl.collider_ckpt_pack(cdt, src, src.stride(0), M, N, None, None, q)
    rows, idx, nk = index(M, 0.5, M + 1)
    dst = torch.full((M, N), 7.0, dtype=tdt, device=gu.DEV)
    cl.collider_ckpt_unpack(cdt, q, cl.ROWS_FULL, M, N, idx, nk, dst, N, cl.ROWS_COMPACT)
    assert same(gu.host(dst)[: rows.size], ock.unpack(want_c, want_e, fmt)[rows])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_code_and_exponent_decodes(fmt):
    """All 256 codes under all 256 exponent bytes (other programs' checkpoints may hold any), exactly in f32."""
    code = np.repeat(np.arange(256, dtype=np.uint8)[None, :], 256, axis=0)
    exps = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, axis=1)
    q = cl.ckpt(FMT[fmt], torch.from_numpy(code).to(gu.DEV), torch.from_numpy(exps).to(gu.DEV))
    dst = torch.empty(256, 256, dtype=torch.float32, device=gu.DEV)
    cl.collider_ckpt_unpack(cl.F32, q, cl.ROWS_FULL, 256, 256, None, None, dst, 256, cl.ROWS_FULL)
    with np.errstate(over="ignore"):
        want = ock.unpack(code, exps, fmt).astype(np.float32)
    assert same(dst.cpu().numpy(), want)


def test_nothing_kept_everything_kept_and_a_bad_index():
    M, N = 300, 96
    v = values(M, N, "bf16", 3)
    src = dev(v, "bf16")
    code = torch.full((M, N), 0xAB, dtype=torch.uint8, device=gu.DEV)
    exps = torch.full((M, 3), 0xCD, dtype=torch.uint8, device=gu.DEV)
    q = cl.ckpt(cl.CKPT_E4M3, code, exps)
    none, zero = gu.i32(np.full(M, -1)), gu.i32([0])
    cl.collider_ckpt_pack(cl.BF16, src, N, M, N, none, zero, q)
    assert bool((code == 0xAB).all()) and bool((exps == 0xCD).all())
    dst = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=gu.DEV)
    cl.collider_ckpt_unpack(cl.BF16, q, cl.ROWS_COMPACT, M, N, none, zero, dst, N, cl.ROWS_COMPACT)
    assert bool((dst == 7).all())
    cl.collider_ckpt_unpack(cl.BF16, q, cl.ROWS_COMPACT, M, N, none, zero, dst, N, cl.ROWS_FULL)
    assert bool((dst == 0).all())
    idx, nk = gu.i32(np.arange(M)), gu.i32([M])
    cl.collider_ckpt_pack(cl.BF16, src, N, M, N, idx, nk, q)
    assert np.array_equal(code.cpu().numpy(), ock.pack(v, "e4m3")[0])
    # an index outside the rows is skipped and reported; the others are there
    cl.collider_check()
    code.fill_(0xAB)
    bad = np.arange(M)
    bad[17] = M
    cl.collider_ckpt_pack(cl.BF16, src, N, M, N, gu.i32(bad), nk, q)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_check()
    assert e.value.status == cl.ERR_INVALID_ARG
    assert bool((code[17] == 0xAB).all()) and bool((code[16] != 0xAB).any())


def test_checkpoint_in_pinned_host_memory():
    M, N = 513, 1024
    v = values(M, N, "bf16", 9)
    src = dev(v, "bf16")
    code = torch.zeros(M, N, dtype=torch.uint8).pin_memory()
    exps = torch.zeros(M, N // 32, dtype=torch.uint8).pin_memory()
    q = cl.ckpt(cl.CKPT_INT8, code, exps)
    rows, idx, nk = index(M, 0.3, 2)
    cl.collider_ckpt_pack(cl.BF16, src, N, M, N, idx, nk, q)
    cl.collider_check()
    c, e = ock.pack(v, "int8")
    assert np.array_equal(code.numpy()[: rows.size], c[rows]) and np.array_equal(exps.numpy()[: rows.size], e[rows])
    dst = torch.empty(M, N, dtype=torch.bfloat16, device=gu.DEV)
    cl.collider_ckpt_unpack(cl.BF16, q, cl.ROWS_COMPACT, M, N, idx, nk, dst, N, cl.ROWS_COMPACT)
    assert same(gu.host(dst)[: rows.size], ock.unpack(c[rows], e[rows], "int8"))


def test_wrong_memory_is_refused():
    M, N = 4, 64
    d = torch.zeros(M, N, dtype=torch.bfloat16, device=gu.DEV)
    h = torch.zeros(M, N, dtype=torch.bfloat16)
    code = torch.zeros(M, N, dtype=torch.uint8, device=gu.DEV)
    exps = torch.zeros(M, 2, dtype=torch.uint8, device=gu.DEV)
    q = cl.ckpt(cl.CKPT_E4M3, code, exps)
    for call in (lambda: cl.collider_ckpt_pack(cl.BF16, h, N, M, N, None, None, q),
                 lambda: cl.collider_ckpt_unpack(cl.BF16, q, 0, M, N, None, None, h, N, 0),
                 lambda: cl.collider_ckpt_pack(cl.BF16, d, N, M, N, None, None, cl.ckpt(0, code.cpu(), exps))):
        with pytest.raises(cl.ColliderError) as e:
            call()
        assert e.value.status == cl.ERR_INVALID_ARG and "memory" in str(e.value)


def test_offsets_beyond_32_bits():
    """Rows of values 2^28 elements apart and of codes 2^29 bytes apart: the last row of ten lies beyond 2^32 bytes."""
    M, N = 10, 96
    v = values(M, N, "bf16", 12)
    big = torch.empty(M << 28, dtype=torch.bfloat16, device=gu.DEV).view(M, 1 << 28)
    src, dst = big[:, :N], big[:, 1024:1024 + N]
    src.copy_(dev(v, "bf16"))
    codes = big.view(torch.uint8).view(M, 1 << 29)
    q = cl.ckpt(cl.CKPT_E4M3, codes[:, 8192:8192 + N], codes[:, 16384:16384 + N // 32])
    cl.collider_ckpt_pack(cl.BF16, src, 1 << 28, M, N, None, None, q)
    cl.collider_ckpt_unpack(cl.BF16, q, cl.ROWS_FULL, M, N, None, None, dst, 1 << 28, cl.ROWS_FULL)
    cl.collider_check()
    c, e = ock.pack(v, "e4m3")
    assert np.array_equal(q.buffers[0].cpu().numpy(), c) and np.array_equal(q.buffers[1].cpu().numpy(), e)
    assert same(gu.host(dst), ock.unpack(c, e, "e4m3"))


# --------------------------------------------------------------------------
# linear backward from a checkpoint
# --------------------------------------------------------------------------
def _mma_tol(ref_abs, steps):
    """f32 accumulation on the tensor core: a step adds 16 products, and may drop up to one unit in the last place
    (2^-23 of the magnitude, at most the sum of all magnitudes) when it aligns the products and one when it adds."""
    return 2 * steps * 2.0 ** -23 * ref_abs


@pytest.mark.parametrize("M,K,N,f", [(1, 32, 8, 0.0), (77, 96, 40, 0.3), (128, 256, 256, 0.4), (700, 512, 1000, 0.6),
                                     (4500, 64, 72, 0.05), (300, 2048, 256, 1.0), (640, 1056, 520, 0.0)])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("x_rows,dy_rows,dx_rows", [(0, 0, 0), (1, 0, 1), (0, 1, 0)])
def test_linear_backward(M, K, N, f, fmt, x_rows, dy_rows, dx_rows):
    rng = np.random.default_rng(M + K + N)
    rows, idx, nk = index(M, f, M + 5)
    n = rows.size
    X = workloads.bf16_representable(rng.normal(size=(M, K)) + 0.5)
    code, exps = ock.pack(X, fmt)
    Xd = ock.unpack(code, exps, fmt)[rows]
    W = workloads.bf16_representable(rng.normal(size=(K, N)) * 0.02).astype(np.float64)
    dY = workloads.bf16_representable(rng.normal(size=(M, N))).astype(np.float64)
    lay = lambda a, r: a if r == 0 else np.concatenate([a[rows], np.full((M - n,) + a.shape[1:], 99)])  # noqa: E731
    c, e = (torch.from_numpy(np.ascontiguousarray(lay(t, x_rows)).astype(np.uint8)).to(gu.DEV) for t in (code, exps))
    q = cl.ckpt(FMT[fmt], c, e)
    dX = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=gu.DEV)
    dW = torch.full((K, N), 7.0, device=gu.DEV)
    db = torch.full((N,), 7.0, device=gu.DEV)
    ws = torch.empty(cl.collider_linear_ckpt_workspace_size(M, K, N), dtype=torch.uint8, device=gu.DEV).fill_(255)
    cl.collider_linear_bwd_ckpt(M, K, N, q, x_rows, gu.bf16(W), gu.bf16(lay(dY, dy_rows)), dy_rows, idx, nk, dX, dx_rows,
                                dW, db, ws)
    cl.collider_check()
    dYk = dY[rows]
    rX, aX = dYk @ W.T, np.abs(dYk) @ np.abs(W).T
    got = gu.host(dX)
    if dx_rows == 0:
        assert np.all(np.delete(got, rows, axis=0) == 0)
        got = got[rows]
    else:
        pad = min(-(-n // 128) * 128, M)
        assert np.all(got[n:pad] == 0) and np.all(got[pad:] == 7)
        got = got[:n]
    tol = _mma_tol(aX, N / 16 + 1)
    assert np.all(np.abs(got - rX) <= tol + 2.0 ** -8 * (np.abs(rX) + tol))
    rW, aW = Xd.T @ dYk, np.abs(Xd).T @ np.abs(dYk)
    assert np.all(np.abs(gu.host(dW) - rW) <= _mma_tol(aW, min(n, 2560) / 16 + 1 + n / 1280))
    # db: f32 sums of at most n terms
    assert np.all(np.abs(gu.host(db) - dYk.sum(0)) <= (n + 1) * 2.0 ** -24 * np.abs(dYk).sum(0))


def test_linear_parts_alone_and_repeat():
    M, K, N = 500, 256, 128
    rng = np.random.default_rng(4)
    rows, idx, nk = index(M, 0.4, 8)
    code, exps = (torch.from_numpy(t).to(gu.DEV) for t in ock.pack(rng.normal(size=(M, K)), "e4m3"))
    q = cl.ckpt(cl.CKPT_E4M3, code, exps)
    W, dY = gu.bf16(rng.normal(size=(K, N))), gu.bf16(rng.normal(size=(M, N)))
    ws = torch.empty(cl.collider_linear_ckpt_workspace_size(M, K, N), dtype=torch.uint8, device=gu.DEV)

    def run(x=q, want_dx=True, want_dw=True, want_db=True):
        dX = torch.empty(M, K, dtype=torch.bfloat16, device=gu.DEV) if want_dx else None
        dW = torch.empty(K, N, device=gu.DEV) if want_dw else None
        db = torch.empty(N, device=gu.DEV) if want_db else None
        cl.collider_linear_bwd_ckpt(M, K, N, x, 0, W if want_dx else None, dY, 0, idx, nk, dX, 0, dW, db, ws)
        return dX, dW, db
    a, b = run(), run()
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    assert torch.equal(run(x=None, want_dw=False)[0], a[0])
    assert torch.equal(run(want_dx=False)[1], a[1])
    assert torch.equal(run(want_dx=False, want_dw=False)[2], a[2])
    # the decoded rows through collider_linear_bwd: the same products; db in the same order, dX and dW perhaps cut elsewhere
    ws = torch.empty(cl.collider_linear_workspace_size(cl.BF16, M, K, N), dtype=torch.uint8, device=gu.DEV)
    X = torch.empty(M, K, dtype=torch.bfloat16, device=gu.DEV)
    cl.collider_ckpt_unpack(cl.BF16, q, 0, M, K, None, None, X, K, 0)
    dX, dW, db = torch.empty_like(a[0]), torch.empty_like(a[1]), torch.empty_like(a[2])
    cl.collider_linear_bwd(cl.BF16, M, K, N, X, 0, W, dY, 0, idx, nk, dX, 0, dW, db, ws)
    assert torch.equal(db, a[2])
    assert gu.rel_err(gu.host(dX), gu.host(a[0])) <= 2.0 ** -7      # half a bf16 step each
    assert gu.rel_err(gu.host(dW), gu.host(a[1])) <= 1e-5


def test_linear_with_a_bad_index():
    """A kept index outside the tokens is reported; its row counts as zeros, and the other rows' results stand."""
    M, K, N = 200, 64, 64
    rng = np.random.default_rng(6)
    code, exps = ock.pack(rng.normal(size=(M, K)), "int8")
    q = cl.ckpt(cl.CKPT_INT8, torch.from_numpy(code).to(gu.DEV), torch.from_numpy(exps).to(gu.DEV))
    W, dY = gu.bf16(rng.normal(size=(K, N))), gu.bf16(rng.normal(size=(M, N)))
    idx = np.arange(M)
    idx[33] = M + 7
    ws = torch.full((cl.collider_linear_ckpt_workspace_size(M, K, N),), 255, dtype=torch.uint8, device=gu.DEV)
    dX = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=gu.DEV)
    dW, db = torch.empty(K, N, device=gu.DEV), torch.empty(N, device=gu.DEV)
    cl.collider_linear_bwd_ckpt(M, K, N, q, 0, W, dY, 0, gu.i32(idx), gu.i32([M]), dX, 0, dW, db, ws)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_check()
    assert e.value.status == cl.ERR_INVALID_ARG
    X, G = ock.unpack(code, exps, "int8"), gu.host(dY)
    X[33] = G[33] = 0
    assert gu.rel_err(gu.host(dW), X.T @ G) <= 1e-5 and gu.rel_err(gu.host(db), G.sum(0)) <= 1e-5
    rows = [r for r in range(M) if r != 33]
    assert gu.rel_err(gu.host(dX)[rows], (G @ gu.host(W).T)[rows]) <= 2.0 ** -7 and bool((dX[33] == 7).all())


def test_linear_of_many_rows():
    """Half a million kept rows: the reduction runs in some two hundred pieces."""
    M, K, N = 1000003, 32, 8
    rows, idx, nk = index(M, 0.5, 3)
    g = torch.Generator(device=gu.DEV).manual_seed(1)
    x = (torch.randn(M, K, generator=g, device=gu.DEV) + 0.5).to(torch.bfloat16)
    code = torch.empty(M, K, dtype=torch.uint8, device=gu.DEV)
    exps = torch.empty(M, 1, dtype=torch.uint8, device=gu.DEV)
    q = cl.ckpt(cl.CKPT_INT8, code, exps)
    cl.collider_ckpt_pack(cl.BF16, x, K, M, K, None, None, q)
    cl.collider_ckpt_unpack(cl.BF16, q, 0, M, K, None, None, x, K, 0)
    W = torch.randn(K, N, generator=g, device=gu.DEV).to(torch.bfloat16)
    dY = torch.randn(M, N, generator=g, device=gu.DEV).to(torch.bfloat16)
    dX = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=gu.DEV)
    dW, db = torch.empty(K, N, device=gu.DEV), torch.empty(N, device=gu.DEV)
    ws = torch.empty(cl.collider_linear_ckpt_workspace_size(M, K, N), dtype=torch.uint8, device=gu.DEV)
    cl.collider_linear_bwd_ckpt(M, K, N, q, 0, W, dY, 0, idx, nk, dX, 0, dW, db, ws)
    cl.collider_check()
    at = torch.from_numpy(rows).to(gu.DEV)
    xk, dk, wd = x[at].double(), dY[at].double(), W.double()
    mag = xk.abs().T @ dk.abs()
    # a piece's steps (2 units of 2^-23 of its magnitude each), and an f32 add of the whole for each piece
    tol = (2 * (2560 / 16 + 1) * 2.0 ** -23 + (rows.size / 2560 + 2) * 2.0 ** -24) * mag
    assert bool(((dW.double() - xk.T @ dk).abs() <= tol).all())
    ref = dk @ wd.T
    off = _mma_tol(1.0, N / 16 + 1) * (dk.abs() @ wd.abs().T)
    assert bool(((dX[at].double() - ref).abs() <= off + 2.0 ** -8 * (ref.abs() + off)).all())
    dX[at] = 0
    assert bool((dX == 0).all())


@pytest.mark.parametrize("dy_rows,dx_rows", [(0, 0), (1, 1), (0, 1)])
def test_linear_dx_in_the_place_of_dy(dy_rows, dx_rows):
    """dX over dY, in the layouts that may: the same bits as apart from it."""
    M, K = 700, 512
    rng = np.random.default_rng(9)
    rows, idx, nk = index(M, 0.4, 2)
    code, exps = (torch.from_numpy(t).to(gu.DEV) for t in ock.pack(rng.normal(size=(M, K)), "e4m3"))
    q = cl.ckpt(cl.CKPT_E4M3, code, exps)
    W, dY = gu.bf16(rng.normal(size=(K, K))), gu.bf16(rng.normal(size=(M, K)))
    ws = torch.empty(cl.collider_linear_ckpt_workspace_size(M, K, K), dtype=torch.uint8, device=gu.DEV)
    got = []
    for apart in (True, False):
        g = dY.clone()
        dX = torch.empty_like(g) if apart else g
        dW, db = torch.empty(K, K, device=gu.DEV), torch.empty(K, device=gu.DEV)
        cl.collider_linear_bwd_ckpt(M, K, K, q, 0, W, g, dy_rows, idx, nk, dX, dx_rows, dW, db, ws)
        cl.collider_check()
        n = M if dx_rows == 0 else min(-(-rows.size // 128) * 128, M)
        got.append((dX[:n], dW, db))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_calls_of_two_threads():
    """Two host threads, each with its own stream, buffers and workspace, issue the linear backward and the join's
    together, the wider one's first calls among them; both get the bits that calls one after the other give."""
    import threading

    def work(D, seed):
        M, K, N = 600, D, 256
        rng = np.random.default_rng(seed)
        rows, idx, nk = index(M, 0.4, seed)
        cu = gu.i32([0, rows.size])
        code, exps = (torch.from_numpy(t).to(gu.DEV) for t in ock.pack(rng.normal(size=(M, K)), "int8"))
        q = cl.ckpt(cl.CKPT_INT8, code, exps)
        W, dY = gu.bf16(rng.normal(size=(K, N))), gu.bf16(rng.normal(size=(M, N)))
        y, da, dh = (gu.bf16(rng.normal(size=(M, D))) for _ in range(3))
        w, rstd = gu.bf16(np.ones(D)), torch.ones(M, device=gu.DEV)
        d = cl.ResidualNormDesc(dtype=cl.BF16, B=1, T=M, D=D, norm=cl.NORM_RMS, post=1, pre=1, eps=1e-5, res_scale=1.0)
        p = cl.residual_norm_params(post_w=w, pre_w=w)
        sv = cl.residual_norm_saved(y=y, h=da, rstd_y=rstd, rstd_h=rstd)
        ws = torch.empty(cl.collider_linear_ckpt_workspace_size(M, K, N), dtype=torch.uint8, device=gu.DEV)
        wj = torch.empty(cl.collider_residual_norm_bwd_workspace_size(d), dtype=torch.uint8, device=gu.DEV)

        def run(stream):
            outs = []
            for _ in range(20):
                dX, dx, dy = (torch.empty(M, D, dtype=torch.bfloat16, device=gu.DEV) for _ in range(3))
                dW, db, dw = (torch.empty(s, device=gu.DEV) for s in ((K, N), (N,), (D,)))
                g = cl.residual_norm_grads(dx=dx, dy=dy, dpre_w=dw)
                cl.collider_linear_bwd_ckpt(M, K, N, q, 0, W, dY, 0, idx, nk, dX, 0, dW, db, ws, stream=stream)
                cl.collider_residual_norm_bwd(d, p, sv, 0, da, dh, 0, idx, cu, nk, g, 0, wj, stream=stream)
                outs.append((dX, dW, db, dx, dy, dw))
            return outs
        return run
    runs = [work(1024, 1), work(6144, 2)]
    streams = [torch.cuda.Stream() for _ in runs]
    got = [None, None]
    gate = threading.Barrier(2, timeout=60)

    def body(i):
        with torch.cuda.stream(streams[i]):
            gate.wait()
            got[i] = runs[i](streams[i].cuda_stream)
            streams[i].synchronize()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=body, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    cl.collider_check()
    for i, run in enumerate(runs):
        assert got[i] is not None
        want = run(0)[0]
        torch.cuda.synchronize()
        for outs in got[i]:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
