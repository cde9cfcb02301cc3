"""The operators around a product on the GPU against plain 64-bit
implementations (ops_ref.py), with bounds that count the roundings: epilogue
products and their gradients, RMS norms and theirs, 8-bit rows and products."""
import itertools

import numpy as np
import pytest
import torch

import fp32_gemm_sgemm_amd as sg
import ops_ref as ref
from gpu_cases import forced, forced_split, note, place

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, scale=1.0):
    return (np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32)


def dev(x, pad=0, shift=0):
    return place(x, pad, shift) if x.ndim == 2 else torch.from_numpy(np.ascontiguousarray(x)).to("cuda")


def guarded(rows, cols, pad=3, dtype=torch.float32):
    """A rows x cols output inside a buffer of sentinels (between rows, before
    and after); returns (view, check that the sentinels stand)."""
    ld = cols + pad
    buf = torch.full((rows * ld + 2 * 64,), 77.0, dtype=torch.float32, device="cuda").to(dtype)
    view = buf[64:64 + rows * ld].view(rows, ld)[:, :cols]

    def check():
        b = buf.float().clone()
        b[64:64 + rows * ld].view(rows, ld)[:, :cols] = 77.0
        want = torch.full((1,), 77.0).to(dtype).float().item()
        b[b == 77.0] = want
        assert bool((b == want).all()), "memory outside the output was written"
    return view, check


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- the product with an epilogue ---------------------------------------------------------

SHAPES = [(1, 1, 1), (1, 65, 130), (3, 40, 17), (16, 16, 64), (5, 7, 0), (33, 31, 257), (64, 64, 512), (70, 130, 96),
          (129, 257, 65), (260, 258, 100), (257, 512, 320)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ta,tb", itertools.product((False, True), repeat=2))
def test_epilogue_shapes(M, N, K, ta, tb):
    """Every layout at small and ragged sizes, activations in turn, with bias,
    residual and the stored pre-activation, rows padded and unaligned."""
    i = SHAPES.index((M, N, K)) + 2 * ta + tb
    name = ref.ACTS[i % len(ref.ACTS)]
    pad, shift = (0, 0) if i % 2 else (1, 1)
    note(f"epilogue {M}x{N}x{K} ta={ta} tb={tb} {name} pad {pad}")
    A = normal(*((K, M) if ta else (M, K)), seed=1)
    B = normal(*((N, K) if tb else (K, N)), seed=2, scale=max(K, 1) ** -0.5)
    bias, R = normal(N, seed=3), normal(M, N, seed=4)
    out, ok = guarded(M, N)
    pre, ok_pre = guarded(M, N, pad=5)
    y = sg.sgemm_epilogue(dev(A, pad, shift), dev(B, pad, shift), bias=dev(bias), activation=name,
                          residual=dev(R, pad, shift), out=out, pre=pre, alpha=0.75, transa=ta, transb=tb)
    torch.cuda.synchronize()
    assert y is out
    a, b = (A.T if ta else A).astype(np.float64), (B.T if tb else B).astype(np.float64)
    Y, Z, ty, tz = ref.product(a, b, K, 0.75, bias.astype(np.float64), name, R.astype(np.float64))
    ref.within(f64(pre), Z, tz, "pre")
    ref.within(f64(out), Y, ty, "out")
    ok()
    ok_pre()


def epilogue_variants():
    out = []
    for v in range(sg.sgemm_f32_num_variants()):
        if sg.sgemm_f32_variant(v).workspace_bytes >= 0:
            out.append(v)
    return out


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("ta,tb", itertools.product((False, True), repeat=2))
@pytest.mark.parametrize("vid", epilogue_variants())
def test_epilogue_every_variant(vid, ta, tb, grad):
    """Each tile that has an epilogue form, forced, over several tiles with
    edges; the others are refused."""
    q = sg.sgemm_f32_variant(vid)
    M, N, K = min(2 * q.bm + 5, 517), min(q.bn + 70, 330), 3 * max(q.bk, 16) + 9
    name = ("gelu", "silu", "gelu_tanh", "relu")[vid % 4]
    note(f"variant {vid} {M}x{N}x{K} ta={ta} tb={tb} grad={grad}")
    # 16-byte aligned rows for one operand set, 4-byte for the other
    pad = 1 if vid % 2 else 0
    A = normal(*((K, M) if ta else (M, K)), seed=5)
    B = normal(*((N, K) if tb else (K, N)), seed=6, scale=K ** -0.5)
    bias, R, Z0 = normal(N, seed=7), normal(M, N, seed=8), normal(M, N, seed=9, scale=2.0)
    kw = {"grad_pre": dev(Z0)} if grad else {"bias": dev(bias)}
    out, ok = guarded(M, N, pad=1)
    cfg = forced(vid)
    served = sg.sgemm_f32_variant_ops(vid) & (1 << (int(ta) + 2 * int(tb)))
    try:
        sg.sgemm_epilogue(dev(A, pad), dev(B, pad), activation=name, residual=dev(R), out=out, transa=ta, transb=tb,
                          cfg=cfg, **kw)
    except sg.SgemmError as e:
        assert e.code == 1
        # only the register-staged tiles and the vector-FMA comparison have no epilogue
        assert vid in (0, 1, 2, 3, 8, 9) or not served
        return
    assert vid not in (0, 1, 2, 3, 8, 9)
    torch.cuda.synchronize()
    a, b = (A.T if ta else A).astype(np.float64), (B.T if tb else B).astype(np.float64)
    Y, _, ty, _ = ref.product(a, b, K, 1.0, None if grad else bias.astype(np.float64), name, R.astype(np.float64),
                              Z0.astype(np.float64) if grad else None)
    ref.within(f64(out), Y, ty, f"variant {vid}")
    ok()


@pytest.mark.parametrize("splits", [2, 5])
@pytest.mark.parametrize("strips", [(0, 0), (3, 0), (0, 2), (4, 4)])
def test_epilogue_splits_and_strips(splits, strips):
    """The epilogue is applied once, by the reduction, to a K split's sum, and
    by the strip kernel to the edge rows and columns."""
    M, N, K = 64 + strips[0], 128 + strips[1], 700
    A, B = normal(M, K, seed=1), normal(K, N, seed=2, scale=K ** -0.5)
    bias, R = normal(N, seed=3), normal(M, N, seed=4)
    for sp, name in ((1, "silu"), (splits, "gelu")):
        cfg = forced_split(11, sp)
        cfg.strip_m, cfg.strip_n = strips
        note(f"splits {sp} strips {strips}")
        out, ok = guarded(M, N)
        pre, ok_pre = guarded(M, N)
        sg.sgemm_epilogue(dev(A), dev(B), bias=dev(bias), activation=name, residual=dev(R), out=out, pre=pre, cfg=cfg)
        torch.cuda.synchronize()
        Y, Z, ty, tz = ref.product(A.astype(np.float64), B.astype(np.float64), K, 1.0, bias.astype(np.float64), name,
                                   R.astype(np.float64))
        ref.within(f64(out), Y, ty)
        ref.within(f64(pre), Z, tz)
        ok()
        ok_pre()


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("M", [1, 2, 4])
def test_epilogue_single_tokens(M, tb):
    """A few rows (strips in either storage order, and the K-split tiles)."""
    N, K = 2049, 4100
    A, B = normal(M, K, seed=1), normal(*((N, K) if tb else (K, N)), seed=2, scale=K ** -0.5)
    bias, R = normal(N, seed=3), normal(M, N, seed=4)
    note(f"tokens {M} tb={tb}")
    for ws in (True, False):
        y = sg.sgemm_epilogue(dev(A), dev(B), bias=dev(bias), activation="silu", residual=dev(R), transb=tb,
                              workspace=ws)
        torch.cuda.synchronize()
        Y, _, ty, _ = ref.product(A.astype(np.float64), (B.T if tb else B).astype(np.float64), K, 1.0,
                                  bias.astype(np.float64), "silu", R.astype(np.float64))
        ref.within(f64(y), Y, ty)


@pytest.mark.parametrize("shape", [(40, 50, 60), (1, 33, 200), (130, 70, 64)])
def test_epilogue_batches(shape):
    """Batches with a shared weight, a bias per entry and one for all, strided
    residual and pre-activation, and a residual shared by the batch."""
    M, N, K = shape
    nb = 3
    A, B = normal(nb, M, K, seed=1), normal(K, N, seed=2, scale=K ** -0.5)
    R = normal(nb, M, N, seed=3)
    note(f"batch {shape}")
    for bias, res in ((normal(nb, N, seed=4), R), (normal(N, seed=5), R[:1]), (None, R)):
        pre = torch.full((nb, M, N + 4), 5.0, device="cuda")[:, :, :N]
        residual = torch.from_numpy(res).cuda()
        y = sg.sgemm_epilogue(torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda(),
                              bias=None if bias is None else torch.from_numpy(bias).cuda(), activation="gelu_tanh",
                              residual=residual if len(res) == nb else residual[0], pre=pre)
        torch.cuda.synchronize()
        b64 = None if bias is None else bias.astype(np.float64)
        b64 = b64[:, None, :] if b64 is not None and b64.ndim == 2 else b64
        Y, Z, ty, tz = ref.product(A.astype(np.float64), B.astype(np.float64)[None], K, 1.0, b64, "gelu_tanh",
                                   res.astype(np.float64))
        ref.within(f64(y), Y, ty)
        ref.within(f64(pre), Z, tz)


def test_epilogue_residual_in_place():
    """The residual may be the output itself, with and without a K split."""
    M, N, K = 70, 90, 1500
    A, B, R = normal(M, K, seed=1), normal(K, N, seed=2, scale=K ** -0.5), normal(M, N, seed=3)
    Y, _, ty, _ = ref.product(A.astype(np.float64), B.astype(np.float64), K, 1.0, None, "relu", R.astype(np.float64))
    for vid, sp in ((11, 1), (11, 4), (14, 1), (24, 1), (20, 1), (4, 1)):
        out = dev(R, 2)
        note(f"in place variant {vid} splits {sp}")
        sg.sgemm_epilogue(dev(A), dev(B), activation="relu", residual=out, out=out, cfg=forced_split(vid, sp))
        torch.cuda.synchronize()
        ref.within(f64(out), Y, ty)


def test_epilogue_of_nothing():
    """K == 0 and alpha == 0 give the epilogue of zero without reading A or B
    (NaN here); no rows or columns write nothing."""
    M, N = 37, 41
    bias, R, Z0 = normal(N, seed=1), normal(M, N, seed=2), normal(M, N, seed=3)
    want = ref.act(bias.astype(np.float64)[None], "gelu") + R
    for K, alpha in ((0, 1.0), (9, 0.0)):
        A = np.full((M, K), np.nan, np.float32)
        B = np.full((K, N), np.nan, np.float32)
        out, ok = guarded(M, N)
        sg.sgemm_epilogue(dev(A), dev(B), bias=dev(bias), activation="gelu", residual=dev(R), out=out, alpha=alpha)
        torch.cuda.synchronize()
        ref.within(f64(out), want, np.abs(want) * 4 * ref.U + ref.ACT_ERR * np.abs(bias) + 1e-37)
        ok()
        out, ok = guarded(M, N)
        sg.sgemm_epilogue(dev(A), dev(B), bias=dev(bias), activation="silu", grad_pre=dev(Z0), out=out, alpha=alpha)
        torch.cuda.synchronize()
        ref.within(f64(out), bias * ref.slope(Z0.astype(np.float64), "silu"),
                   np.abs(bias) * (ref.SLOPE_ERR + 2 * ref.U) + 1e-37)
    for M2, N2 in ((0, 5), (5, 0)):
        y = sg.sgemm_epilogue(torch.zeros(M2, 3, device="cuda"), torch.zeros(3, N2, device="cuda"), activation="silu",
                              bias=torch.zeros(N2, device="cuda"))
        assert tuple(y.shape) == (M2, N2)


@pytest.mark.parametrize("name", ref.ACTS[1:])
def test_activation_values_and_special_cases(name):
    """The activation alone (a 1 x 1 identity product) over its whole range,
    and the formula's own special values."""
    x = np.concatenate([np.linspace(-30, 30, 4001), [0.0, -0.0, 1e-30, -1e-30, 88, -88, 104, -104, 1e4, -1e4, 3e38,
                                                     -3e38, np.inf, -np.inf, np.nan]]).astype(np.float32)
    one = torch.ones(1, 1, device="cuda")
    z = torch.from_numpy(x).cuda()[None, :].contiguous()
    y = f64(sg.sgemm_epilogue(one, z, activation=name))[0]
    d = f64(sg.sgemm_epilogue(one, torch.ones_like(z), activation=name, grad_pre=z))[0]
    with np.errstate(all="ignore"):
        want, dwant = ref.act(x.astype(np.float64), name), ref.slope(x.astype(np.float64), name)
    fin = np.isfinite(x)
    small = fin & (np.abs(x) <= 104)
    assert np.all(np.abs(y[small] - want[small]) <= ref.ACT_ERR * np.abs(x[small]) + 1e-37)
    assert np.all(np.abs(d[small] - dwant[small]) <= ref.SLOPE_ERR)
    big = fin & ~small
    assert np.all(np.abs(y[big] - np.where(x[big] > 0, x[big], 0)) <= 2 * ref.U * np.abs(x[big]))
    assert np.all(d[big] == (x[big] > 0))
    assert np.isnan(y[-1])
    assert y[-3] == np.inf
    if name == "relu":
        assert y[-2] == 0
    else:
        assert np.isnan(y[-2])  # minus infinity times zero


# ---- the elementwise gradient ---------------------------------------------------------------

@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (5, 3), (64, 64), (257, 129), (1000, 130), (3000, 7), (517, 1030)])
@pytest.mark.parametrize("name", ref.ACTS)
def test_activation_grad(M, N, name):
    note(f"activation_grad {M}x{N} {name}")
    i = ref.ACTS.index(name)
    dy, z = normal(M, N, seed=i), normal(M, N, seed=i + 10, scale=2.0)
    DZ, DB, tz, tb = ref.act_grad(dy.astype(np.float64), z.astype(np.float64), name)
    out, ok = guarded(M, N)
    dbias, okb = guarded(1, N)
    sg.activation_grad(dev(dy, i % 3, i % 2), dev(z, 1, 1), name, out=out, dbias=dbias[0])
    torch.cuda.synchronize()
    ref.within(f64(out), DZ, tz, "dZ")
    ref.within(f64(dbias[0]), DB, tb, "dbias")
    ok()
    okb()
    # each alone, and in place
    a, none = sg.activation_grad(dev(dy), dev(z), name, dbias=False)
    assert none is None and torch.equal(a, out)
    none, b = sg.activation_grad(dev(dy, 2), dev(z), name, out=False)
    assert none is None and torch.equal(b, dbias[0])
    g = dev(dy, 1)
    sg.activation_grad(g, dev(z), name, out=g, dbias=False)
    torch.cuda.synchronize()
    assert torch.equal(g, out)


def test_activation_grad_of_no_rows():
    z, b = sg.activation_grad(torch.zeros(0, 9, device="cuda"), None, None)
    assert tuple(z.shape) == (0, 9) and bool((b == 0).all())
    z, b = sg.activation_grad(torch.zeros(9, 0, device="cuda"), None, None)
    assert b.numel() == 0


@pytest.mark.parametrize("ta,tb", itertools.product((False, True), repeat=2))
@pytest.mark.parametrize("M,N,K", [(1, 5, 9), (33, 70, 40), (200, 130, 257)])
def test_epilogue_backward(M, N, K, ta, tb):
    """dA (back through the layer below's activation), dB and dbias against the
    formula."""
    note(f"backward {M}x{N}x{K} ta={ta} tb={tb}")
    A = normal(*((K, M) if ta else (M, K)), seed=1)
    B = normal(*((N, K) if tb else (K, N)), seed=2, scale=K ** -0.5)
    dY, Z, P = normal(M, N, seed=3), normal(M, N, seed=4), normal(*A.shape, seed=5)
    a, b = (A.T if ta else A).astype(np.float64), (B.T if tb else B).astype(np.float64)
    DZ, DB, tdz, tdb = ref.act_grad(dY.astype(np.float64), Z.astype(np.float64), "gelu")
    dA, dB, dbias = sg.sgemm_epilogue_backward(dev(dY, 1), dev(A), dev(B, 2), pre=dev(Z), activation="gelu",
                                               a_pre=dev(P), a_activation="silu", transa=ta, transb=tb, alpha=0.5)
    torch.cuda.synchronize()
    ref.within(f64(dbias), DB, tdb, "dbias")
    wa = 0.5 * DZ @ b.T
    ta_ = (N + 3) * ref.U * 0.5 * np.abs(DZ) @ np.abs(b.T) + 0.5 * tdz @ np.abs(b.T)
    p = (P.T if ta else P).astype(np.float64)
    sl = ref.slope(p, "silu")
    got = f64(dA).T if ta else f64(dA)
    ref.within(got, wa * sl, ref.LIPSCHITZ * ta_ + ref.SLOPE_ERR * np.abs(wa) + ref.U * np.abs(wa * sl), "dA")
    wb = 0.5 * a.T @ DZ
    tb_ = (M + 3) * ref.U * 0.5 * np.abs(a.T) @ np.abs(DZ) + 0.5 * np.abs(a.T) @ tdz + 1e-37
    ref.within(f64(dB).T if tb else f64(dB), wb, tb_, "dB")
    x, y, z = sg.sgemm_epilogue_backward(dev(dY), dev(A), dev(B), transa=ta, transb=tb, need=("bias",))
    assert x is None and y is None
    ref.within(f64(z), dY.astype(np.float64).sum(0), np.abs(dY).sum(0) * (M + 1) * ref.U + 1e-37)


@pytest.mark.parametrize("M,N,K", [(0, 5, 7), (6, 0, 7), (6, 5, 0)])
def test_epilogue_backward_of_nothing(M, N, K):
    """An empty dimension: gradients of the operands' shapes, zeros where the
    sum is empty."""
    note(f"backward of nothing {M}x{N}x{K}")
    g, pre = torch.ones(M, N, device="cuda"), torch.ones(M, N, device="cuda")
    A, B = torch.ones(M, K, device="cuda"), torch.ones(K, N, device="cuda")
    dA, dB, db = sg.sgemm_epilogue_backward(g, A, B, pre=pre, activation="relu", a_pre=A, a_activation="relu")
    assert dA.shape == A.shape and dB.shape == B.shape and db.shape == (N,)
    assert bool((dA == 0).all()) and bool((dB == 0).all()) and bool((db == M).all())


@pytest.mark.parametrize("name", ref.ACTS)
def test_gradients_against_differences(name):
    """Central differences of the 64-bit forward pass along random directions.
    The step h leaves a truncation error of order h^2 (activations have third
    derivatives below 3) and the kernel's own bound; 2e-4 of the gradient's
    magnitude covers both at these sizes (h = 1e-4: 1e-7; float32 sums of 60
    terms: 4e-6).  ReLU's kinks are kept 1e-3 away."""
    M, N, K = 12, 20, 30
    A, B, bias, G = normal(M, K, seed=1), normal(K, N, seed=2, scale=K ** -0.5), normal(N, seed=3), normal(M, N, seed=4)
    f = lambda a, b, c: float((G * ref.act(a @ b + c, name)).sum())  # noqa: E731
    a, b, c = A.astype(np.float64), B.astype(np.float64), bias.astype(np.float64)
    assert name != "relu" or np.abs(a @ b + c).min() > 1e-3
    pre = torch.empty(M, N, device="cuda")
    sg.sgemm_epilogue(dev(A), dev(B), bias=dev(bias), activation=name, pre=pre)
    dA, dB, db = sg.sgemm_epilogue_backward(dev(G), dev(A), dev(B), pre=pre, activation=name)
    rng = np.random.default_rng(5)
    h = 1e-5 if name == "relu" else 1e-4
    for x, grad, at in ((a, f64(dA), 0), (b, f64(dB), 1), (c, f64(db), 2)):
        d = rng.standard_normal(x.shape)
        args = [[a, b, c], [a, b, c]]
        args[0][at], args[1][at] = x + h * d, x - h * d
        num = (f(*args[0]) - f(*args[1])) / (2 * h)
        assert abs(num - float((grad * d).sum())) <= 2e-4 * np.linalg.norm(grad) * np.linalg.norm(d)


# ---- norms -------------------------------------------------------------------------------------

WIDTHS = [1, 3, 64, 255, 256, 257, 512, 700, 1024, 1025, 2048, 3001, 4096, 5000, 8192, 10001, 16384, 16385, 40003]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(D, residual):
    rows = 9 if D < 5000 else 5
    i = WIDTHS.index(D)
    note(f"rmsnorm {rows}x{D} residual={residual}")
    x, w = normal(rows, D, seed=i) * np.exp(normal(rows, 1, seed=99)), 1 + 0.2 * normal(D, seed=i + 1)
    R = normal(rows, D, seed=i + 2) if residual else None
    w = w.astype(np.float32) if i % 4 else None
    eps = (1e-6, 0.0, 1e-2)[i % 3]
    Y, S, ty, rho = ref.rmsnorm(x.astype(np.float64), None if w is None else w.astype(np.float64), eps,
                                None if R is None else R.astype(np.float64))
    pad, shift = (0, 0) if i % 2 else (1, 1)
    X, Rd, wd = dev(x, pad, shift), None if R is None else dev(R, 4), None if w is None else dev(w)
    out, ok = guarded(rows, D)
    s_out, ok_s = guarded(rows, D, pad=1)
    y, s = sg.rmsnorm(X, wd, eps=eps, residual=Rd, out=out, sum_out=s_out if residual else None)
    torch.cuda.synchronize()
    ref.within(f64(out), Y, ty, "y")
    if residual:
        assert s is s_out
        ref.within(f64(s), S, ref.U * np.abs(S) + 1e-37, "s")
    else:
        assert s is X
    ok()
    ok_s()
    q, scale, s8 = sg.rmsnorm_e4m3(X, wd, eps=eps, residual=Rd)
    torch.cuda.synchronize()
    assert q.stride(0) % 16 == 0 and q.dtype == torch.float8_e4m3fn
    ref.check_codes(f64(q.float()), f64(scale), Y, ty, rho + 8 * ref.U)
    if residual:
        assert torch.equal(s8, s)


@pytest.mark.parametrize("D", [4100, 8192, 8200, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_many_long_rows(D, residual):
    """The forms that long rows take once there are many of them: the same
    values as the first rows alone, within the bounds, to the last row."""
    rows = 1030
    note(f"rmsnorm {rows}x{D} residual={residual}")
    x, w = normal(rows, D, seed=1), (1 + 0.2 * normal(D, seed=2)).astype(np.float32)
    R = normal(rows, D, seed=3) if residual else None
    Y, S, ty, rho = ref.rmsnorm(x.astype(np.float64), w.astype(np.float64), 1e-6,
                                None if R is None else R.astype(np.float64))
    out, ok = guarded(rows, D)
    y, s = sg.rmsnorm(dev(x, 1), dev(w), residual=None if R is None else dev(R), out=out)
    torch.cuda.synchronize()
    ref.within(f64(out), Y, ty)
    ok()
    q, scale, _ = sg.rmsnorm_e4m3(dev(x, 1), dev(w), residual=None if R is None else dev(R))
    torch.cuda.synchronize()
    ref.check_codes(f64(q.float()), f64(scale), Y, ty, rho + 8 * ref.U)
    q, scale = sg.quantize_e4m3(dev(x, 3))
    torch.cuda.synchronize()
    x64 = x.astype(np.float64)
    ref.check_codes(f64(q.float()), f64(scale), x64, np.zeros_like(x64), 0.0)


def test_quantize_codes_are_the_formulas():
    """Every code is the rounding of x / (max|x| / 448) in 64 bits: values are
    carried to float32 with one rounding, so only one that lies within half a
    unit of float32's last place of the border of two codes could differ."""
    for rows, D in ((3, 700), (300, 4096), (1500, 5000)):
        x = normal(rows, D, seed=D)
        q, _ = sg.quantize_e4m3(dev(x))
        v = x.astype(np.float64) / (np.abs(x.astype(np.float64)).max(1, keepdims=True) / 448)
        got = f64(q.float())
        step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3), 2.0 ** -9)
        assert np.all(np.abs(got - v) <= step / 2 + ref.U * np.abs(v))


def test_rmsnorm_in_place():
    """The residual stream updated in place; y over x."""
    for D in (300, 4096, 20000):
        x, R = normal(6, D, seed=1), normal(6, D, seed=2)
        y0, s0 = sg.rmsnorm(dev(x), residual=dev(R))
        for target in ("residual", "x"):
            X, Rd = dev(x), dev(R)
            y, s = sg.rmsnorm(X, residual=Rd, sum_out=Rd if target == "residual" else X)
            assert torch.equal(s, s0) and torch.equal(y, y0)
        X = dev(x)
        y, _ = sg.rmsnorm(X, out=X)
        y1, _ = sg.rmsnorm(dev(x))
        assert torch.equal(y, y1)


def test_rmsnorm_special_rows():
    """A row of zeros, one with an infinity and one with a NaN leave the other
    rows alone; eps == 0 on zeros is 0 / 0."""
    for D in (100, 3000, 20000):
        x = normal(5, D, seed=3)
        x[1] = 0
        x[2, 5] = np.inf
        x[3, 7] = np.nan
        y, _ = sg.rmsnorm(dev(x))
        y = f64(y)
        assert np.isfinite(y[[0, 1, 4]]).all() and (y[1] == 0).all()
        assert np.isnan(y[2, 5]) and (np.delete(y[2], 5) == 0).all() and np.isnan(y[3]).all()
        q, scale, _ = sg.rmsnorm_e4m3(dev(x))
        q, scale = f64(q.float()), f64(scale)
        assert np.isfinite(q[[0, 1, 4]]).all() and (q[1] == 0).all() and scale[1] == 2.0 ** -126
        assert np.isnan(q[2, 5]) and (np.delete(q[2], 5) == 0).all() and np.isnan(q[3]).all()
        # a row below the smallest scale: its codes are Y / 2^-126
        tiny = np.full((1, D), 1e-41, np.float32)
        tiny[0, 1:] = 0
        q, scale, _ = sg.rmsnorm_e4m3(dev(tiny), eps=1e-6)
        want = float(np.float64(tiny[0, 0]) * 1e3 / 2.0 ** -126)
        assert scale.item() == 2.0 ** -126 and abs(q[0, 0].float().item() - want) <= want / 16
        y, _ = sg.rmsnorm(dev(x), eps=0.0)
        assert np.isnan(f64(y)[1]).all() and np.isfinite(f64(y)[0]).all()


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("rows", [1, 37])
def test_rmsnorm_backward(D, rows):
    i = WIDTHS.index(D)
    if rows * D > 10 ** 6:
        rows = 11
    note(f"rmsnorm_backward {rows}x{D}")
    s, dy = normal(rows, D, seed=i) * np.exp(normal(rows, 1, seed=98)), normal(rows, D, seed=i + 1)
    w = (1 + 0.2 * normal(D, seed=i + 2)).astype(np.float32)
    ds = normal(rows, D, seed=i + 3) if i % 2 else None
    DX, DW, tx, tw = ref.rmsnorm_grad(dy.astype(np.float64), s.astype(np.float64), w.astype(np.float64), 1e-6,
                                      None if ds is None else ds.astype(np.float64))
    out, ok = guarded(rows, D)
    dx, dw = sg.rmsnorm_backward(dev(dy, i % 3), dev(s, 1, 1), dev(w), dsum=None if ds is None else dev(ds, 4), out=out)
    torch.cuda.synchronize()
    ref.within(f64(dx), DX, tx, "dx")
    ref.within(f64(dw), DW, tw, "dw")
    ok()
    if ds is not None:  # in place over the residual stream's gradient
        d = dev(ds, 4)
        dx2, none = sg.rmsnorm_backward(dev(dy), dev(s), dev(w), dsum=d, out=d, need_weight=False)
        torch.cuda.synchronize()
        assert none is None and torch.equal(dx2, dx)
    else:
        DX, _, tx, _ = ref.rmsnorm_grad(dy.astype(np.float64), s.astype(np.float64), None, 1e-6)
        dx, none = sg.rmsnorm_backward(dev(dy), dev(s))
        torch.cuda.synchronize()
        assert none is None
        ref.within(f64(dx), DX, tx, "dx without a weight")


@pytest.mark.parametrize("rows,D", [(5000, 64), (3000, 700), (2500, 2048), (1500, 5000)])
def test_rmsnorm_backward_many_rows(rows, D):
    """More rows than workgroups: the weight gradient's sums over several rows
    each and over all workgroups."""
    s, dy, w = normal(rows, D, seed=1), normal(rows, D, seed=2), normal(D, seed=3)
    note(f"rmsnorm_backward {rows}x{D}")
    DX, DW, tx, tw = ref.rmsnorm_grad(dy.astype(np.float64), s.astype(np.float64), w.astype(np.float64), 1e-6)
    dx, dw = sg.rmsnorm_backward(dev(dy), dev(s), dev(w))
    torch.cuda.synchronize()
    ref.within(f64(dx), DX, tx)
    ref.within(f64(dw), DW, tw)


@pytest.mark.parametrize("rows,D", [(513, 4100), (600, 8192), (1030, 6001)])
def test_rmsnorm_backward_long_rows_without_weight(rows, D):
    """The form of many long rows without a weight gradient, to the last row,
    with and without the residual stream's gradient."""
    s, dy, w, ds = normal(rows, D, seed=1), normal(rows, D, seed=2), normal(D, seed=3), normal(rows, D, seed=4)
    note(f"rmsnorm_backward {rows}x{D} without dw")
    DX, _, tx, _ = ref.rmsnorm_grad(dy.astype(np.float64), s.astype(np.float64), w.astype(np.float64), 1e-6)
    out, ok = guarded(rows, D)
    dx, none = sg.rmsnorm_backward(dev(dy, 1), dev(s), dev(w), out=out, need_weight=False)
    torch.cuda.synchronize()
    assert none is None
    ref.within(f64(out), DX, tx)
    ok()
    g = dev(ds)
    sg.rmsnorm_backward(dev(dy), dev(s, 3), dev(w), dsum=g, out=g, need_weight=False)
    torch.cuda.synchronize()
    ref.within(f64(g), DX + ds, tx + ref.U * np.abs(DX + ds), "with the stream's")


def test_rmsnorm_backward_of_no_rows():
    dx, dw = sg.rmsnorm_backward(torch.zeros(0, 40, device="cuda"), torch.zeros(0, 40, device="cuda"),
                                 torch.ones(40, device="cuda"))
    assert tuple(dx.shape) == (0, 40) and bool((dw == 0).all())


def test_rmsnorm_gradient_against_differences():
    """As test_gradients_against_differences: 64-bit forward, random directions."""
    rows, D = 4, 50
    x, w, G = normal(rows, D, seed=1), normal(D, seed=2), normal(rows, D, seed=3)
    f = lambda a, b: float((G * ref.rmsnorm(a, b, 1e-6)[0]).sum())  # noqa: E731
    dx, dw = sg.rmsnorm_backward(dev(G), dev(x), dev(w))
    a, b = x.astype(np.float64), w.astype(np.float64)
    rng, h = np.random.default_rng(4), 1e-4
    d, e = rng.standard_normal(a.shape), rng.standard_normal(b.shape)
    num = (f(a + h * d, b) - f(a - h * d, b)) / (2 * h)
    assert abs(num - float((f64(dx) * d).sum())) <= 2e-4 * np.linalg.norm(f64(dx)) * np.linalg.norm(d)
    num = (f(a, b + h * e) - f(a, b - h * e)) / (2 * h)
    assert abs(num - float((f64(dw) * e).sum())) <= 2e-4 * np.linalg.norm(f64(dw)) * np.linalg.norm(e)


# ---- 8 bits ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("D", WIDTHS)
def test_quantize(D):
    rows = 7
    i = WIDTHS.index(D)
    x = normal(rows, D, seed=i) * np.exp(3 * normal(rows, 1, seed=97))
    note(f"quantize {rows}x{D}")
    q, scale = sg.quantize_e4m3(dev(x.astype(np.float32), i % 3, i % 2))
    torch.cuda.synchronize()
    y = x.astype(np.float32).astype(np.float64)
    ref.check_codes(f64(q.float()), f64(scale), y, np.zeros_like(y), 0.0)


def test_quantize_special_values():
    D = 40
    x = np.zeros((6, D), np.float32)
    x[1] = 1e-40                       # below the smallest scale: rounds to zero steps of 2^-126
    x[2] = np.linspace(-3e38, 3e38, D)
    x[3] = normal(1, D)
    x[3, 4] = np.nan
    x[4] = normal(1, D)
    x[4, 9] = -np.inf
    x[5] = np.float32(448) * np.float32(2.0) ** -3
    q, scale = sg.quantize_e4m3(dev(x))
    q, scale = f64(q.float()), f64(scale)
    assert (q[0] == 0).all() and scale[0] == 2.0 ** -126 and scale[1] == 2.0 ** -126
    assert np.isfinite(q[[0, 1, 2, 5]]).all() and q[2].max() == 448 and q[2].min() == -448
    assert (q[5] == 448).all() and scale[5] == 2.0 ** -3
    assert np.isnan(q[3, 4]) and np.isfinite(np.delete(q[3], 4)).all()
    assert scale[3] == np.float32(np.nanmax(np.abs(x[3])) / np.float32(448))
    assert np.isinf(scale[4]) and np.isnan(q[4, 9]) and (np.delete(q[4], 9) == 0).all()


def test_quantize_rounds_to_nearest_even():
    """Every code comes back as itself, and ties between codes go to the even one."""
    v = ref.E4M3[np.isfinite(ref.E4M3)]
    q, scale = sg.quantize_e4m3(dev(v.astype(np.float32)[None]))
    assert scale.item() == 1.0 and np.array_equal(f64(q.float())[0], v)
    pos = np.sort(v[(v >= 0) & ~np.signbit(v)])
    ties = ((pos[:-1] + pos[1:]) / 2).astype(np.float32)
    x = np.concatenate([ties, [448.0]]).astype(np.float32)
    q, scale = sg.quantize_e4m3(dev(x[None]))
    even = np.where(np.arange(len(ties)) % 2 == 0, pos[:-1], pos[1:])
    assert scale.item() == 1.0 and np.array_equal(f64(q.float())[0][:-1], even)


def codes(rows, cols, seed, pad=0):
    """Random codes (no NaN) in a buffer whose padding holds NaN codes, and
    their values."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (rows, cols + pad), dtype=np.uint8)
    c[(c & 0x7f) == 0x7f] = 0x30
    c[:, cols:] = 0x7f
    t = torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)
    return t[:, :cols], ref.E4M3[c[:, :cols]]


E4M3_SHAPES = [(1, 1, 1), (1, 40, 15), (1, 300, 4096), (2, 16, 128), (5, 33, 200), (16, 100, 1000), (17, 64, 129),
               (33, 70, 2100), (64, 130, 64), (65, 65, 127), (70, 200, 16), (100, 129, 700), (129, 300, 513),
               (200, 520, 1040), (257, 260, 96), (300, 70, 3000), (1030, 1100, 130), (7, 9, 0)]


@pytest.mark.parametrize("pad", [0, 1, 4, 16])
@pytest.mark.parametrize("M,N,K", E4M3_SHAPES)
def test_gemm_e4m3(M, N, K, pad):
    """Every kernel (few rows, tiles, K splits) at ragged sizes, with rows that
    start 16-byte aligned (pad to 16) and that do not; the bytes between rows
    hold NaN codes and are never read as values."""
    i = E4M3_SHAPES.index((M, N, K))
    name = ref.ACTS[i % len(ref.ACTS)]
    if pad in (0, 16):
        pad += -K % 16
    note(f"e4m3 {M}x{N}x{K} pad {pad} {name}")
    (a, A), (b, B) = codes(M, K, 2 * i, pad), codes(N, K, 2 * i + 1, pad)
    sa, sb = np.exp(normal(M, seed=3)), (np.exp(normal(N, seed=4)) / max(1, K) ** 0.5 / 5000).astype(np.float32)
    bias, R = normal(N, seed=5), normal(M, N, seed=6)
    out, ok = guarded(M, N)
    pre, ok_pre = guarded(M, N, pad=2)
    for ws in (True, False):
        sg.gemm_e4m3(a, dev(sa), b, dev(sb), bias=dev(bias), activation=name, residual=dev(R, pad % 3), out=out, pre=pre,
                     workspace=ws)
        torch.cuda.synchronize()
        # the two scale factors round once each
        x, y = A * sa.astype(np.float64)[:, None], (B * sb.astype(np.float64)[:, None]).T
        Y, Z, ty, tz = ref.product(x, y, K + 2, 1.0, bias.astype(np.float64), name, R.astype(np.float64))
        ref.within(f64(pre), Z, tz, "pre")
        ref.within(f64(out), Y, ty, "out")
        ok()
        ok_pre()


def test_gemm_e4m3_gradient_epilogue_and_plain():
    M, N, K = 90, 140, 300
    (a, A), (b, B) = codes(M, K, 1), codes(N, K, 2)
    y = sg.gemm_e4m3(a, None, b, None)
    Y, _, ty, _ = ref.product(A, B.T, K)
    ref.within(f64(y), Y, ty)
    Z0 = normal(M, N, seed=3)
    y = sg.gemm_e4m3(a, None, b, None, grad_pre=dev(Z0), activation="gelu")
    Y, _, ty, _ = ref.product(A, B.T, K, 1.0, None, "gelu", None, Z0.astype(np.float64))
    ref.within(f64(y), Y, ty)


def test_gemm_e4m3_nan_codes():
    """A NaN code spreads to its row (or column) of the result and no further."""
    for M, N, K in ((3, 50, 300), (100, 200, 300)):
        (a, _), (b, _) = codes(M, K, 1), codes(N, K, 2)
        a.view(torch.uint8)[1, 17] = 0x7f
        b.view(torch.uint8)[8, 250] = 0xff
        y = f64(sg.gemm_e4m3(a, None, b, None))
        bad = np.zeros((M, N), bool)
        bad[1] = True
        bad[:, 8] = True
        assert np.array_equal(np.isnan(y), bad)


# ---- far apart ---------------------------------------------------------------------------------------

def test_rows_further_apart_than_32_bits():
    """Row strides of 2^30 floats: the third row starts 2^33 bytes in.  Inputs
    and outputs of the row operators, and the epilogue's tensors."""
    M, D, ld = 3, 700, 1 << 30
    big = [torch.empty(2 * ld + D + 4, device="cuda") for _ in range(4)]

    def far(i, x=None):
        v = big[i][1:].as_strided((M, D), (ld, 1), 1)
        if x is not None:
            v.copy_(x)
        return v
    x, r, w = (dev(normal(*s, seed=i)) for i, s in enumerate(((M, D), (M, D), (D,))))
    y, s = sg.rmsnorm(x, w, residual=r)
    Y, S = sg.rmsnorm(far(0, x), w, residual=far(1, r), sum_out=far(2), out=far(3))
    assert torch.equal(Y, y) and torch.equal(S, s)
    q, c, _ = sg.rmsnorm_e4m3(x, w, residual=r)
    Q, C, S = sg.rmsnorm_e4m3(far(0, x), w, residual=far(1, r), sum_out=far(2))
    assert torch.equal(Q.float(), q.float()) and torch.equal(C, c) and torch.equal(S, s)
    d, dw = sg.rmsnorm_backward(y, s, w, dsum=r)
    Dx, Dw = sg.rmsnorm_backward(far(0, y), far(1, s), w, dsum=far(2, r), out=far(3))
    assert torch.equal(Dx, d) and torch.equal(Dw, dw)
    z, b = sg.activation_grad(x, r, "gelu")
    Z, B = sg.activation_grad(far(0, x), far(1, r), "gelu", out=far(2))
    assert torch.equal(Z, z) and torch.equal(B, b)
    K = 40
    A, Bm = normal(M, K, seed=5), normal(K, D, seed=6)
    pre, out = far(2), far(3)
    sg.sgemm_epilogue(dev(A), dev(Bm), activation="silu", residual=far(1, r), pre=pre, out=out)
    Yr, Zr, ty, tz = ref.product(A.astype(np.float64), Bm.astype(np.float64), K, 1.0, None, "silu", f64(r))
    ref.within(f64(pre), Zr, tz, "pre")
    ref.within(f64(out), Yr, ty, "out")
    sg.sgemm_epilogue(dev(A), dev(Bm), activation="silu", grad_pre=far(0, x), out=out)
    Yr, _, ty, _ = ref.product(A.astype(np.float64), Bm.astype(np.float64), K, 1.0, None, "silu", None, f64(x))
    ref.within(f64(out), Yr, ty, "gradient")


@pytest.mark.parametrize("M", [5, 70])
def test_codes_further_apart_than_32_bits(M):
    """8-bit rows whose last starts past 2^32 bytes, both operands in turn: the
    kernel of few rows and the tiles."""
    N, K = 70, 300
    ld = (1 << 32) // (M - 1) + 5
    (a, A), (b, B) = codes(M, K, 1), codes(N, K, 2)
    buf = torch.empty((M - 1) * ld + K, dtype=torch.uint8, device="cuda")
    far = buf.as_strided((M, K), (ld, 1))
    far.copy_(a.view(torch.uint8))
    far = far.view(torch.float8_e4m3fn)
    Y, _, ty, _ = ref.product(A, B.T, K)
    ref.within(f64(sg.gemm_e4m3(far, None, b, None)), Y, ty)
    ref.within(f64(sg.gemm_e4m3(b, None, far, None)).T, Y, ty)


def test_gemm_e4m3_more_columns_than_one_grid():
    """So many outputs that a workgroup's next column passes 2^31."""
    N = 1_620_000_000
    b = torch.randint(0, 0x78, (N, 1), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    one = torch.ones(1, 1, device="cuda").to(torch.float8_e4m3fn)
    y = sg.gemm_e4m3(one, None, b, None)
    for i in range(0, N, 1 << 28):
        assert torch.equal(y[0, i:i + (1 << 28)], b[i:i + (1 << 28), 0].float())


# ---- together ---------------------------------------------------------------------------------------

def test_training_block_together():
    """A residual block's forward and backward pass as a program makes it: norm,
    widening product with activation, narrowing product onto the residual
    stream, norm; every gradient against float64 autograd.  2e-5 of a
    gradient's norm is what chained float32 sums of up to 300 terms may leave."""
    T, D, F = 75, 96, 300
    x, w1, w2 = normal(T, D, seed=1), normal(D, F, seed=2, scale=D ** -0.5), normal(F, D, seed=3, scale=F ** -0.5)
    b1, b2, g1, g2 = normal(F, seed=4), normal(D, seed=5), 1 + 0.1 * normal(D, seed=6), 1 + 0.1 * normal(D, seed=7)
    G = normal(T, D, seed=8)
    X, W1, W2, B1, B2, G1, G2 = (dev(v.astype(np.float32)) for v in (x, w1, w2, b1, b2, g1, g2))
    # forward
    y1, _ = sg.rmsnorm(X, G1)
    pre = torch.empty(T, F, device="cuda")
    h = sg.sgemm_epilogue(y1, W1, bias=B1, activation="gelu", pre=pre)
    s = sg.sgemm_epilogue(h, W2, bias=B2, residual=X)
    y2, _ = sg.rmsnorm(s, G2)
    # backward of sum(G * y2) (+ the stream's own use below: none)
    ds, dg2 = sg.rmsnorm_backward(dev(G), s, G2)
    dpre, dW2, db2 = sg.sgemm_epilogue_backward(ds, h, W2, a_pre=pre, a_activation="gelu")
    dy1, dW1, db1 = sg.sgemm_epilogue_backward(dpre, y1, W1)
    dx, dg1 = sg.rmsnorm_backward(dy1, X, G1, dsum=ds)
    torch.cuda.synchronize()
    # float64 autograd
    t = [torch.from_numpy(v.astype(np.float32)).double().requires_grad_() for v in (x, w1, b1, w2, b2, g1, g2)]
    tx, tw1, tb1, tw2, tb2, tg1, tg2 = t

    def norm(v, g):
        return v / (v.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * g
    hh = torch.nn.functional.gelu(norm(tx, tg1) @ tw1 + tb1)
    ss = hh @ tw2 + tb2 + tx
    yy = norm(ss, tg2)
    (yy * torch.from_numpy(G).double()).sum().backward()
    for got, want in ((y2, yy.detach()), (dx, tx.grad), (dW1, tw1.grad), (db1, tb1.grad), (dW2, tw2.grad),
                      (db2, tb2.grad), (dg1, tg1.grad), (dg2, tg2.grad)):
        e = (got.cpu().double() - want).norm() / want.norm()
        assert e <= 2e-5, float(e)


def test_serving_block_together():
    """One token and a prompt through norm, 8-bit product, quantise, 8-bit
    product onto the stream: each step against 64 bits on what it was given."""
    D, F = 256, 640
    w1, w2 = normal(F, D, seed=1, scale=D ** -0.5), normal(D, F, seed=2, scale=F ** -0.5)
    q1, s1 = sg.quantize_e4m3(dev(w1))
    q2, s2 = sg.quantize_e4m3(dev(w2))
    for T in (1, 90):
        x, r, g = normal(T, D, seed=3), normal(T, D, seed=4), normal(D, seed=5)
        stream = dev(r)
        q, sc, s = sg.rmsnorm_e4m3(dev(x), dev(g), residual=stream, sum_out=stream)
        h = sg.gemm_e4m3(q, sc, q1, s1, activation="silu")
        qh, sh = sg.quantize_e4m3(h)
        y = sg.gemm_e4m3(qh, sh, q2, s2, residual=stream, out=stream)
        torch.cuda.synchronize()
        S = (x.astype(np.float64) + r)
        Y, _, ty, rho = ref.rmsnorm(x.astype(np.float64), g.astype(np.float64), 1e-6, r.astype(np.float64))
        ref.check_codes(f64(q.float()), f64(sc), Y, ty, rho + 8 * ref.U)
        a, b = f64(q.float()) * f64(sc)[:, None], (f64(q1.float()) * f64(s1)[:, None]).T
        H, _, th, _ = ref.product(a, b, D + 2, 1.0, None, "silu")
        ref.within(f64(h), H, th)
        a, b = f64(qh.float()) * f64(sh)[:, None], (f64(q2.float()) * f64(s2)[:, None]).T
        W, _, tw, _ = ref.product(a, b, F + 2, 1.0, None, "none", S)
        ref.within(f64(y), W, tw + ref.U * np.abs(S))


# ---- how they are called ------------------------------------------------------------------------------

def all_ops(seed=0):
    """Every operator once, at sizes that use workspaces; a dict of outputs."""
    A, B = dev(normal(70, 900, seed=seed)), dev(normal(900, 64, seed=seed + 1, scale=0.03))
    R, bias = dev(normal(70, 64, seed=seed + 2)), dev(normal(64, seed=seed + 3))
    pre = torch.empty(70, 64, device="cuda")
    o = {"y": sg.sgemm_epilogue(A, B, bias=bias, activation="gelu", residual=R, pre=pre), "pre": pre}
    o["dA"], o["dB"], o["db"] = sg.sgemm_epilogue_backward(R, A, B, pre=pre, activation="gelu")
    x, w = dev(normal(700, 520, seed=seed + 4)), dev(normal(520, seed=seed + 5))
    o["dz"], o["dzb"] = sg.activation_grad(x, x, "silu")
    o["n"], _ = sg.rmsnorm(x, w)
    o["dx"], o["dw"] = sg.rmsnorm_backward(x, x, w)
    q, s, _ = sg.rmsnorm_e4m3(x, w)
    o["q"], o["s"] = q.view(torch.uint8), s
    q2, s2 = sg.quantize_e4m3(x[:130])
    for m in (1, 20, 130):
        o[f"e{m}"] = sg.gemm_e4m3(q2[:m], s2[:m], q[:96], s[:96], bias=None, activation="silu")
    long = dev(normal(5, 20000, seed=seed + 6))
    o["ldx"], o["ldw"] = sg.rmsnorm_backward(long, long, long[0])
    return o


def test_reproducible_and_race_free():
    """The same bits again, and from the build that sets LDS to NaN before each
    refill."""
    a, b = all_ops(), all_ops()
    with sg.library(sg.POISON_LIB_PATH):
        c = all_ops()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k].contiguous().view(torch.uint8), b[k].contiguous().view(torch.uint8)), k
        assert torch.equal(a[k].contiguous().view(torch.uint8), c[k].contiguous().view(torch.uint8)), f"{k} (race check)"


def test_race_check_every_e4m3_kernel_and_epilogue_tile():
    """The race check build over each tile of the 8-bit product and of the
    epilogue product, bitwise equal to the normal build."""
    def run():
        out = []
        for M, N, K, pad in ((300, 600, 1000, 0), (300, 600, 999, 1), (100, 100, 2000, 0), (1100, 1030, 512, 0),
                             (2600, 2570, 300, 0), (5000, 4200, 256, 0), (40, 300, 700, 0)):
            (a, _), (b, _) = codes(M, K, 1, pad + (-K % 16 if not pad else 0)), codes(N, K, 2, pad + (-K % 16 if not pad else 0))
            out += [sg.gemm_e4m3(a, None, b, None, activation="silu", workspace=w) for w in (True, False)]
        for v in range(sg.sgemm_f32_num_variants()):
            if v in (0, 1, 2, 3, 8, 9):
                continue
            for name, kw in (("gelu", {}), ("silu", {"grad_pre": dev(normal(300, 330, seed=4))})):
                out.append(sg.sgemm_epilogue(dev(normal(300, 200, seed=1)), dev(normal(200, 330, seed=2)), activation=name,
                                             residual=dev(normal(300, 330, seed=3)), cfg=forced(v), **kw))
        return out
    a = run()
    with sg.library(sg.POISON_LIB_PATH):
        b = run()
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


def test_another_stream():
    """Work on a stream that is not torch's current one, inputs made on it and
    outputs used on it."""
    want = all_ops(3)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    x, w = dev(normal(700, 520, seed=7)), dev(normal(520, seed=8))
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = all_ops(3)
    st.synchronize()
    for k in want:
        assert torch.equal(want[k].contiguous().view(torch.uint8), got[k].contiguous().view(torch.uint8)), k
    # and named as an argument, while another stream is current
    y, _ = sg.rmsnorm(x, w, stream=st)
    q, s = sg.quantize_e4m3(x, stream=st)
    e = sg.gemm_e4m3(q[:100], s[:100], q, s, stream=st)
    d = sg.sgemm_epilogue_backward(x[:64], x[:64, :100], x[:100], pre=x[:64], activation="gelu", stream=st)
    st.synchronize()
    y2, _ = sg.rmsnorm(x, w)
    q2, s2 = sg.quantize_e4m3(x)
    e2 = sg.gemm_e4m3(q2[:100], s2[:100], q2, s2)
    d2 = sg.sgemm_epilogue_backward(x[:64], x[:64, :100], x[:100], pre=x[:64], activation="gelu")
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(e, e2) and all(torch.equal(p, r) for p, r in zip(d, d2))


def test_threads_on_their_streams():
    """Calls of four threads, each on a stream of its own, at the same time."""
    import threading
    A, B, x, w = (dev(normal(*s, seed=i)) for i, s in enumerate(((70, 300), (200, 300), (515, 2051), (2051,))))

    def calls():
        y = sg.sgemm_epilogue(A, B, activation="gelu", transb=True)
        q, scale = sg.quantize_e4m3(x)
        d, dw = sg.rmsnorm_backward(x, x, w)
        return [y, q.float(), scale, d, dw, *sg.sgemm_epilogue_backward(y, A, B, transb=True)]
    want = calls()
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for k in range(40):
                got = calls()
                stream.synchronize()
                if not all(torch.equal(g, v) for g, v in zip(got, want)):
                    bad.append((i, k))
            stream.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_graph_replays():
    """Every operator captured once and replayed, with eager calls of the same
    operators between the replays."""
    A, B = dev(normal(70, 900, seed=1)), dev(normal(900, 64, seed=2, scale=0.03))
    x, w, z = dev(normal(300, 520, seed=3)), dev(normal(520, seed=4)), dev(normal(70, 64, seed=5))
    qw, sw = sg.quantize_e4m3(dev(normal(200, 520, seed=6)))

    def step():
        pre = torch.empty(70, 64, device="cuda")
        y = sg.sgemm_epilogue(A, B, activation="gelu", residual=z, pre=pre)
        da, db, dbias = sg.sgemm_epilogue_backward(y, A, B, pre=pre, activation="gelu")
        q, s, _ = sg.rmsnorm_e4m3(x, w)
        e, e1 = sg.gemm_e4m3(q, s, qw, sw, activation="silu"), sg.gemm_e4m3(q[:1], s[:1], qw, sw)
        dx, dw = sg.rmsnorm_backward(x, x, w)
        n, _ = sg.activation_grad(x, None, None, out=False), None
        return [y, pre, da, db, dbias, e, e1, dx, dw, n[1]]
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        held = step()
    for r in range(4):
        x.copy_(dev(normal(300, 520, seed=20 + r)))
        A.copy_(dev(normal(70, 900, seed=30 + r)))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (r, i)
