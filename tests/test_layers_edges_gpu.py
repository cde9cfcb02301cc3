"""Operators of sgemm_layers.h at the ends of their ranges, against plain 64-bit
implementations with the bounds of layers_bounds.py."""
import numpy as np
import pytest
import torch

import fp32_gemm_sgemm_amd as sg
import layers_bounds as bounds
import layers_cases
import layers_ref
import ops_ref
from gpu_cases import note

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-5))


def normal(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape).astype(np.float32)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda")


def f64(t):
    return t.detach().cpu().double().numpy() if isinstance(t, torch.Tensor) else t.astype(np.float64)


# ---- layer norm -----------------------------------------------------------------------------------

@pytest.mark.parametrize("D", [5, 700, 1500, 3000, 6000, 9000, 17000])
def test_layernorm_rows_of_every_size(D):
    """Rows from 1e-3 to 1e36, far from zero, with one value of 1e30; every form."""
    note(f"layernorm {D}")
    s, w, b = bounds.rows_of(D), normal(D, seed=1), normal(D, seed=2)
    y, _ = sg.layernorm(dev(s), dev(w), dev(b))
    ops_ref.within(f64(y), *bounds.forward(f64(s), f64(w), f64(b), EPS))


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("D", [5, 700, 1500, 3000, 6000, 9000, 17000])
def test_layernorm_gradient_rows_of_every_size(D, stream):
    """The gradient of the same rows, whose third term is (1/sigma^2) d times a
    mean; then constant rows and rows that hold an infinity or NaN beside them."""
    note(f"layernorm_backward {D} stream={stream}")
    s = bounds.rows_of(D)
    dy, w = normal(*s.shape, seed=1), normal(D, seed=2)
    ds = normal(*s.shape, seed=3) if stream else None
    S, DY, W, DS = dev(s), dev(dy), dev(w), dev(ds) if stream else None
    dx, dw, db = sg.layernorm_backward(DY, S, W, dsum=DS)
    X, DW, DB, tx, tw, tb = bounds.backward(f64(dy), f64(s), f64(w), EPS, f64(ds) if stream else None)
    ops_ref.within(f64(dx), X, tx, "dx")
    ops_ref.within(f64(dw), DW, tw, "dw")
    ops_ref.within(f64(db), DB, tb, "db")
    S[0] = 3.0
    S[3, D // 2] = float("inf")
    S[6, D - 1] = float("nan")
    dx, _, _ = sg.layernorm_backward(DY, S, W, dsum=DS, need_weight=False, need_bias=False)
    keep = [i for i in range(len(s)) if i not in (3, 6)]
    X, _, _, tx, _, _ = bounds.backward(f64(dy)[keep], f64(S)[keep], f64(w), EPS, f64(ds)[keep] if stream else None)
    ops_ref.within(f64(dx)[keep], X, tx, "dx beside rows that are not finite")
    assert np.isnan(f64(dx)[[3, 6]]).all()


def test_layernorm_gradient_of_many_rows_of_every_size():
    """More than 512 rows of 4097 to 8192 values without sums have a form of their own."""
    D = 5000
    s, w = np.tile(bounds.rows_of(D), (60, 1)), normal(D, seed=2)
    dy = normal(*s.shape, seed=1)
    dx, dw, db = sg.layernorm_backward(dev(dy), dev(s), dev(w), need_weight=False, need_bias=False)
    assert dw is None and db is None
    X, _, _, tx, _, _ = bounds.backward(f64(dy), f64(s), f64(w), EPS)
    ops_ref.within(f64(dx), X, tx)


@pytest.mark.parametrize("D", [5, 700, 1500, 3000, 6000, 9000, 17000])
def test_layernorm_gradient_of_small_rows_without_eps(D):
    """r^3 of rows of 1e-20 and 1e-24 is past float32's range, r and dX are not."""
    s = normal(4, D, seed=1) * np.float32([[1e-20], [1e-24], [1e-15], [1.0]])
    dy, w = normal(4, D, seed=2), normal(D, seed=3)
    dx, _, _ = sg.layernorm_backward(dev(dy), dev(s), dev(w), eps=0.0)
    X, _, _, tx, _, _ = bounds.backward(f64(dy), f64(s), f64(w), 0.0)
    ops_ref.within(f64(dx), X, tx)
    s[1] = 7.0  # 0 / 0
    dx, _, _ = sg.layernorm_backward(dev(dy), dev(s), dev(w), eps=0.0)
    assert np.isnan(f64(dx)[1]).all() and np.isfinite(f64(dx)[[0, 2, 3]]).all()


@pytest.mark.parametrize("D", [64, 700, 2052, 5000, 9000, 20004])
def test_row_sums_are_float64(D):
    """Large values that cancel beside ones that count, in a thread's own sums."""
    s, t, dy = bounds.planted(D)
    y, _ = sg.layernorm(dev(s), eps=0.0)
    ops_ref.within(f64(y), *bounds.forward(f64(s), None, None, 0.0), "y")
    dx, _, _ = sg.layernorm_backward(dev(dy), dev(t), eps=0.0)
    X, _, _, tx, _, _ = bounds.backward(f64(dy), f64(t), None, 0.0)
    ops_ref.within(f64(dx), X, tx, "dx")


@pytest.mark.parametrize("D", [300, 1500, 3000, 6000, 9000, 20001])
def test_layernorm_onto_its_operands(D):
    """With weight and bias, to the bit: S onto X and onto R, Y onto X and onto R,
    both at once, and S in place beside codes."""
    rows = 9
    x, r = normal(rows, D, seed=1) + np.float32(2), normal(rows, D, seed=2)
    w, b = dev(normal(D, seed=3)), dev(normal(D, seed=4))
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    want, s = sg.layernorm(dev(x), w, b, residual=dev(r))
    q, scale, _ = sg.layernorm_e4m3(dev(x), w, b, residual=dev(r))
    alone, _ = sg.layernorm(dev(x), w, b)
    t = dev(x)
    y, same = sg.layernorm(t, w, b, out=t)
    assert y is t and same is t and torch.equal(t, alone)
    for onto in (0, 1):
        t = [dev(x), dev(r)]
        y, got = sg.layernorm(t[0], w, b, residual=t[1], sum_out=t[onto])
        assert got is t[onto] and torch.equal(got, s) and torch.equal(y, want), onto
        assert np.array_equal(t[1 - onto].cpu().numpy(), (r, x)[onto])
        t = [dev(x), dev(r)]
        kept = torch.empty(rows, D, device="cuda")
        y, got = sg.layernorm(t[0], w, b, residual=t[1], sum_out=kept, out=t[onto])
        assert y is t[onto] and torch.equal(y, want) and torch.equal(kept, s), onto
        t = [dev(x), dev(r)]
        y, got = sg.layernorm(t[0], w, b, residual=t[1], sum_out=t[onto], out=t[1 - onto])
        assert torch.equal(t[onto], s) and torch.equal(t[1 - onto], want), onto
        t = [dev(x), dev(r)]
        q2, scale2, got = sg.layernorm_e4m3(t[0], w, b, residual=t[1], sum_out=t[onto])
        assert torch.equal(got, s) and torch.equal(bits(q2), bits(q)) and torch.equal(scale2, scale), onto


# ---- the gated block of 8-bit operands ----------------------------------------------------------------

# one size for each 8-bit kernel, whole and with K split, aligned and not
E4M3_FORMS = list({(c[0], c[4], c[6] > 1, c[2] > 4080): c for c in layers_cases.E4M3_GATED}.values())


@pytest.mark.parametrize("case", E4M3_FORMS, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-" +
                         ("aligned" if c[4] else "any") + ("-split" if c[6] > 1 else ""))
def test_scales_whose_product_leaves_float32(case):
    """A row's scale and a column's act one after the other, as in the plain 8-bit
    product: 2^-100 and 2^-52 on sums of 2^23 and more leave values that
    float32 holds, 2^70 and 2^70 on a sum of zero leave zero."""
    _, M, N, K, aligned, workspace, _ = case
    note(f"gated e4m3 scales {case}")

    def rows(n, value):
        buf = torch.zeros(n, K if not aligned else -(-K // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")[:, :K]
        return buf.copy_(value[:, None].to(torch.float8_e4m3fn)) if n else buf
    m, n = torch.arange(M, device="cuda"), torch.arange(N, device="cuda")
    empty = m % 3 == 1  # rows of zeros, with the large scale
    a = rows(M, torch.where(empty, 0.0, 448.0))
    bg, bu = rows(N, torch.full((N,), 448.0, device="cuda")), rows(N, torch.where(n % 2 == 0, 448.0, -448.0))
    sa = torch.where(empty, 1.3 * 2.0 ** 70, 1.1 * 2.0 ** -100)
    s1 = torch.where(n % 2 == 0, 1.7 * 2.0 ** -52, 1.9 * 2.0 ** 70)
    s2 = torch.where(n % 3 == 0, 1.5 * 2.0 ** 70, 1.3 * 2.0 ** -52)
    G, U_, out = (torch.empty(M, N, device="cuda") for _ in range(3))
    total = 448.0 * 448.0 * K  # (a multiple of 2^12 below 2^36: exact in any order)

    def near(got, sign, scale, what):
        want = torch.where(empty, 0.0, total)[:, None].double() * sign.double() * sa.double()[:, None] * scale.double()
        off = (got.double() - want).abs() > want.abs() * (2 * bounds.U) + 2.0 ** -149
        assert not bool((off | got.isnan()).any()), (what, int(off.sum()), int(got.isnan().sum()))
    one, up = torch.ones(N, device="cuda"), torch.where(n % 2 == 0, 1.0, -1.0)
    sg.gemm_e4m3_gated(a, sa, bg, s1, bu, s2, activation="none", pre_gate=G, pre_up=U_, out=out, workspace=workspace)
    near(G, one, s1, "pre_gate")
    near(U_, up, s2, "pre_up")
    want = G.double() * U_.double()
    assert bool(((out.double() - want).abs() <= want.abs() * bounds.U + 2.0 ** -149).all())
    sg.gemm_e4m3_gated(a, sa, bg, None, bu, s2, activation="none", pre_gate=G, pre_up=U_, out=out, workspace=workspace)
    near(G, one, one, "pre_gate without a column scale")
    near(U_, up, s2, "pre_up beside it")


# ---- the gated block's gradient -------------------------------------------------------------------------

@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 3, 5), (33, 65, 40), (70, 130, 96), (129, 257, 65), (300, 64, 100)])
def test_gradient_of_weights_with_the_gate_second(M, N, K, tb, pad):
    """One tensor of both weights, the gate's the second half: the gradients are
    halves of one tensor in the weights' order."""
    note(f"gate second {M}x{N}x{K} tb={tb} pad={pad}")
    A, dy, G, U_ = normal(M, K, seed=1), normal(M, N, seed=2), normal(M, N, seed=3), normal(M, N, seed=4)
    hu, hg = (normal(*((N, K) if tb else (K, N)), seed=i) for i in (5, 6))
    host = np.concatenate([hu, hg], 0 if tb else 1)
    both = torch.zeros(host.shape[0], host.shape[1] + pad, device="cuda")[:, :host.shape[1]].copy_(dev(host))
    Bu, Bg = (both[:N], both[N:]) if tb else (both[:, :N], both[:, N:])
    got = sg.sgemm_gated_backward(dev(dy), dev(A), Bg, Bu, pre_gate=dev(G), pre_up=dev(U_), activation="silu", transb=tb)
    w = [f64(v) for v in (dy, A, G, U_)]
    wg, wu = (f64(hg.T), f64(hu.T)) if tb else (f64(hg), f64(hu))
    dA, dBg, dBu, ta, tg, tu = layers_ref.gated_backward(w[0], w[1], wg, wu, w[2], w[3], "silu")
    _, _, sums_g, sums_u, _, _, tsg, tsu = layers_ref.gated_grad(w[0], w[2], w[3], "silu")
    if tb:
        dBg, dBu, tg, tu = dBg.T, dBu.T, tg.T, tu.T
    for what, g, want, t in zip(("dA", "dB_gate", "dB_up", "dbias_gate", "dbias_up"), got, (dA, dBg, dBu, sums_g, sums_u),
                                (ta, tg, tu, tsg, tsu)):
        ops_ref.within(f64(g), want, t, what)
    step = got[1].data_ptr() - got[2].data_ptr()
    assert got[1].stride() == got[2].stride() and step == 4 * N * (K if tb else 1)
    for need in (("A",), ("B",), ("bias",)):
        part = sg.sgemm_gated_backward(dev(dy), dev(A), Bg, Bu, pre_gate=dev(G), pre_up=dev(U_), activation="silu",
                                       transb=tb, need=need)
        for x, y, name in zip(part, got, ("A", "B", "B", "bias", "bias")):
            assert (x is not None) == (name in need) and (x is None or torch.equal(x, y))


def stored(host, tb):
    """float64 K x N weights of stored ones."""
    return f64(host.T if tb else host)


@pytest.mark.parametrize("order", ["one tensor, gate second", "gate at the higher address", "the same weights"])
@pytest.mark.parametrize("tb", [False, True])
def test_weights_in_any_place(tb, order):
    """Forward in every form and backward with the gate's weights behind the other
    ones (a batch of the two has a negative stride), and with the two the same."""
    for M, N, K in ((70, 130, 96), (5, 260, 1100), (40, 2000, 50)):
        note(f"{order} {M}x{N}x{K} tb={tb}")
        shape = (N, K) if tb else (K, N)
        hu, hg = normal(*shape, seed=5) * np.float32(K ** -0.5), normal(*shape, seed=6) * np.float32(K ** -0.5)
        if order == "the same weights":
            hu = hg
            Bg = Bu = dev(hg)
        elif order == "gate at the higher address":
            buf = torch.zeros(2 * N * K + 8, device="cuda")
            Bu, Bg = buf[:N * K].view(shape), buf[N * K + 8:].view(shape)
            Bu.copy_(dev(hu))
            Bg.copy_(dev(hg))
        else:
            both = dev(np.concatenate([hu, hg], 0 if tb else 1))
            Bu, Bg = (both[:N], both[N:]) if tb else (both[:, :N], both[:, N:])
        A, dy, G, U_ = normal(M, K, seed=1), normal(M, N, seed=2), normal(M, N, seed=3), normal(M, N, seed=4)
        wg, wu = stored(hg, tb), stored(hu, tb)
        Y, _, _, ty, _, _ = layers_ref.gated(f64(A), wg, wu, K)
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        for form in (sg.GATED_AUTO, *range(8)):
            ops_ref.within(f64(sg.sgemm_gated(dev(A), Bg, Bu, transb=tb, form=form, workspace=ws)), Y, ty, f"form {form}")
        w = [f64(v) for v in (dy, A, G, U_)]
        dA, dBg, dBu, ta, tg, tu = layers_ref.gated_backward(w[0], w[1], wg, wu, w[2], w[3], "silu")
        if tb:
            dBg, dBu, tg, tu = dBg.T, dBu.T, tg.T, tu.T
        for space in (True, False, ws):
            got = sg.sgemm_gated_backward(dev(dy), dev(A), Bg, Bu, pre_gate=dev(G), pre_up=dev(U_), transb=tb, workspace=space)
            for what, g, want, t in zip(("dA", "dB_gate", "dB_up"), got, (dA, dBg, dBu), (ta, tg, tu)):
                ops_ref.within(f64(g), want, t, what)


# ---- norms over many tensors ------------------------------------------------------------------------------

@pytest.mark.parametrize("size", [2.0 ** 40, 1e30, 1e37])
@pytest.mark.parametrize("limit", [1e-5, 1e-10, 1e-25, 1e-37])
def test_clipping_by_factors_below_float32(size, limit):
    """The factor of large values and a small limit is below float32's normal
    range, or all of it; what it leaves of the values is not."""
    for shapes in ([(1000,)], [(3, 5), (70000,), (9, 4097), (2000, 17)], [(i % 7 + 1,) for i in range(300)]):
        host = [normal(*s, seed=i) * np.float32(size) for i, s in enumerate(shapes)]
        n = np.sqrt(sum((f64(x) ** 2).sum() for x in host))
        f = float(np.float32(limit)) / n
        xs, outs = [dev(x) for x in host], [torch.empty(s, device="cuda") for s in shapes]
        got = sg.clip_grad_norm(xs, limit, eps=0.0, out=outs)
        sg.clip_grad_norm(xs, limit, eps=0.0)
        assert n > 3.4e38 or abs(float(got) - n) <= 2 * bounds.U * n
        for x, o, h in zip(xs, outs, host):
            # the factor's rounding and the product's
            ops_ref.within(f64(o), f64(h) * f, np.abs(f64(h) * f) * (2.01 * bounds.U) + 2.0 ** -148)
            assert torch.equal(x, o)


def test_clipping_partly_in_place():
    """Some tensors are scaled onto themselves and some elsewhere in one call."""
    host = [normal(300, 70, seed=1), normal(5000, seed=2), normal(9, 11, seed=3)]
    xs = [dev(x) for x in host]
    outs = [xs[0], torch.empty(5000, device="cuda"), xs[2]]
    n = np.sqrt(sum((f64(x) ** 2).sum() for x in host))
    for limit, f in ((1e9, 1.0), (0.25, 0.25 / n)):
        sg.clip_grad_norm(xs, limit, eps=0.0, out=outs)
        for o, h in zip(outs, host):
            ops_ref.within(f64(o), f64(h) * f, np.abs(f64(h) * f) * (2.01 * bounds.U))
    assert np.array_equal(xs[1].cpu().numpy(), host[1])


def test_long_lists_in_graphs():
    """A list whose table goes to the workspace, captured: every replay scales what
    the memory holds then, as an eager call does; two graphs of one pool."""
    shapes = [(i % 13 + 1, i % 7 + 1) for i in range(230)] + [(70000,)]
    xs, outs = [torch.empty(s, device="cuda") for s in shapes], [torch.empty(s, device="cuda") for s in shapes]

    def fill(seed):
        for i, x in enumerate(xs):
            x.copy_(torch.from_numpy(normal(*x.shape, seed=1000 * seed + i)))
    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.clip_grad_norm(xs, 0.5, out=outs)
    torch.cuda.current_stream().wait_stream(side)
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        na = sg.clip_grad_norm(xs, 0.5, out=outs)
    with torch.cuda.graph(b, pool=a.pool()):
        nb = sg.clip_grad_norm(xs[::2], 0.25, out=outs[::2])
    for i in range(1, 4):
        fill(i)
        for graph, norm, part, limit in ((a, na, slice(None), 0.5), (b, nb, slice(None, None, 2), 0.25)):
            want = [torch.empty_like(x) for x in xs[part]]
            n = sg.clip_grad_norm(xs[part], limit, out=want)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(n, norm) and all(torch.equal(o, w) for o, w in zip(outs[part], want))
