"""The operators of sgemm_layers.h on the GPU against plain 64-bit
implementations (layers_ref.py), with bounds that count the roundings."""
import itertools
import threading

import numpy as np
import pytest
import torch

import fp32_gemm_sgemm_amd as sg
import layers_ref as ref
import ops_ref
from gpu_cases import note, place

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, scale=1.0, mean=0.0):
    return (np.random.default_rng(seed).standard_normal(shape) * scale + mean).astype(np.float32)


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
        assert bool((b == 77.0).all()), "memory outside the output was written"
    return view, check


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- layer norm -----------------------------------------------------------------------------------

# both sides of every form's limit (256, 512, 1024, 2048, 4096, 8192, 16384), odd widths
WIDTHS = [1, 2, 3, 5, 64, 100, 255, 257, 511, 513, 1000, 1025, 2047, 2049, 4095, 4100, 8191, 8193, 16383, 16385, 20003]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("D", WIDTHS)
def test_layernorm(D, residual):
    """Every form, rows padded and unaligned, with and without weight and bias,
    in float32 and as codes."""
    rows = 7 if D > 5000 else 23
    i = WIDTHS.index(D) + residual
    pad, shift = (0, 0) if i % 2 else (1, 1)
    note(f"layernorm {rows}x{D} residual={residual} pad {pad}")
    x, w, b = normal(rows, D, seed=1, mean=1.5), normal(D, seed=2) if i % 3 else None, normal(D, seed=3) if i % 4 else None
    r = normal(rows, D, seed=4) if residual else None
    out, ok = guarded(rows, D)
    so, ok_s = guarded(rows, D, pad=1)
    kw = {"residual": dev(r, pad, shift), "sum_out": so} if residual else {}
    tw, tb = (dev(v) if v is not None else None for v in (w, b))
    X = dev(x, pad, shift)
    y, s = sg.layernorm(X, tw, tb, eps=1e-4, out=out, **kw)
    q, scale, s8 = sg.layernorm_e4m3(X, tw, tb, eps=1e-4, residual=kw.get("residual"))
    torch.cuda.synchronize()
    assert y is out and s is (so if residual else X)
    S = x + r if residual else x
    assert np.array_equal(s.cpu().numpy(), S) and np.array_equal(s8.cpu().numpy(), S)
    Y, ty = ref.layernorm(S.astype(np.float64), None if w is None else w.astype(np.float64),
                          None if b is None else b.astype(np.float64), 1e-4)
    ops_ref.within(f64(out), Y, ty, "y")
    ok()
    ok_s()
    ops_ref.check_codes(f64(q.float()), f64(scale), Y, ty, ref.VAR_ERR)


@pytest.mark.parametrize("rows,D", [(600, 4097), (600, 8192), (300, 8200), (300, 16384), (2000, 64), (1030, 2000)])
@pytest.mark.parametrize("residual", [False, True])
def test_layernorm_many_rows(rows, D, residual):
    """Where workgroups of other sizes take over, and where a grid has several
    rows a workgroup."""
    note(f"layernorm {rows}x{D} residual={residual}")
    x, w, b, r = normal(rows, D, seed=1), normal(D, seed=2), normal(D, seed=3), normal(rows, D, seed=4)
    R = dev(r) if residual else None
    y, s = sg.layernorm(dev(x), dev(w), dev(b), residual=R)
    q, scale, _ = sg.layernorm_e4m3(dev(x), dev(w), dev(b), residual=R)
    torch.cuda.synchronize()
    S = (x + r if residual else x).astype(np.float64)
    Y, ty = ref.layernorm(S, w.astype(np.float64), b.astype(np.float64), 1e-5)
    ops_ref.within(f64(y), Y, ty)
    ops_ref.check_codes(f64(q.float()), f64(scale), Y, ty, ref.VAR_ERR)


@pytest.mark.parametrize("rows,D", [(512, 8192), (100, 16384), (300, 1000), (3, 20000)])
def test_layernorm_codes_are_the_formulas(rows, D):
    """Next to the border of two codes the formula's side: on float32 inputs
    everything up to the code's value is float64, so no code differs."""
    x, w, b = normal(rows, D, seed=1), 1 + 0.1 * normal(D, seed=2), 0.1 * normal(D, seed=3)
    q, scale, _ = sg.layernorm_e4m3(dev(x), dev(w), dev(b))
    t = dev(x).double()
    d = t - t.mean(1, keepdim=True)
    y = d / (d.pow(2).mean(1, keepdim=True) + np.float32(1e-5)).sqrt() * dev(w).double() + dev(b).double()
    s = y.abs().amax(1, keepdim=True) / 448
    want = (y / s).float().to(torch.float8_e4m3fn)
    differ = int((q.view(torch.uint8) != want.view(torch.uint8)).sum())
    assert differ == 0, f"{differ} of {x.size} codes differ"
    assert torch.equal(scale, s[:, 0].float())


def test_layernorm_in_place():
    """y on x; s on x or on the residual."""
    x, r, w, b = normal(31, 300, seed=1), normal(31, 300, seed=2), normal(300, seed=3), normal(300, seed=4)
    W, B = dev(w), dev(b)
    want, _ = sg.layernorm(dev(x), W, B)
    t = dev(x, 2)
    y, _ = sg.layernorm(t, W, B, out=t)
    assert y is t and torch.equal(t, want)
    want, s = sg.layernorm(dev(x), W, B, residual=dev(r))
    for D in (300, 20001):
        x, r = normal(9, D, seed=1), normal(9, D, seed=2)
        want, s = sg.layernorm(dev(x), residual=dev(r))
        for onto in (0, 1):
            t = [dev(x), dev(r)]
            y, got = sg.layernorm(t[0], residual=t[1], sum_out=t[onto])
            assert got is t[onto] and torch.equal(got, s) and torch.equal(y, want), (D, onto)


@pytest.mark.parametrize("D", [5, 700, 3000, 9000, 17000])
def test_layernorm_special_rows(D):
    """Constant rows, means far from zero, rows that hold infinities or NaN, large
    and tiny values; the other rows are as without them."""
    w, b = normal(D, seed=2), normal(D, seed=3)
    x = normal(9, D, seed=1)
    x[1] = 3.0
    x[2] += 1e6
    x[3, D // 2] = np.inf
    x[4, D - 1] = np.nan
    x[5] *= 1e15
    x[6] *= 1e-18
    x[7] = 0.0
    x[7, 0] = -1e30  # its squared distance from the mean is past float32's range
    X, W, B = dev(x), dev(w), dev(b)
    y, _ = sg.layernorm(X, W, B)
    q, scale, _ = sg.layernorm_e4m3(X, W, B)
    got, codes = f64(y), f64(q.float())
    for i in (0, 1, 2, 5, 6, 7, 8):
        Y, ty = ref.layernorm(x[i:i + 1].astype(np.float64), w.astype(np.float64), b.astype(np.float64), 1e-5)
        ops_ref.within(got[i:i + 1], Y, ty, f"row {i}")
        ops_ref.check_codes(codes[i:i + 1], f64(scale)[i:i + 1], Y, ty, ref.VAR_ERR)
    assert np.array_equal(got[1], b)  # a constant row is the bias
    assert np.isnan(got[3]).all() and np.isnan(got[4]).all()
    assert np.isnan(codes[3]).all() and np.isnan(codes[4]).all()
    # without eps a constant row is 0 / 0
    y, _ = sg.layernorm(X, eps=0.0)
    got = f64(y)
    assert np.isnan(got[1]).all()
    small = x[6:7] * np.float32(1e12)
    Y, ty = ref.layernorm(small.astype(np.float64), None, None, 0.0)
    t, _ = sg.layernorm(dev(small), eps=0.0)
    ops_ref.within(f64(t), Y, ty)


def test_layernorm_of_no_rows():
    x, w = torch.empty(0, 70, device="cuda"), torch.ones(70, device="cuda")
    y, s = sg.layernorm(x, w, w, residual=x)
    q, scale, _ = sg.layernorm_e4m3(x, w)
    dx, dw, db = sg.layernorm_backward(x, x, w)
    assert y.shape == s.shape == q.shape == dx.shape == (0, 70) and scale.shape == (0,)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    with pytest.raises(ValueError):
        sg.layernorm(torch.empty(3, 0, device="cuda"))


GRAD_CASES = [(D, 9 if D > 5000 else 37) for D in WIDTHS] + [(64, 3000), (300, 1), (2051, 515), (4096, 1100), (8000, 700)]


@pytest.mark.parametrize("D,rows", GRAD_CASES)
def test_layernorm_backward(D, rows):
    i = GRAD_CASES.index((D, rows))
    pad, shift = (0, 0) if i % 2 else (1, 1)
    note(f"layernorm_backward {rows}x{D} pad {pad}")
    dy, s, w = normal(rows, D, seed=1), normal(rows, D, seed=2, mean=0.7), normal(D, seed=3)
    ds = normal(rows, D, seed=4) if i % 3 else None
    weight = dev(w) if i % 5 else None
    out, ok = guarded(rows, D)
    dx, dw, db = sg.layernorm_backward(dev(dy, pad, shift), dev(s, pad, shift), weight, eps=1e-4,
                                       dsum=dev(ds) if ds is not None else None, out=out)
    torch.cuda.synchronize()
    X, DW, DB, tx, tw, tb = ref.layernorm_grad(dy.astype(np.float64), s.astype(np.float64),
                                               w.astype(np.float64) if weight is not None else None, 1e-4,
                                               ds.astype(np.float64) if ds is not None else None)
    assert dx is out
    ops_ref.within(f64(dx), X, tx, "dx")
    ok()
    if weight is None:
        assert dw is None
    else:
        ops_ref.within(f64(dw), DW, tw, "dw")
    ops_ref.within(f64(db), DB, tb, "db")


@pytest.mark.parametrize("rows,D", [(700, 8000), (40, 300), (6, 17000)])
def test_layernorm_backward_of_one_part(rows, D):
    """dx, dweight and dbias do not depend on what else is asked for; onto dsum."""
    dy, s, w, ds = (dev(normal(rows, D, seed=i)) for i in range(4))
    w = w[0].clone()
    dx, dw, db = sg.layernorm_backward(dy, s, w, dsum=ds)
    for nw, nb in itertools.product((False, True), repeat=2):
        a, b, c = sg.layernorm_backward(dy, s, w, dsum=ds, need_weight=nw, need_bias=nb)
        assert (b is not None) == nw and (c is not None) == nb
        # (without sums long rows go to other workgroups: other sums of the same terms)
        assert float((a - dx).abs().max()) <= 1e-4
        assert b is None or torch.equal(b, dw)
        assert c is None or torch.equal(c, db)
    t = ds.clone()
    a, _, _ = sg.layernorm_backward(dy, s, w, dsum=t, out=t)
    assert a is t and torch.equal(a, dx)


def test_layernorm_gradient_against_differences():
    """dx against central differences of the float32 forward pass in a direction:
    a step of 2^-7 leaves (2^-7)^2 of the third derivative and 2 U / 2^-7 of the
    forward's values, 1e-4 and 2e-5 of the norms in play."""
    rows, D = 5, 70
    s, w, b, dy, v = (normal(*shape, seed=i) for i, shape in enumerate([(rows, D), (D,), (D,), (rows, D), (rows, D)]))
    dx, _, _ = sg.layernorm_backward(dev(dy), dev(s), dev(w))
    h = 2.0 ** -7
    up, _ = sg.layernorm(dev((s + h * v).astype(np.float32)), dev(w), dev(b))
    down, _ = sg.layernorm(dev((s - h * v).astype(np.float32)), dev(w), dev(b))
    num = ((f64(up) - f64(down)) * dy).sum() / (2 * h)
    ana = (f64(dx) * v).sum()
    assert abs(num - ana) <= 2e-3 * np.linalg.norm(f64(dx)) * np.linalg.norm(v)


# ---- norms over many tensors -------------------------------------------------------------------------------

LISTS = {
    "one value": [(1,)],
    "a few": [(7,), (3, 5), ()],
    "little tensors": [(i % 37 + 1, i % 11 + 1) for i in range(90)],
    "as many as travel with a launch": [(17,)] * 96,
    "one more": [(17,)] * 97,
    "hundreds": [(i + 1,) for i in range(400)],
    "around a chunk": [(4095,), (4096,), (4097,), (8193,)],
    "long rows": [(3, 5000), (2, 4096), (9, 4097)],
    "narrow rows": [(5000, 1), (3000, 3), (1025, 5), (2000, 17)],
    "empty ones": [(0,), (3, 4), (0, 5), (5, 0)],
    "large": [(3000, 2051), (64, 64), (1 << 22,)],
    "three dimensions": [(4, 5, 6), (2, 300, 70)],
}


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("what", LISTS)
def test_clipping(what, padded):
    """The norm, and the tensors scaled to another list and in place; tensors as
    runs and with gaps between rows, which stay as they are."""
    shapes = LISTS[what]
    note(f"clip {what} padded={padded}")
    xs, bufs = [], []
    for i, shape in enumerate(shapes):
        x = normal(*shape, seed=i, scale=10.0 ** (-(i % 5))) if shape else np.float32(0.5)
        if padded and len(shape) == 2:
            buf = torch.full((shape[0], shape[1] + 1 + i % 4), 55.0, device="cuda")
            buf[:, :shape[1]] = torch.from_numpy(x)
            bufs.append((buf, shape[1]))
            xs.append(buf[:, :shape[1]])
        else:
            xs.append(torch.from_numpy(np.asarray(x)).to("cuda"))
    host = [t.cpu().numpy() for t in xs]
    n, f = ref.clip(host, 0.25, 1e-6)
    got = sg.grad_norm(xs)
    assert got.shape == () and got.is_cuda
    assert abs(float(got) - n) <= 2 * ref.U * n
    outs = [torch.empty(x.shape, device="cuda") for x in xs]
    got = sg.clip_grad_norm(xs, 0.25, out=outs)
    assert abs(float(got) - n) <= 2 * ref.U * n
    for x, h, o in zip(xs, host, outs):
        assert np.array_equal(x.cpu().numpy(), h), "an input was written"
        ops_ref.within(f64(o), h.astype(np.float64) * f, np.abs(h.astype(np.float64) * f) * 2 * ref.U + 1e-44)
    got = sg.clip_grad_norm(xs, 0.25)
    assert abs(float(got) - n) <= 2 * ref.U * n
    for x, o in zip(xs, outs):
        assert torch.equal(x, o)
    for buf, cols in bufs:
        assert bool((buf[:, cols:] == 55.0).all())


def test_clipping_below_the_limit():
    """A norm below max_norm leaves the values as they are, to the bit."""
    xs = [dev(normal(300, 70, seed=1)), dev(normal(9, seed=2))]
    before = [x.clone() for x in xs]
    outs = [torch.empty_like(x) for x in xs]
    n = sg.clip_grad_norm(xs, 1e9, out=outs)
    m = sg.clip_grad_norm(xs, 1e9)
    assert float(n) == float(m) > 0
    for x, b, o in zip(xs, before, outs):
        assert torch.equal(x, b) and torch.equal(o, b)


def test_clipping_special_values():
    """Squares past float32's range, values below it, limits of zero, norms of
    zero, infinities and NaN."""
    for scale in (1e30, 1e-30, 1e-40):
        x = (normal(1000, seed=1).astype(np.float64) * scale).astype(np.float32)
        n, f = ref.clip([x], scale, 0.0)
        out = torch.empty(1000, device="cuda")
        got = sg.clip_grad_norm([dev(x)], scale, eps=0.0, out=[out])
        assert abs(float(got) - n) <= 2 * ref.U * n + 1e-45
        ops_ref.within(f64(out), x.astype(np.float64) * f, np.abs(x.astype(np.float64) * f) * 4 * ref.U + 1e-44)
    x = dev(normal(5000, seed=2))
    assert bool((sg.clip_grad_norm([x], 0.0) > 0).all()) and bool((x == 0).all())
    z = torch.zeros(5000, device="cuda")
    assert float(sg.clip_grad_norm([z], 1.0)) == 0.0 and bool((z == 0).all())
    x = normal(5000, seed=3)
    x[77] = np.inf
    t = dev(x)
    assert float(sg.clip_grad_norm([t], 1.0)) == np.inf
    got = f64(t)
    assert np.isnan(got[77]) and (np.delete(got, 77) == 0).all()
    x[77] = np.nan
    t = dev(x)
    assert np.isnan(float(sg.clip_grad_norm([t], 1.0))) and np.isnan(f64(t)).all()


def test_clipping_halves_of_one_matrix():
    """The two column halves of one gradient, as sgemm_gated_backward gives
    them, are two tensors; overlapping ones and one named twice are refused."""
    both = dev(normal(50, 120, seed=1))
    whole = both.clone()
    a, b = both[:, :60], both[:, 60:]
    n = sg.clip_grad_norm([a, b], 0.5)
    m = sg.clip_grad_norm([whole], 0.5)
    assert abs(float(n) - float(m)) <= 2 * ref.U * float(m)
    assert float((both - whole).abs().max()) <= 2 * ref.U * float(whole.abs().max())
    assert abs(float(sg.grad_norm([a, a])) - np.sqrt(2) * float(sg.grad_norm([a]))) <= 1e-6
    for bad in ([both[:, :61], b], [a, a]):
        with pytest.raises(sg.SgemmError):
            sg.clip_grad_norm(bad, 0.5)


def test_norm_of_more_than_32_bits():
    """Element offsets past 2^31: every element counts."""
    free, _ = torch.cuda.mem_get_info()
    if free < 14 << 30:
        pytest.skip("too little memory")
    x = torch.zeros(2 ** 31 + 4099, device="cuda")
    x[-1] = 3.0
    x[2 ** 31 - 1] = 4.0
    assert float(sg.grad_norm([x])) == 5.0
    sg.clip_grad_norm([x], 1.0, eps=0.0)
    assert abs(float(x[-1]) - 0.6) < 1e-6 and abs(float(x[2 ** 31 - 1]) - 0.8) < 1e-6
    tall = x[:2 ** 31].view(2 ** 21, 1024)[:, :1023]
    tall[2 ** 21 - 1, 1022] = 1.0
    assert abs(float(sg.grad_norm([tall])) - 1.0) < 1e-6
