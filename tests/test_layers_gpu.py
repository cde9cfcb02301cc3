"""The operators of sgemm_layers.h on the GPU against plain 64-bit
implementations (layers_ref.py), with bounds that count the roundings."""
import itertools
import threading

import numpy as np
import pytest
import torch

import fp32_gemm_sgemm_amd as sg
import layers_cases
import layers_ref as ref
import ops_ref
from gpu_cases import note, place
from test_e4m3_kernels_gpu import codes as half_codes

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


# ---- the gated block ----------------------------------------------------------------------------------------

def weights(n, k, tb, merged, pad=0, shift=0, seed=0):
    """(device weights, float64 K x N ones): stored (n, k) or (k, n), as halves of
    one tensor or apart."""
    shape = (n, k) if tb else (k, n)
    host = [normal(*shape, seed=seed + h, scale=max(k, 1) ** -0.5) for h in range(2)]
    if merged:
        both = dev(np.concatenate(host, 0 if tb else 1), pad, shift)
        stored = (both[:n], both[n:]) if tb else (both[:, :n], both[:, n:])
    else:
        stored = tuple(dev(h, pad, shift) for h in host)
    return stored, [(h.T if tb else h).astype(np.float64) for h in host]


SHAPES = [(1, 1, 1), (1, 65, 130), (1, 1000, 64), (3, 40, 17), (2, 64, 5000), (16, 16, 64), (5, 7, 0), (33, 31, 257), (64, 64, 512),
          (70, 130, 96), (129, 257, 65), (260, 258, 100), (257, 512, 320)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("tb,merged", itertools.product((False, True), repeat=2))
def test_gated_shapes(M, N, K, tb, merged):
    """Both layouts, weights in one tensor or two, activations in turn, with
    biases and stored pre-activations, rows padded and unaligned."""
    i = SHAPES.index((M, N, K)) + 2 * tb + merged
    name = ops_ref.ACTS[i % 5]
    pad, shift = (0, 0) if i % 2 else (1, 1)
    note(f"gated {M}x{N}x{K} tb={tb} merged={merged} {name} pad {pad}")
    A = normal(M, K, seed=1)
    (Bg, Bu), (hg, hu) = weights(N, K, tb, merged, pad, shift, 2)
    bg, bu = normal(N, seed=5), normal(N, seed=6)
    out, ok = guarded(M, N)
    pg, ok_g = guarded(M, N, pad=5)
    pu, ok_u = guarded(M, N, pad=1)
    y = sg.sgemm_gated(dev(A, pad, shift), Bg, Bu, bias_gate=dev(bg), bias_up=dev(bu) if i % 3 else None, activation=name,
                       pre_gate=pg, pre_up=pu, out=out, transb=tb)
    torch.cuda.synchronize()
    assert y is out
    Y, G, U, ty, tg, tu = ref.gated(A.astype(np.float64), hg, hu, K, bg.astype(np.float64),
                                    bu.astype(np.float64) if i % 3 else None, name)
    ops_ref.within(f64(pg), G, tg, "pre_gate")
    ops_ref.within(f64(pu), U, tu, "pre_up")
    ops_ref.within(f64(out), Y, ty, "out")
    for check in (ok, ok_g, ok_u):
        check()


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("form", range(8))
def test_gated_every_form(form, tb):
    """Each form, forced, over several tiles with edges and slices that are cut,
    on rows that are 16-byte aligned and not; without biases or with one."""
    for M, N, K, pad in ((517, 330, 105, 0), (517, 330, 108, 4), (300, 201, 1, 0), (130, 140, 31, 1), (6, 260, 4200, 0),
                         (300, 256, 256, 0), (64, 32, 64, 0), (2, 40, 1500, 3), (257, 131, 33, 2)):
        name = ("gelu", "silu", "gelu_tanh", "relu")[(form + M) % 4]
        note(f"form {form} {M}x{N}x{K} tb={tb} pad {pad}")
        A = normal(M, K, seed=1)
        (Bg, Bu), (hg, hu) = weights(N, K, tb, bool(M % 2), pad, 0, 2)
        bias = normal(N, seed=5) if K % 2 else None
        out, ok = guarded(M, N, pad=M % 3)
        ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda") if form == sg.GATED_PRODUCTS else False
        sg.sgemm_gated(dev(A, pad), Bg, Bu, bias_up=dev(bias) if bias is not None else None, activation=name, out=out,
                       transb=tb, workspace=ws, form=form)
        torch.cuda.synchronize()
        Y, _, _, ty, _, _ = ref.gated(A.astype(np.float64), hg, hu, K, None,
                                      bias.astype(np.float64) if bias is not None else None, name)
        ops_ref.within(f64(out), Y, ty, f"form {form}")
        ok()


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 9])
def test_gated_few_rows(M, tb):
    """Each kernel for few rows: with and without K split over a workgroup's waves (K up from 1024, fewer than 8192
    columns), K staged once and several times, lengths that are no multiple of four, columns that a wave does not
    fill; the same bits from the build that sets LDS to NaN before each refill."""
    for N, K, pad in ((1, 1024, 0), (67, 1027, 1), (33, 1021, 0), (130, 4097, 3), (300, 9001, 0), (8195, 1026, 0), (515, 3, 1)):
        name = ops_ref.ACTS[(M + N) % 5]
        note(f"few rows {M}x{N}x{K} tb={tb} pad {pad}")
        A = normal(M, K, seed=1)
        (Bg, Bu), (hg, hu) = weights(N, K, tb, bool(N % 2), pad, 0, 2)
        bg, bu = normal(N, seed=5), normal(N, seed=6)
        Y, G, U, ty, tg, tu = ref.gated(A.astype(np.float64), hg, hu, K, bg.astype(np.float64), bu.astype(np.float64), name)
        a, b, c = dev(A, pad), dev(bg), dev(bu)
        out, ok = guarded(M, N)
        pg, ok_g = guarded(M, N, pad=5)
        pu, ok_u = guarded(M, N, pad=1)

        def call():
            sg.sgemm_gated(a, Bg, Bu, bias_gate=b, bias_up=c, activation=name, pre_gate=pg, pre_up=pu, out=out, transb=tb,
                           form=sg.GATED_ROWS)
            torch.cuda.synchronize()
        call()
        ops_ref.within(f64(pg), G, tg, "pre_gate")
        ops_ref.within(f64(pu), U, tu, "pre_up")
        ops_ref.within(f64(out), Y, ty, "out")
        for check in (ok, ok_g, ok_u):
            check()
        held = out.clone(), pg.clone(), pu.clone()
        with sg.library(sg.POISON_LIB_PATH):
            call()
        assert all(torch.equal(x, y) for x, y in zip((out, pg, pu), held)), "race check"


@pytest.mark.parametrize("tb", [False, True])
def test_gated_weights_of_unlike_strides(tb):
    """The two weights' rows are not the same distance apart; more workspace and
    none."""
    for M, N, K in ((70, 96, 1000), (3, 300, 257), (300, 260, 64)):
        A = normal(M, K, seed=1)
        (Bg, _), (hg, _) = weights(N, K, tb, False, 0, 0, 2)
        (_, Bu), (_, hu) = weights(N, K, tb, False, 7, 0, 2)
        Y, _, _, ty, _, _ = ref.gated(A.astype(np.float64), hg, hu, K)
        for form, ws in ((sg.GATED_AUTO, True), (sg.GATED_AUTO, False),
                         (sg.GATED_PRODUCTS, torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))):
            y = sg.sgemm_gated(dev(A), Bg, Bu, transb=tb, workspace=ws, form=form)
            ops_ref.within(f64(y), Y, ty, f"{M}x{N}x{K} form {form}")


def test_gated_of_nothing():
    """No rows, no columns; an empty sum leaves the biases, and 0 / 0 nothing."""
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    assert sg.sgemm_gated(e(0, 5), e(5, 7), e(5, 7)).shape == (0, 7)
    assert sg.sgemm_gated(e(3, 5), e(5, 0), e(5, 0)).shape == (3, 0)
    bg, bu = normal(7, seed=1), normal(7, seed=2)
    y = sg.sgemm_gated(e(3, 0), e(0, 7), e(0, 7), bias_gate=dev(bg), bias_up=dev(bu), activation="none")
    assert np.array_equal(y.cpu().numpy(), np.tile(bg * bu, (3, 1)))
    assert bool((sg.sgemm_gated(e(3, 0), e(7, 0), e(7, 0), transb=True) == 0).all())


def test_gated_special_values():
    """NaN and infinities go where the formula takes them and nowhere else."""
    M, N, K = 40, 50, 70
    A, (stored, host) = normal(M, K, seed=1), weights(N, K, True, True, 0, 0, 2)
    A[3, 5] = np.nan
    A[7, 0] = np.inf
    for form in range(8):
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda") if form == sg.GATED_PRODUCTS else False
        y = f64(sg.sgemm_gated(dev(A), *stored, transb=True, form=form, workspace=ws))
        assert np.isnan(y[3]).all(), form
        assert not np.isfinite(y[7]).any(), form
        rest = [i for i in range(M) if i not in (3, 7)]
        Y, _, _, ty, _, _ = ref.gated(A[rest].astype(np.float64), *host, K)
        ops_ref.within(y[rest], Y, ty, f"form {form}")


@pytest.mark.parametrize("tb", [False, True])
def test_gated_backward_of_unlike_strides(tb):
    """Two weight tensors whose rows are not the same distance apart, and sizes at
    which the two products of dA run together and one after the other; with a
    workspace, a little one and none."""
    for M, N, K, pad in ((70, 130, 96, 3), (40, 2000, 50, 0), (40, 2000, 50, 2), (600, 700, 600, 0)):
        A, dy, G, U = normal(M, K, seed=1), normal(M, N, seed=2), normal(M, N, seed=3), normal(M, N, seed=4)
        (Bg, _), (hg, _) = weights(N, K, tb, False, 0, 0, 5)
        (_, Bu), (_, hu) = weights(N, K, tb, False, pad, 0, 5)
        w = [v.astype(np.float64) for v in (dy, A, G, U)]
        dA, dBg, dBu, ta, tg, tu = ref.gated_backward(w[0], w[1], hg, hu, w[2], w[3], "silu")
        if tb:
            dBg, dBu, tg, tu = dBg.T, dBu.T, tg.T, tu.T
        for ws in (True, False, torch.empty(1 << 12, dtype=torch.uint8, device="cuda"),
                   torch.empty(1 << 26, dtype=torch.uint8, device="cuda")):
            got = sg.sgemm_gated_backward(dev(dy), dev(A), Bg, Bu, pre_gate=dev(G), pre_up=dev(U), transb=tb, workspace=ws)
            for what, g, want, t in zip(("dA", "dB_gate", "dB_up"), got, (dA, dBg, dBu), (ta, tg, tu)):
                ops_ref.within(f64(g), want, t, f"{what} {M}x{N}x{K}")


GRAD_SHAPES = [(1, 1, 1), (1, 300, 65), (5, 3, 40), (70, 130, 96), (129, 257, 65), (300, 64, 100), (33, 1030, 20)]


@pytest.mark.parametrize("M,N,K", GRAD_SHAPES)
@pytest.mark.parametrize("tb,merged", itertools.product((False, True), repeat=2))
def test_gated_backward(M, N, K, tb, merged):
    i = GRAD_SHAPES.index((M, N, K)) + 2 * tb + merged
    name = ops_ref.ACTS[i % 5]
    pad = i % 3
    note(f"gated_backward {M}x{N}x{K} tb={tb} merged={merged} {name} pad {pad}")
    A, dy, G, U = normal(M, K, seed=1), normal(M, N, seed=2), normal(M, N, seed=3, scale=2.0), normal(M, N, seed=4)
    (Bg, Bu), (hg, hu) = weights(N, K, tb, merged, pad, 0, 5)
    got = sg.sgemm_gated_backward(dev(dy, pad), dev(A, pad), Bg, Bu, pre_gate=dev(G, pad), pre_up=dev(U), activation=name,
                                  transb=tb)
    torch.cuda.synchronize()
    w = [v.astype(np.float64) for v in (dy, A, G, U)]
    _, _, BG, BU, _, _, tbg, tbu = ref.gated_grad(w[0], w[2], w[3], name)
    dA, dBg, dBu, ta, tg, tu = ref.gated_backward(w[0], w[1], hg, hu, w[2], w[3], name)
    if tb:
        dBg, dBu, tg, tu = dBg.T, dBu.T, tg.T, tu.T
    for what, g, want, t in zip(("dA", "dB_gate", "dB_up", "dbias_gate", "dbias_up"), got, (dA, dBg, dBu, BG, BU),
                                (ta, tg, tu, tbg, tbu)):
        ops_ref.within(f64(g), want, t, what)
    if merged and M * N * K > 1:
        # one tensor's halves, as the weights are
        step = got[2].data_ptr() - got[1].data_ptr()
        assert step == 4 * N * (got[1].stride(0) if tb else 1)
    for need in (("A",), ("B",), ("bias",), ()):
        part = sg.sgemm_gated_backward(dev(dy, pad), dev(A, pad), Bg, Bu, pre_gate=dev(G, pad), pre_up=dev(U),
                                       activation=name, transb=tb, need=need)
        for x, y, n in zip(part, got, ("A", "B", "B", "bias", "bias")):
            assert (x is not None) == (n in need)
            assert x is None or torch.equal(x, y)


@pytest.mark.parametrize("M,N,K", [(0, 5, 7), (5, 0, 7), (5, 7, 0)])
@pytest.mark.parametrize("tb", [False, True])
def test_gated_backward_of_nothing(M, N, K, tb):
    z = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    B = z(N, K) if tb else z(K, N)
    dA, dBg, dBu, bg, bu = sg.sgemm_gated_backward(z(M, N), z(M, K), B, B.clone(), pre_gate=z(M, N), pre_up=z(M, N),
                                                   activation="none", transb=tb)
    assert dA.shape == (M, K) and dBg.shape == dBu.shape == B.shape and bg.shape == bu.shape == (N,)
    if N == 0:
        assert bool((dA == 0).all())
    if M == 0:
        assert all(bool((t == 0).all()) for t in (dBg, dBu, bg, bu))


@pytest.mark.parametrize("M,N", [(1, 1), (3, 300), (1000, 7), (513, 130), (70, 2051), (5000, 64)])
def test_gated_grad(M, N):
    """Every activation; to other tensors, to the halves of one and in place."""
    for i, name in enumerate(ops_ref.ACTS):
        dy, G, U = normal(M, N, seed=1), normal(M, N, seed=2, scale=3.0), normal(M, N, seed=3)
        want = ref.gated_grad(*(v.astype(np.float64) for v in (dy, G, U)), name)
        og, ok_g = guarded(M, N)
        ou, ok_u = guarded(M, N, pad=1)
        got = sg.gated_grad(dev(dy, i % 2), dev(G, i % 3), dev(U), name, out_gate=og, out_up=ou)
        for what, g, w, t in zip(("dG", "dU", "dbias_gate", "dbias_up"), got, want[:4], want[4:]):
            ops_ref.within(f64(g), w, t, f"{name} {what}")
        ok_g()
        ok_u()
        both = torch.empty(M, 2 * N, device="cuda")
        sg.gated_grad(dev(dy), dev(G), dev(U), name, out_gate=both[:, :N], out_up=both[:, N:], dbias_gate=False,
                      dbias_up=False)
        assert torch.equal(both[:, :N], got[0]) and torch.equal(both[:, N:], got[1])
        y, g, u = dev(dy), dev(G), dev(U)
        a, b, bias, none = sg.gated_grad(y, g, u, name, out_gate=u, out_up=g, dbias_up=False)
        assert a is u and b is g and none is None
        assert torch.equal(u, got[0]) and torch.equal(g, got[1]) and torch.equal(bias, got[2])
        a, b, _, bias = sg.gated_grad(y, dev(G), dev(U), name, out_gate=False, out_up=y, dbias_gate=False)
        assert a is None and b is y and torch.equal(y, got[1]) and torch.equal(bias, got[3])


def test_gated_gradients_against_differences():
    """The gradients against central differences of the float32 forward pass in
    a direction: a step of 2^-7 leaves (2^-7)^2 of the third derivative and
    2 K U / 2^-7 of the forward's values, below 2e-3 of the norms in play."""
    M, N, K, h = 9, 20, 15, 2.0 ** -7
    base = [normal(M, K, seed=1), normal(K, N, seed=2, scale=0.3), normal(K, N, seed=3, scale=0.3), normal(N, seed=4),
            normal(N, seed=5)]
    dy = normal(M, N, seed=6)
    for name in ("gelu", "gelu_tanh", "silu", "none"):
        def forward(args):
            a, bg, bu, x, y = (dev(v.astype(np.float32)) for v in args)
            return f64(sg.sgemm_gated(a, bg, bu, bias_gate=x, bias_up=y, activation=name))
        t = [dev(v) for v in base]
        pg, pu = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        sg.sgemm_gated(*t[:3], bias_gate=t[3], bias_up=t[4], activation=name, pre_gate=pg, pre_up=pu)
        got = sg.sgemm_gated_backward(dev(dy), *t[:3], pre_gate=pg, pre_up=pu, activation=name)
        for k in range(5):
            v = normal(*base[k].shape, seed=10 + k)
            up, down = list(base), list(base)
            up[k], down[k] = base[k] + h * v, base[k] - h * v
            num = ((forward(up) - forward(down)) * dy).sum() / (2 * h)
            ana = (f64(got[k]) * v).sum()
            assert abs(num - ana) <= 2e-3 * np.linalg.norm(f64(got[k])) * np.linalg.norm(v), (name, k)


# ---- the gated block of 8-bit operands -------------------------------------------------------------------------

def codes(rows, cols, seed, pad=0):
    """(8-bit device rows with their scales, the float64 values they stand for)."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (rows, cols), dtype=np.uint8)
    c[(c & 127) == 127] = 0  # no NaN
    buf = torch.zeros(rows, cols + pad, dtype=torch.uint8, device="cuda")
    buf[:, :cols] = torch.from_numpy(c)
    s = (2.0 ** rng.integers(-9, -5, rows)).astype(np.float32)
    q = buf.view(torch.float8_e4m3fn)[:, :cols] if rows * cols else torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    return q, dev(s), ops_ref.E4M3[c] * s[:, None].astype(np.float64)


# one of each kernel (streaming for 16, 32 and 64 rows; four tiles, whole and as two K-split products; rows that
# are not 16-byte aligned), slices that are cut, fewer slices than stages
E4M3_SHAPES = [(1, 1, 1), (1, 130, 70), (16, 257, 1030), (7, 40, 8000), (17, 300, 300), (33, 40, 500), (64, 64, 512), (5, 7, 0),
               (70, 130, 96), (129, 257, 65), (260, 258, 100), (257, 512, 320), (100, 64, 9000), (200, 100, 20000),
               (1100, 1030, 512), (2600, 2570, 300), (4100, 2200, 128)]


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("M,N,K", E4M3_SHAPES)
def test_gemm_e4m3_gated(M, N, K, pad):
    pad += -(K + pad) % 16 if not pad else 0
    i = E4M3_SHAPES.index((M, N, K))
    name = ops_ref.ACTS[i % 5]
    note(f"e4m3 gated {M}x{N}x{K} pad {pad} {name}")
    (a, sa, A), (b, sb, Bg), (c, sc, Bu) = (codes(r, K, s, pad) for r, s in ((M, 1), (N, 2), (N, 3)))
    bg, bu = normal(N, seed=5), normal(N, seed=6)
    small = M * N <= 1 << 18
    pg, ok_g = guarded(M, N) if small else (None, None)
    pu, ok_u = guarded(M, N, pad=1) if small else (None, None)
    Y, G, U, ty, tg, tu = ref.gated(A, Bg.T, Bu.T, K + 3, bg.astype(np.float64), bu.astype(np.float64), name)
    for ws in (True, False):
        out, ok = guarded(M, N)
        sg.gemm_e4m3_gated(a, sa, b, sb, c, sc, bias_gate=dev(bg), bias_up=dev(bu), activation=name, pre_gate=pg, pre_up=pu,
                           out=out, workspace=ws)
        torch.cuda.synchronize()
        ops_ref.within(f64(out), Y, ty, f"out, workspace {ws}")
        ok()
        if small:
            ops_ref.within(f64(pg), G, tg, "pre_gate")
            ops_ref.within(f64(pu), U, tu, "pre_up")
            ok_g()
            ok_u()
    # without scales or biases
    Y, _, _, ty, _, _ = ref.gated(A / f64(sa)[:, None], Bg.T / f64(sb), Bu.T, K + 3, None, None, name)
    y = sg.gemm_e4m3_gated(a, None, b, None, c, sc, activation=name)
    ops_ref.within(f64(y), Y, ty, "no scales")


@pytest.mark.parametrize("case", layers_cases.E4M3_GATED, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-" +
                         ("aligned" if c[4] else "any") + ("-split" if c[6] > 1 else ""))
def test_each_gated_e4m3_kernel(case):
    """Each kernel with every part of its epilogue against 64 bits, and the same
    bits from the build that sets LDS to NaN before each refill.  The codes are
    multiples of 1/2 up to 8: products are multiples of 1/4 up to 64, so up to
    2^16 of them add to an exact float32 in any order, and only the epilogue's
    roundings are left."""
    _, M, N, K, aligned, workspace, _ = case
    note(f"gated e4m3 {case}")
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256
    i = layers_cases.E4M3_GATED.index(case)
    gen = torch.Generator(device="cuda").manual_seed(i)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    # rows that are not aligned: those of A, of the gate's weights or of the other half's, by stride or start
    off = None if aligned else i % 3
    a, bg, bu = (half_codes(r, K, off != j, 3 if off == j and i % 2 else 0, gen) for j, r in enumerate((M, N, N)))
    sa, sg_, su = torch.exp(rand(M)), torch.exp(rand(N)) / (10 * K ** 0.5), torch.exp(rand(N)) / (10 * K ** 0.5)
    bias_g, bias_u = rand(N), rand(N)
    out, ok = guarded(M, N)
    pg, ok_g = guarded(M, N, pad=2)
    pu, ok_u = guarded(M, N, pad=1)

    def call():
        sg.gemm_e4m3_gated(a, sa, bg, sg_, bu, su, bias_gate=bias_g, bias_up=bias_u, activation="silu", pre_gate=pg,
                           pre_up=pu, out=out, workspace=workspace)

    def half(b, scale, bias):
        s = torch.mm(a.float().double(), b.float().double().T.contiguous()).mul_(sa.double()[:, None]).mul_(scale.double())
        t = s.abs() * (2 * ops_ref.U)  # two scale factors
        s += bias.double()
        return s, t.add_(s.abs() * ops_ref.U).add_(1e-37)

    def near(got, want, bound, what):
        off = (got.double() - want).abs_() > bound
        assert not bool((off | torch.isnan(got)).any()), (what, int(off.sum()), torch.nonzero(off)[:1].tolist())
    call()
    torch.cuda.synchronize()
    ok(), ok_g(), ok_u()
    g, tg = half(bg, sg_, bias_g)
    near(pg, g, tg, "pre_gate")
    act = g * torch.sigmoid(g)
    ta = tg.mul_(ops_ref.LIPSCHITZ).add_(g.abs_() * ops_ref.ACT_ERR)
    del g
    u, tu = half(bu, su, bias_u)
    near(pu, u, tu, "pre_up")
    # (ta tu: both factors off at once)
    y, ty = act * u, ta * u.abs() + act.abs() * tu + ta * tu
    near(out, y, ty + ops_ref.U * y.abs() + 1e-37, "out")
    del act, ta, u, tu, y, ty
    held = out.clone(), pg.clone(), pu.clone()
    with sg.library(sg.POISON_LIB_PATH):
        call()
        assert all(torch.equal(x, y) for x, y in zip((out, pg, pu), held)), "race check"


def test_gemm_e4m3_gated_nan_codes():
    """A NaN code reaches its row or its columns, whatever kernel."""
    for M, N, K in ((1, 40, 200), (40, 50, 300), (300, 260, 128)):
        (a, sa, _), (b, sb, _), (c, sc, _) = (codes(r, K, s) for r, s in ((M, 1), (N, 2), (N, 3)))
        c.view(torch.uint8)[N // 2, K // 2] = 0x7f
        y = f64(sg.gemm_e4m3_gated(a, sa, b, sb, c, sc))
        assert np.isnan(y[:, N // 2]).all() and np.isfinite(np.delete(y, N // 2, 1)).all()


# ---- together ----------------------------------------------------------------------------------------------------

def test_training_layer_together():
    """A layer's forward and backward pass as a program makes them: layer norm,
    gated block, narrowing product onto the residual stream, layer norm; every
    gradient against float64 autograd, then all of them clipped.  2e-5 of a
    gradient's norm is what chained float32 sums of up to 300 terms may leave."""
    T, D, F = 75, 96, 300
    host = [normal(T, D, seed=1), normal(D, 2 * F, seed=2, scale=D ** -0.5), normal(F, D, seed=3, scale=F ** -0.5),
            normal(2 * F, seed=4), normal(D, seed=5), 1 + 0.1 * normal(D, seed=6), 0.1 * normal(D, seed=7),
            1 + 0.1 * normal(D, seed=8), 0.1 * normal(D, seed=9)]
    X, W1, W2, B1, B2, G1, C1, G2, C2 = (dev(v.astype(np.float32)) for v in host)
    G = normal(T, D, seed=10)
    # forward
    y1, _ = sg.layernorm(X, G1, C1)
    pre = torch.empty(T, 2 * F, device="cuda")
    h = sg.sgemm_gated(y1, W1[:, :F], W1[:, F:], bias_gate=B1[:F], bias_up=B1[F:], activation="silu", pre_gate=pre[:, :F],
                       pre_up=pre[:, F:])
    s = sg.sgemm_epilogue(h, W2, bias=B2, residual=X)
    y2, _ = sg.layernorm(s, G2, C2)
    # backward of sum(G * y2)
    ds, dg2, dc2 = sg.layernorm_backward(dev(G), s, G2)
    dh, dW2, db2 = sg.sgemm_epilogue_backward(ds, h, W2)
    dy1, dWg, dWu, dbg, dbu = sg.sgemm_gated_backward(dh, y1, W1[:, :F], W1[:, F:], pre_gate=pre[:, :F], pre_up=pre[:, F:])
    dx, dg1, dc1 = sg.layernorm_backward(dy1, X, G1, dsum=ds)
    grads = [dWg, dWu, dW2, dbg, dbu, db2, dg1, dc1, dg2, dc2]
    before = [g.clone() for g in grads]
    norm = sg.clip_grad_norm(grads, 0.5)
    torch.cuda.synchronize()
    # float64 autograd
    t = [torch.from_numpy(v.astype(np.float32)).double().requires_grad_() for v in host]
    x, w1, w2, b1, b2, g1, c1, g2, c2 = t

    def ln(v, g, c):
        d = v - v.mean(1, keepdim=True)
        return d / (d.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * g + c
    z = ln(x, g1, c1) @ w1 + b1
    yy = ln(torch.nn.functional.silu(z[:, :F]) * z[:, F:] @ w2 + b2 + x, g2, c2)
    (yy * torch.from_numpy(G).double()).sum().backward()
    want = [w1.grad[:, :F], w1.grad[:, F:], w2.grad, b1.grad[:F], b1.grad[F:], b2.grad, g1.grad, c1.grad, g2.grad, c2.grad]
    for got, w in [(y2, yy.detach()), (dx, x.grad), *zip(before, want)]:
        e = (got.cpu().double() - w).norm() / w.norm()
        assert e <= 2e-5, float(e)
    n = torch.cat([w.reshape(-1) for w in want]).norm()
    assert abs(float(norm) - float(n)) <= 2e-5 * float(n) and float(n) > 0.5
    for g, b in zip(grads, before):
        assert float((g - b * (0.5 / float(norm))).abs().max()) <= 4 * ref.U * float(b.abs().max())


def test_serving_layer_together():
    """One token and a prompt through layer norm to 8 bits, the gated 8-bit block,
    rows to 8 bits and an 8-bit product onto the stream: each step against 64
    bits on what it was given."""
    D, F = 256, 640
    (qg, sgt), (qu, su), (q2, s2) = (sg.quantize_e4m3(dev(normal(*s, seed=i, scale=s[1] ** -0.5)))
                                     for i, s in enumerate(((F, D), (F, D), (D, F))))
    value = lambda q, s: f64(q.float()) * f64(s)[:, None]  # noqa: E731
    for T in (1, 90):
        x, r, g, b = normal(T, D, seed=3), normal(T, D, seed=4), normal(D, seed=5), normal(D, seed=6)
        stream = dev(r)
        q, sc, s = sg.layernorm_e4m3(dev(x), dev(g), dev(b), residual=stream, sum_out=stream)
        h = sg.gemm_e4m3_gated(q, sc, qg, sgt, qu, su)
        qh, sh = sg.quantize_e4m3(h)
        y = sg.gemm_e4m3(qh, sh, q2, s2, residual=stream, out=stream)
        torch.cuda.synchronize()
        S = (x + r).astype(np.float64)
        Y, ty = ref.layernorm(S, g.astype(np.float64), b.astype(np.float64), 1e-5)
        ops_ref.check_codes(f64(q.float()), f64(sc), Y, ty, ref.VAR_ERR)
        H, _, _, th, _, _ = ref.gated(value(q, sc), value(qg, sgt).T, value(qu, su).T, D + 3)
        ops_ref.within(f64(h), H, th)
        W, _, tw, _ = ops_ref.product(value(qh, sh), value(q2, s2).T, F + 2, 1.0, None, "none", S)
        ops_ref.within(f64(y), W, tw + ref.U * np.abs(S))


# ---- how they are called ------------------------------------------------------------------------------------------

def all_ops(seed=0):
    """Every operator once, at sizes that use workspaces; a dict of outputs."""
    A = dev(normal(70, 900, seed=seed))
    (Bg, Bu), _ = weights(130, 900, False, True, 0, 0, seed + 1)
    (Tg, Tu), _ = weights(64, 900, True, False, 0, 0, seed + 3)
    pg, pu = torch.empty(70, 130, device="cuda"), torch.empty(70, 130, device="cuda")
    o = {"g": sg.sgemm_gated(A, Bg, Bu, activation="gelu", pre_gate=pg, pre_up=pu), "pg": pg, "pu": pu}
    for m in (1, 2, 4):
        o[f"r{m}"] = sg.sgemm_gated(A[:m], Bg, Bu)
        o[f"t{m}"] = sg.sgemm_gated(A[:m], Tg, Tu, transb=True)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    for form in range(8):
        o[f"f{form}"] = sg.sgemm_gated(A, Tg, Tu, transb=True, form=form, workspace=ws)
        o[f"x{form}"] = sg.sgemm_gated(A, Bg, Bu, form=form, workspace=ws)
    o["dA"], o["dBg"], o["dBu"], o["bg"], o["bu"] = sg.sgemm_gated_backward(pg, A, Bg, Bu, pre_gate=pg, pre_up=pu)
    x, w = dev(normal(700, 520, seed=seed + 5)), dev(normal(520, seed=seed + 6))
    o["n"], _ = sg.layernorm(x, w, w)
    o["dx"], o["dw"], o["db"] = sg.layernorm_backward(x, x, w)
    q, s, _ = sg.layernorm_e4m3(x, w, w)
    o["q"], o["s"] = q.view(torch.uint8), s
    for m in (1, 20, 50, 130, 300):
        o[f"e{m}"] = sg.gemm_e4m3_gated(q[:m], s[:m], q[:96], s[:96], q[96:192], s[96:192])
    o["ek"] = sg.gemm_e4m3_gated(*(t for n in (100, 48, 48) for t in sg.quantize_e4m3(dev(normal(n, 9000, seed=seed + n)))))
    for D in (200, 1500, 5000, 9000, 20000):
        t = dev(normal(5, D, seed=seed + 7))
        o[f"n{D}"], _ = sg.layernorm(t, t[0])
        o[f"q{D}"] = sg.layernorm_e4m3(t, t[0])[0].view(torch.uint8)
        o[f"dx{D}"], o[f"dw{D}"], o[f"db{D}"] = sg.layernorm_backward(t, t, t[0])
    xs = [x.clone(), w.clone(), t.clone()]
    o["norm"] = sg.clip_grad_norm(xs, 0.5)
    o["c0"], o["c1"], o["c2"] = xs
    o["one"] = sg.grad_norm([w])
    o["many"] = sg.grad_norm([w] * 100)
    return o


def same(a, b, what=""):
    for k in a:
        assert torch.equal(a[k].contiguous().reshape(-1).view(torch.uint8), b[k].contiguous().reshape(-1).view(torch.uint8)), (k, what)


def test_reproducible_and_race_free():
    """The same bits again, and from the build that sets LDS to NaN before each
    refill."""
    a, b = all_ops(), all_ops()
    same(a, b)
    with sg.library(sg.POISON_LIB_PATH):
        c = all_ops()
    torch.cuda.synchronize()
    same(a, c, "race check")


def test_race_check_of_every_8_bit_gated_kernel():
    def run():
        out = {}
        for i, (M, N, K) in enumerate(((300, 600, 1000), (100, 64, 9000), (1100, 1030, 512), (2600, 2570, 300), (40, 300, 700))):
            for pad in (-K % 16, 1):
                (a, sa, _), (b, sb, _), (c, sc, _) = (codes(r, K, s, pad) for r, s in ((M, 1), (N, 2), (N, 3)))
                for ws in (True, False):
                    out[f"{i} {pad} {ws}"] = sg.gemm_e4m3_gated(a, sa, b, sb, c, sc, workspace=ws)
        return out
    a = run()
    with sg.library(sg.POISON_LIB_PATH):
        b = run()
    torch.cuda.synchronize()
    same(a, b)


def test_another_stream():
    """On a stream that is not the current one, given as an argument."""
    want = all_ops()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    A = dev(normal(70, 900))
    (Bg, Bu), _ = weights(130, 900, False, True, 0, 0, 1)
    s.wait_stream(torch.cuda.current_stream())
    pg, pu = torch.empty(70, 130, device="cuda"), torch.empty(70, 130, device="cuda")
    y = sg.sgemm_gated(A, Bg, Bu, activation="gelu", pre_gate=pg, pre_up=pu, stream=s)
    back = sg.sgemm_gated_backward(pg, A, Bg, Bu, pre_gate=pg, pre_up=pu, stream=s)
    n = sg.grad_norm([y, pg], stream=s)
    s.synchronize()
    assert torch.equal(y, want["g"])
    for got, k in zip(back, ("dA", "dBg", "dBu", "bg", "bu")):
        assert torch.equal(got, want[k])
    assert abs(float(n) - float(torch.cat([y, pg]).double().norm())) <= 1e-6 * float(n)
    with torch.cuda.stream(s):
        got = all_ops()
    s.synchronize()
    same(want, got)


def test_threads_on_their_streams():
    """Several threads at once, each on its own stream, give the bits one gives."""
    want = all_ops()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(2):
                    got = all_ops()
                    torch.cuda.current_stream().synchronize()
                    same(want, got)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


def test_graph_replays():
    """Captured and replayed with other inputs in the same memory, with eager work
    of its own between the replays; two graphs whose workspaces come from one
    pool."""
    T, D, F = 40, 96, 200
    x, w = dev(normal(T, D, seed=1)), dev(normal(D, seed=2))
    (Bg, Bu), _ = weights(F, D, False, True, 0, 0, 3)
    (q1, s1), (q2, s2) = (sg.quantize_e4m3(dev(normal(F, D, seed=i))) for i in (4, 5))

    def step():
        y, _ = sg.layernorm(x, w, w)
        pg, pu = torch.empty(T, F, device="cuda"), torch.empty(T, F, device="cuda")
        h = sg.sgemm_gated(y, Bg, Bu, pre_gate=pg, pre_up=pu)
        back = sg.sgemm_gated_backward(h, y, Bg, Bu, pre_gate=pg, pre_up=pu)
        dx, dw, db = sg.layernorm_backward(back[0], x, w)
        grads = [*back[1:], dx, dw, db]
        norm = sg.clip_grad_norm(grads, 0.1)
        q, s, _ = sg.layernorm_e4m3(x, w, w)
        e = sg.gemm_e4m3_gated(q, s, q1, s1, q2, s2)
        return [y, h, norm, e, *grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        out_a = step()
    with torch.cuda.graph(b, pool=a.pool()):
        out_b = step()
    for i in range(4):
        x.copy_(torch.from_numpy(normal(T, D, seed=20 + i)))
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        a.replay()
        torch.cuda.synchronize()
        for g, e in zip(out_a, eager):
            assert torch.equal(g, e)
        step()
        b.replay()
        torch.cuda.synchronize()
        for g, e in zip(out_b, eager):
            assert torch.equal(g, e)


def test_rows_further_apart_than_32_bits():
    """Row strides whose byte offsets pass 2^31 and 2^32: few rows of weights a
    long way apart, where only the forms that address in 64 bits serve."""
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("too little memory")
    K, N, M, ld = 40, 6, 5, (1 << 28) + 5
    buf = torch.empty(N * ld, device="cuda")
    hg, hu = normal(N, K, seed=1), normal(N, K, seed=2)
    Bg = buf[:(N - 1) * ld + K].as_strided((N, K), (ld, 1))
    Bu = buf[K:].as_strided((N, K), (ld, 1))
    Bg.copy_(torch.from_numpy(hg))
    Bu.copy_(torch.from_numpy(hu))
    A = normal(M, K, seed=3)
    Y, _, _, ty, _, _ = ref.gated(A.astype(np.float64), hg.T.astype(np.float64), hu.T.astype(np.float64), K)
    for ws in (True, False):
        ops_ref.within(f64(sg.sgemm_gated(dev(A), Bg, Bu, transb=True, workspace=ws)), Y, ty)
    # the same memory as K x N weights: 6 values of k, 40 columns
    A = normal(M, N, seed=4)
    Y, _, _, ty, _, _ = ref.gated(A.astype(np.float64), hg.astype(np.float64), hu.astype(np.float64), N)
    for ws in (True, False):
        ops_ref.within(f64(sg.sgemm_gated(dev(A), Bg, Bu, workspace=ws)), Y, ty)
    # the gradient's halves, rows of a norm and of many tensors
    dy, w = normal(N, K, seed=5), normal(K, seed=6)
    want = ref.gated_grad(dy.astype(np.float64), hg.astype(np.float64), hu.astype(np.float64), "silu")
    og = buf[2 * K:].as_strided((N, K), (ld, 1))
    ou = buf[3 * K:].as_strided((N, K), (ld, 1))
    dG, dU, bg, bu = sg.gated_grad(dev(dy), Bg, Bu, out_gate=og, out_up=ou)
    for g, v, t in zip((dG, dU, bg, bu), want[:4], want[4:]):
        ops_ref.within(f64(g), v, t)
    Y, ty = ref.layernorm(hg.astype(np.float64), w.astype(np.float64), None, 1e-5)
    ops_ref.within(f64(sg.layernorm(Bg, dev(w), out=og)[0]), Y, ty)
    dx, _, _, tx, _, _ = ref.layernorm_grad(dy.astype(np.float64), hg.astype(np.float64), w.astype(np.float64), 1e-5)
    ops_ref.within(f64(sg.layernorm_backward(dev(dy), Bg, dev(w), out=ou)[0]), dx, tx)
    n, f = ref.clip([hg, hu], 0.5, 1e-6)
    assert abs(float(sg.clip_grad_norm([Bg, Bu], 0.5)) - n) <= 2 * ref.U * n
    ops_ref.within(f64(Bu), hu.astype(np.float64) * f, np.abs(hu * f) * 2 * ref.U)


def test_arguments_are_checked():
    """Shapes, types, devices and names that do not fit are refused by the binding."""
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)  # noqa: E731
    A, B = e(4, 8), e(8, 6)
    for call in (lambda: sg.sgemm_gated(A, B, e(8, 5)), lambda: sg.sgemm_gated(A, e(7, 6), e(7, 6)),
                 lambda: sg.sgemm_gated(A, B, B, transb=True), lambda: sg.sgemm_gated(A, B, B, activation="tanh"),
                 lambda: sg.sgemm_gated(A, B, B, bias_gate=e(5)), lambda: sg.sgemm_gated(A, B, B, pre_up=e(4, 5)),
                 lambda: sg.sgemm_gated(A, B, B, out=e(4, 5)), lambda: sg.sgemm_gated(A, B, B.cpu()),
                 lambda: sg.sgemm_gated(A.T, B, B), lambda: sg.sgemm_gated(A, B, B, workspace=e(16).cpu()),
                 lambda: sg.gated_grad(A, A, e(4, 7)), lambda: sg.gated_grad(A, A, A, out_up=e(5, 8)),
                 lambda: sg.gated_grad(A, A, A, dbias_up=e(7)), lambda: sg.layernorm(A, e(7)), lambda: sg.layernorm(A, e(8), e(9)),
                 lambda: sg.layernorm_backward(A, e(4, 9)), lambda: sg.clip_grad_norm([A], 1.0, out=[A, A]),
                 lambda: sg.clip_grad_norm([A, B], 1.0, out=[A, e(8, 7)]), lambda: sg.grad_norm([A, B.cpu()]),
                 lambda: sg.grad_norm([A.T])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sg.sgemm_gated(A.double(), B, B), lambda: sg.grad_norm([A.half()]), lambda: sg.layernorm(A.bfloat16()),
                 lambda: sg.gemm_e4m3_gated(A, None, B, None, B, None)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: sg.sgemm_gated(A, B, e(8, 6), form=8), lambda: sg.clip_grad_norm([A], -1.0),
                 lambda: sg.clip_grad_norm([A], float("nan")), lambda: sg.layernorm(A, eps=-1.0)):
        with pytest.raises(sg.SgemmError):
            call()
