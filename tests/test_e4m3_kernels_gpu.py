"""Each kernel of the 8-bit product against 64 bits, with every part of the
epilogue, and from the build that sets LDS to NaN before each refill.

The codes are multiples of 1/2 up to 8, so that products are multiples of 1/4
up to 64 and every partial sum of at most 2^16 of them is exact in float32, in
whatever order: what is left are the epilogue's roundings, U = 2^-24 of the
value each, and the activation's own (16 U of its argument, 32 U of a slope, as
ops_ref counts them)."""
import math

import pytest
import torch

import e4m3_cases as cases
import fp32_gemm_sgemm_amd as sg
import ops_ref as ref
from gpu_cases import note

pytestmark = pytest.mark.gpu

U = ref.U


def half_codes():
    """The bytes of the multiples of 1/2 in [-8, 8]."""
    return [c for c, v in enumerate(ref.E4M3) if abs(v) <= 8 and (2 * v) % 1 == 0]


def codes(rows, cols, aligned, shift, gen):
    """rows x cols random codes, the bytes between and around rows NaN codes."""
    ld = (cols + 15) // 16 * 16 + (16 if aligned else 5)
    buf = torch.full((rows * ld + 32,), 0x7f, dtype=torch.uint8, device="cuda")
    t = buf[16 + shift:].as_strided((rows, cols), (ld, 1), 16 + shift)
    some = torch.tensor(half_codes(), dtype=torch.uint8, device="cuda")
    t.copy_(some[torch.randint(0, len(some), (rows, cols), generator=gen, device="cuda")])
    return t.view(torch.float8_e4m3fn)


def guarded(rows, cols, pad=3):
    """A rows x cols output inside a buffer of sentinels; (view, check)."""
    ld = cols + pad
    buf = torch.full((rows * ld + 64,), 77.0, device="cuda")
    inner = buf[32:32 + rows * ld].view(rows, ld)

    def check():
        assert bool((inner[:, cols:] == 77.0).all()) and bool((buf[:32] == 77.0).all()) and \
            bool((buf[32 + rows * ld:] == 77.0).all()), "memory outside the output was written"
    return inner[:, :cols], check


def silu(z):
    return z * torch.sigmoid(z)


def gelu_slope(z):
    return torch.special.erfc(z * -math.sqrt(0.5)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def within(got, want, bound, what):
    err = (got.double() - want).abs_()
    bad = ~(err <= bound)
    n = int(bad.sum())
    if n:
        first = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {n} of {bad.numel()} off, first at {first}: "
                             f"{got[tuple(first)].item()} for {want[tuple(first)].item()}")


@pytest.mark.parametrize("case", cases.CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-" +
                         ("aligned" if c[4] else "any") + ("-split" if c[6] > 1 else ""))
def test_each_kernel(case):
    _, M, N, K, aligned, workspace, _ = case
    note(f"e4m3 {case}")
    # (the cases reach their kernels on this many compute units)
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256
    i = cases.CASES.index(case)
    gen = torch.Generator(device="cuda").manual_seed(i)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    # rows that are not aligned: by their stride (A) or by their start (B)
    a, b = codes(M, K, aligned or i % 2 == 1, 0, gen), codes(N, K, True, 0 if aligned or i % 2 == 0 else 3, gen)
    sa, sb = torch.exp(normal(M)), torch.exp(normal(N)) / (10 * K ** 0.5)
    bias, R, Z0 = normal(N), normal(M, N), normal(M, N)
    out, ok = guarded(M, N)
    pre, ok_pre = guarded(M, N, pad=2)

    def value():
        return sg.gemm_e4m3(a, sa, b, sb, bias=bias, activation="silu", residual=R, out=out, pre=pre,
                            workspace=workspace)

    def gradient():
        return sg.gemm_e4m3(a, sa, b, sb, activation="gelu", grad_pre=Z0, out=out, workspace=workspace)

    s = torch.mm(a.float().double(), b.float().double().T.contiguous())
    s.mul_(sa.double()[:, None]).mul_(sb.double())
    value()
    torch.cuda.synchronize()
    ok()
    ok_pre()
    z = s + bias.double()
    # two scale factors, the bias
    tz = 2 * U * s.abs() + U * z.abs() + 1e-37
    within(pre, z, tz, "pre")
    y = silu(z)
    ty = ref.LIPSCHITZ * tz + ref.ACT_ERR * z.abs()
    y += R.double()
    ty += U * y.abs()
    within(out, y, ty, "out")
    del z, tz, y, ty
    held, held_pre = out.clone(), pre.clone()
    gradient()
    torch.cuda.synchronize()
    ok()
    y = s * gelu_slope(Z0.double())
    # (the slope is at most 1.2)
    within(out, y, (2 * U * ref.LIPSCHITZ + ref.SLOPE_ERR) * s.abs() + U * y.abs() + 1e-37, "gradient")
    del y, s
    slope = out.clone()
    with sg.library(sg.POISON_LIB_PATH):
        gradient()
        same = torch.equal(out, slope)
        value()
        same = same and torch.equal(out, held) and torch.equal(pre, held_pre)
    assert same, "race check"
