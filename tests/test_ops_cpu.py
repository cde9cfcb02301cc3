"""The operators around a product on the host: exported as declared, and every
refused call comes back as an error before any HIP call (there may be no GPU)."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import fp32_gemm_sgemm_amd as sg
import ops_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sgemm_ops.h")
INVALID = 1
P = 1 << 20  # made-up device addresses, a megabyte apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sg.LIB_PATH):
        from fp32_gemm_sgemm_amd import build
        build.build()
    return sg.load()


def declared():
    return sorted(set(re.findall(r"^\s*int\s+(sgemm_\w+)\s*\(", open(HEADER).read(), re.M)))


@pytest.mark.parametrize("path", [sg.LIB_PATH, sg.POISON_LIB_PATH, sg.TIMELINE_LIB_PATH])
def test_declared_functions_are_exported(lib, path):
    out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True, check=True).stdout
    names = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert len(declared()) == 10 and set(declared()) <= names


def test_activations_match_the_header(lib):
    text = open(HEADER).read()
    for name, value in sg.ACTIVATIONS.items():
        assert re.search(rf"#define\s+SGEMM_ACT_{name.upper()}\s+{value}\b", text)


def test_epilogue_structure_matches_the_header(lib):
    """The ctypes structure has the C layout: compiled and compared."""
    src = '#include <stdio.h>\n#include <stddef.h>\n#define __HIP_PLATFORM_AMD__ 1\n#include "sgemm_ops.h"\nint main(void){' + "".join(
        f'printf("%zu ", offsetof(sgemm_epilogue, {f}));' for f, _ in sg.SgemmEpilogue._fields_) + \
        'printf("%zu", sizeof(sgemm_epilogue)); return 0;}'
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        c = os.path.join(d, "t.c")
        open(c, "w").write(src)
        subprocess.run(["gcc", f"-I{ROOT}/include", "-I/opt/rocm/include", c, "-o", os.path.join(d, "t")], check=True)
        got = [int(v) for v in subprocess.run([os.path.join(d, "t")], capture_output=True, text=True).stdout.split()]
    want = [getattr(sg.SgemmEpilogue, f).offset for f, _ in sg.SgemmEpilogue._fields_]
    assert got == want + [ctypes.sizeof(sg.SgemmEpilogue)]


def epi(**kw):
    e = sg.SgemmEpilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def product(lib, e, M=8, N=8, K=8, ta=0, tb=0, A=P, lda=8, B=2 * P, ldb=8, C=3 * P, ldc=8, batch=1, sa=0, sb=0, sc=0,
            ws=0, ws_bytes=0, cfg=None):
    return lib.sgemm_f32_epilogue(ta, tb, M, N, K, 1.0, A, lda, sa, B, ldb, sb, C, ldc, sc, batch,
                                  ctypes.byref(e) if e is not None else None, ws, ws_bytes, 0,
                                  ctypes.byref(cfg) if cfg is not None else None)


BAD_EPILOGUES = {
    "unknown activation": dict(activation=5),
    "negative activation": dict(activation=-1),
    "pre and grad_pre": dict(pre=4 * P, ld_pre=8, grad_pre=5 * P, ld_grad_pre=8),
    "misaligned bias": dict(bias=4 * P + 2),
    "bias over C": dict(bias=3 * P + 4),
    "negative bias stride": dict(bias=4 * P, stride_bias=-1),
    "short pre rows": dict(pre=4 * P, ld_pre=7),
    "misaligned pre": dict(pre=4 * P + 1, ld_pre=8),
    "pre over C": dict(pre=3 * P, ld_pre=8),
    "pre over A": dict(pre=P, ld_pre=8),
    "pre over B": dict(pre=2 * P, ld_pre=8),
    "pre over bias": dict(pre=4 * P, ld_pre=8, bias=4 * P),
    "pre over the residual": dict(pre=4 * P, ld_pre=8, residual=4 * P, ld_residual=8),
    "short residual rows": dict(residual=4 * P, ld_residual=7),
    "misaligned residual": dict(residual=4 * P + 2, ld_residual=8),
    "residual half over C": dict(residual=3 * P + 32, ld_residual=8),
    "residual as C with another stride": dict(residual=3 * P, ld_residual=9),
    "short grad_pre rows": dict(grad_pre=4 * P, ld_grad_pre=7),
    "grad_pre over C": dict(grad_pre=3 * P, ld_grad_pre=8),
    "negative residual stride": dict(residual=4 * P, ld_residual=8, stride_residual=-8),
    "huge rows": dict(residual=4 * P, ld_residual=2 ** 31 - 1),
}


@pytest.mark.parametrize("what", BAD_EPILOGUES)
def test_epilogues_refused(lib, what):
    e = epi(**BAD_EPILOGUES[what])
    assert product(lib, e) == INVALID
    assert lib.sgemm_e4m3(8, 8, 8, P, 8, None, 2 * P, 8, None, 3 * P, 8, ctypes.byref(e), 0, 0, 0) == INVALID


def test_epilogue_products_refused(lib):
    e = epi(residual=4 * P, ld_residual=8)
    for kw in (dict(M=-1), dict(K=-1), dict(lda=7), dict(ldb=7), dict(ldc=7), dict(A=0), dict(B=0), dict(C=0),
               dict(A=P + 2), dict(C=P), dict(ta=2), dict(ws=3 * P, ws_bytes=64), dict(ws=4 * P, ws_bytes=64),
               dict(ws=5 * P + 4, ws_bytes=64), dict(batch=2, sc=8), dict(batch=2, sc=64, sa=-1)):
        assert product(lib, e, **kw) == INVALID, kw
    # a bias per entry must lie outside C, pre must keep its entries apart
    assert product(lib, epi(pre=4 * P, ld_pre=8, stride_pre=8), batch=2, sc=64, sa=64) == INVALID
    # forced variants without an epilogue form
    for vid in (0, 1, 2, 3, 8, 9):
        cfg = sg.SgemmCfg()
        cfg.id = vid
        assert product(lib, e, cfg=cfg) == INVALID
    # nothing to do is no error, whatever the pointers
    assert product(lib, epi(activation=1), M=0, A=0, B=0, C=0) == 0


def row(lib, rows=4, D=8, X=P, ldx=8, R=2 * P, ldr=8, w=3 * P, eps=1e-6, S=4 * P, lds=8, Y=5 * P, ldy=8):
    return lib.sgemm_rmsnorm_f32(rows, D, X, ldx, R, ldr, w, eps, S, lds, Y, ldy, 0)


def row8(lib, rows=4, D=8, X=P, ldx=8, R=2 * P, ldr=8, w=3 * P, eps=1e-6, S=4 * P, lds=8, Q=5 * P, ldq=8, scale=6 * P):
    return lib.sgemm_rmsnorm_e4m3(rows, D, X, ldx, R, ldr, w, eps, S, lds, Q, ldq, scale, 0)


def test_norms_refused(lib):
    for kw in (dict(rows=-1), dict(D=0), dict(D=-3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(X=0), dict(X=P + 2), dict(ldx=7), dict(ldr=7), dict(R=2 * P + 1), dict(w=3 * P + 1), dict(lds=7),
               dict(ldx=2 ** 31 - 1),
               dict(S=P + 32), dict(S=P, ldx=9), dict(S=2 * P, ldr=9), dict(S=3 * P)):
        assert row(lib, **kw) == INVALID, kw
        assert row8(lib, **kw) == INVALID, kw
    for kw in (dict(Y=0), dict(Y=5 * P + 2), dict(ldy=7), dict(Y=4 * P), dict(Y=3 * P), dict(Y=P + 4), dict(Y=P, ldx=9),
               dict(Y=P, S=P), dict(Y=2 * P, S=2 * P)):
        assert row(lib, **kw) == INVALID, kw
    for kw in (dict(Q=0), dict(ldq=7), dict(Q=P), dict(Q=2 * P), dict(Q=4 * P), dict(Q=6 * P), dict(scale=0),
               dict(scale=6 * P + 2), dict(scale=P), dict(scale=3 * P), dict(scale=4 * P)):
        assert row8(lib, **kw) == INVALID, kw
    assert row(lib, rows=0, X=0, Y=0) == 0
    q = lambda rows=4, D=8, X=P, ldx=8, Q=2 * P, ldq=8, s=3 * P: lib.sgemm_quantize_e4m3(rows, D, X, ldx, Q, ldq, s, 0)  # noqa: E731
    for kw in (dict(rows=-1), dict(D=0), dict(X=0), dict(Q=0), dict(s=0), dict(ldx=7), dict(ldq=7), dict(Q=P), dict(s=P),
               dict(s=2 * P)):
        assert q(**kw) == INVALID, kw


def grad(lib, rows=4, D=8, dY=P, ldy=8, S=2 * P, lds=8, w=3 * P, eps=1e-6, dS=4 * P, ldds=8, dX=5 * P, lddx=8, dw=6 * P,
         ws=7 * P, ws_bytes=1 << 16):
    return lib.sgemm_rmsnorm_f32_grad(rows, D, dY, ldy, S, lds, w, eps, dS, ldds, dX, lddx, dw, ws, ws_bytes, 0)


def workspace(fn, *args):
    n = ctypes.c_size_t()
    assert fn(*args, ctypes.byref(n)) == 0
    return n.value


def test_norm_gradients_refused(lib):
    rows = 40
    need = workspace(lib.sgemm_rmsnorm_f32_grad_workspace, rows, 8)
    assert need > 0
    for kw in (dict(rows=-1), dict(D=0), dict(eps=-1.0), dict(dY=0), dict(S=0), dict(dX=0), dict(ldy=7), dict(lds=7),
               dict(ldds=7), dict(lddx=7), dict(dw=6 * P + 2), dict(w=2), dict(dX=P), dict(dX=2 * P), dict(dX=3 * P),
               dict(dX=4 * P, ldds=9), dict(dw=P), dict(dw=5 * P), dict(dw=3 * P), dict(ws=0, ws_bytes=0),
               dict(ws_bytes=need - 1), dict(ws=7 * P + 4), dict(ws=P), dict(ws=5 * P), dict(ws=6 * P)):
        assert grad(lib, **{"rows": rows, **kw}) == INVALID, kw
    n = ctypes.c_size_t()
    assert lib.sgemm_rmsnorm_f32_grad_workspace(-1, 8, ctypes.byref(n)) == INVALID
    assert lib.sgemm_rmsnorm_f32_grad_workspace(1, 0, ctypes.byref(n)) == INVALID
    assert lib.sgemm_rmsnorm_f32_grad_workspace(1, 8, None) == INVALID


def act_grad(lib, M=40, N=8, act=4, dY=P, ldy=8, Z=2 * P, ldz=8, dZ=3 * P, lddz=8, db=4 * P, ws=5 * P, ws_bytes=1 << 20):
    return lib.sgemm_f32_activation_grad(M, N, act, dY, ldy, Z, ldz, dZ, lddz, db, ws, ws_bytes, 0)


def test_activation_gradients_refused(lib):
    M = 4000
    need = workspace(lib.sgemm_f32_activation_grad_workspace, M, 8)
    assert need > 0 and need % 32 == 0
    for kw in (dict(M=-1), dict(N=-1), dict(act=5), dict(act=-1), dict(dY=0), dict(Z=0), dict(Z=2), dict(ldy=7),
               dict(ldz=7), dict(lddz=7), dict(dZ=3 * P + 2), dict(db=4 * P + 1), dict(dZ=2 * P), dict(dZ=P + 32),
               dict(dZ=P, ldy=9), dict(db=P), dict(db=2 * P), dict(db=3 * P), dict(ws=0, ws_bytes=0),
               dict(ws_bytes=need - 1), dict(ws=5 * P + 8), dict(ws=P), dict(ws=3 * P)):
        assert act_grad(lib, **{"M": M, **kw}) == INVALID, kw
    assert act_grad(lib, N=0, dY=0) == 0
    # nothing asked for
    assert act_grad(lib, dZ=None, db=None) == 0


def e8(lib, M=8, N=8, K=8, A=P, lda=8, sa=2 * P, B=3 * P, ldb=8, sb=4 * P, C=5 * P, ldc=8, ws=0, ws_bytes=0):
    return lib.sgemm_e4m3(M, N, K, A, lda, sa, B, ldb, sb, C, ldc, None, ws, ws_bytes, 0)


def test_e4m3_products_refused(lib):
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=7), dict(ldb=7), dict(ldc=7), dict(A=0), dict(B=0), dict(C=0),
               dict(C=5 * P + 2), dict(sa=2 * P + 1), dict(sb=4 * P + 2), dict(C=P), dict(C=2 * P), dict(C=3 * P),
               dict(C=4 * P), dict(ws=6 * P + 4, ws_bytes=64), dict(ws=5 * P, ws_bytes=64), dict(ws=P, ws_bytes=64),
               dict(ws=4 * P, ws_bytes=64), dict(lda=2 ** 31 - 1)):
        assert e8(lib, **kw) == INVALID, kw
    assert e8(lib, M=0, A=0, B=0, C=0) == 0
    n = ctypes.c_size_t()
    assert lib.sgemm_e4m3_workspace_size(-1, 1, 1, ctypes.byref(n)) == INVALID
    assert lib.sgemm_e4m3_workspace_size(1, 1, 1, None) == INVALID


def test_workspaces_cover_what_is_summed(lib):
    """Sizes are multiples of a row of column sums, and zero where one
    workgroup holds all rows."""
    for M, N in ((1, 5), (10, 100), (5000, 3), (70000, 8192)):
        n = workspace(lib.sgemm_f32_activation_grad_workspace, M, N)
        assert n % (4 * N) == 0 and (n == 0 or n // (4 * N) <= M)
    assert workspace(lib.sgemm_rmsnorm_f32_grad_workspace, 1, 4096) == 0
    assert workspace(lib.sgemm_rmsnorm_f32_grad_workspace, 0, 4096) == 0
    assert workspace(lib.sgemm_rmsnorm_f32_grad_workspace, 100, 4096) == 100 * 4096 * 4


def test_rows_that_overlap_are_refused():
    """A broadcast (stride 0) tensor is no row-major matrix."""
    torch = pytest.importorskip("torch")
    from fp32_gemm_sgemm_amd import binding
    with pytest.raises(ValueError):
        binding._row_major_view(torch.zeros(1, 8).expand(4, 8), "A")
    assert binding._row_major_view(torch.zeros(1, 8).expand(1, 8), "A") == (1, 8, 8)
    with pytest.raises(ValueError):
        binding._row_major_view(torch.zeros(8, 4).t(), "A")


def test_sizes_past_the_abi_are_refused():
    """Sizes and strides that an int does not hold must not be cut to one that
    it does (tensors without memory: only their shapes are read)."""
    torch = pytest.importorskip("torch")
    from fp32_gemm_sgemm_amd import ops
    most = 2**31 - 1 - 1024

    def meta(rows, cols, ld):
        return torch.empty_strided((rows, cols), (ld, 1), device="meta")
    assert ops._rows(meta(2, 8, most), "x") == (2, 8, most)
    assert ops._rows(meta(most, 1, 1), "x") == (most, 1, 1)
    for x in (meta(2, 8, most + 1), meta(2, 8, 2**32 + 8), meta(2**32, 1, 1), meta(1, 2**32 + 4, 1),
              meta(2, 2**32 + 4, 2**33)):
        with pytest.raises(ValueError, match="must not pass"):
            ops._rows(x, "x")
    with pytest.raises(ValueError, match="batch entries"):
        ops._batch_view(torch.empty_strided((2**32 + 1, 2, 2), (0, 2, 1), device="meta"), "x")
    x = torch.zeros(4)
    assert ops._supplied(x, x.device) == (x.data_ptr(), 16)
    with pytest.raises(ValueError, match="contiguous"):
        ops._supplied(torch.zeros(1).expand(1 << 20), x.device)


def test_host_tensors_and_types_are_refused():
    torch = pytest.importorskip("torch")
    x, q = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.uint8).view(torch.float8_e4m3fn)
    for call in (lambda: sg.sgemm_epilogue(x, x, transb=True), lambda: sg.rmsnorm(x), lambda: sg.rmsnorm_e4m3(x),
                 lambda: sg.quantize_e4m3(x), lambda: sg.activation_grad(x), lambda: sg.rmsnorm_backward(x, x),
                 lambda: sg.gemm_e4m3(q, None, q, None), lambda: sg.sgemm_epilogue_backward(x, x, x)):
        with pytest.raises(ValueError):
            call()


# ---- the reference itself ------------------------------------------------------------------------------

def test_reference_slopes_are_the_values_derivatives():
    z = np.linspace(-6, 6, 1201) + 1e-3
    h = 1e-6
    for name in ref.ACTS:
        num = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
        assert np.abs(num - ref.slope(z, name)).max() < 1e-8
        assert np.abs(ref.slope(z, name)).max() <= ref.LIPSCHITZ


def test_reference_codes_are_e4m3():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t, ref.E4M3.astype(np.float32), equal_nan=True)


def test_no_column_kernel_that_no_call_reaches(lib):
    """The norm's column pass serves rows past 16384 values, so its narrow form
    (16 lanes along at most 128 columns) would never run and is not compiled."""
    names = open(sg.LIB_PATH, "rb").read()
    forms = {(kind, tx): f"col_kernelILi{kind}ELi{tx}EE".encode() in names for kind in (0, 1) for tx in (16, 64)}
    assert forms == {(0, 16): True, (0, 64): True, (1, 16): False, (1, 64): True}
