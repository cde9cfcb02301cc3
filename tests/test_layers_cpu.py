"""The operators of sgemm_layers.h on the host: exported as declared, and every
refused call comes back as an error before any HIP call (there may be no GPU)."""
import ctypes
import os
import re
import subprocess
import tempfile

import numpy as np
import pytest

import e4m3_cases
import fp32_gemm_sgemm_amd as sg
import layers_cases
import layers_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sgemm_layers.h")
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
    assert len(declared()) == 15 and set(declared()) <= names


def layout(struct, name):
    """The C layout of a structure of the header: offsets of its fields and its size."""
    src = '#include <stdio.h>\n#include <stddef.h>\n#define __HIP_PLATFORM_AMD__ 1\n#include "sgemm_layers.h"\n' \
        'int main(void){' + "".join(f'printf("%zu ", offsetof({name}, {f}));' for f, _ in struct._fields_) + \
        f'printf("%zu", sizeof({name})); return 0;}}'
    with tempfile.TemporaryDirectory() as d:
        c = os.path.join(d, "t.c")
        open(c, "w").write(src)
        subprocess.run(["gcc", f"-I{ROOT}/include", "-I/opt/rocm/include", c, "-o", os.path.join(d, "t")], check=True)
        got = subprocess.run([os.path.join(d, "t")], capture_output=True, text=True).stdout.split()
    return [int(v) for v in got]


def test_tensor_structure_matches_the_header(lib):
    want = [getattr(sg.SgemmTensor, f).offset for f, _ in sg.SgemmTensor._fields_]
    assert layout(sg.SgemmTensor, "sgemm_tensor") == want + [ctypes.sizeof(sg.SgemmTensor)]


def test_gate_structure_matches_the_header(lib):
    want = [getattr(sg.SgemmGate, f).offset for f, _ in sg.SgemmGate._fields_]
    assert layout(sg.SgemmGate, "sgemm_gate") == want + [ctypes.sizeof(sg.SgemmGate)]


def test_forms_match_the_header():
    text = open(HEADER).read()
    for name in ("TILES", "ROWS", "PRODUCTS"):
        assert re.search(rf"#define\s+SGEMM_GATED_{name}\s+{getattr(sg, 'GATED_' + name)}\b", text)
    assert sg.GATED_AUTO == -1


# ---- the gated block ---------------------------------------------------------------------------------

def gate(**kw):
    e = sg.SgemmGate()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def gated(lib, e=None, tb=0, M=8, N=8, K=8, A=P, lda=8, Bg=2 * P, ldg=8, Bu=3 * P, ldu=8, C=4 * P, ldc=8, ws=0, ws_bytes=0,
          form=-1):
    e = gate() if e is None else e
    return lib.sgemm_f32_gated(tb, M, N, K, A, lda, Bg, ldg, Bu, ldu, C, ldc, ctypes.byref(e), ws, ws_bytes, form, 0)


def gated8(lib, e=None, M=8, N=8, K=8, A=P, lda=8, sa=8 * P, Bg=2 * P, ldg=8, sgate=9 * P, Bu=3 * P, ldu=8, su=10 * P, C=4 * P,
           ldc=8, ws=0, ws_bytes=0):
    e = gate() if e is None else e
    return lib.sgemm_e4m3_gated(M, N, K, A, lda, sa, Bg, ldg, sgate, Bu, ldu, su, C, ldc, ctypes.byref(e), ws, ws_bytes, 0)


BAD_GATES = {
    "unknown activation": dict(activation=5),
    "negative activation": dict(activation=-1),
    "misaligned gate bias": dict(bias_gate=5 * P + 2),
    "misaligned up bias": dict(bias_up=5 * P + 1),
    "bias over C": dict(bias_gate=4 * P + 4),
    "up bias over C": dict(bias_up=4 * P),
    "short pre_gate rows": dict(pre_gate=5 * P, ld_pre_gate=7),
    "short pre_up rows": dict(pre_up=5 * P, ld_pre_up=7),
    "misaligned pre_gate": dict(pre_gate=5 * P + 2, ld_pre_gate=8),
    "pre_gate over C": dict(pre_gate=4 * P, ld_pre_gate=8),
    "pre_gate over A": dict(pre_gate=P, ld_pre_gate=8),
    "pre_gate over the gate's weights": dict(pre_gate=2 * P, ld_pre_gate=8),
    "pre_up over the other weights": dict(pre_up=3 * P, ld_pre_up=8),
    "pre_up over pre_gate": dict(pre_up=5 * P, ld_pre_up=8, pre_gate=5 * P, ld_pre_gate=8),
    "pre_up over the last of pre_gate": dict(pre_up=5 * P + 252, ld_pre_up=9, pre_gate=5 * P, ld_pre_gate=8),
    "pre_gate over its bias": dict(pre_gate=5 * P, ld_pre_gate=8, bias_gate=5 * P),
    "pre_up over the gate's bias": dict(pre_up=5 * P, ld_pre_up=8, bias_gate=5 * P),
    "columns that meet": dict(pre_gate=5 * P, ld_pre_gate=16, pre_up=5 * P + 28, ld_pre_up=16),
    "huge rows": dict(pre_gate=5 * P, ld_pre_gate=2 ** 31 - 1),
}


@pytest.mark.parametrize("what", BAD_GATES)
def test_gates_refused(lib, what):
    assert gated(lib, gate(**BAD_GATES[what])) == INVALID
    assert gated8(lib, gate(**BAD_GATES[what])) == INVALID


def test_gated_blocks_refused(lib):
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=7), dict(ldg=7), dict(ldu=7), dict(ldc=7), dict(A=0), dict(Bg=0),
               dict(Bu=0), dict(C=0), dict(C=4 * P + 2), dict(C=P), dict(C=2 * P), dict(C=3 * P + 16),
               dict(ws=4 * P, ws_bytes=64), dict(ws=P, ws_bytes=64), dict(ws=2 * P, ws_bytes=64),
               dict(ws=3 * P, ws_bytes=64), dict(ws=6 * P + 4, ws_bytes=64), dict(M=2 ** 31 - 1), dict(K=2 ** 31 - 1),
               dict(lda=2 ** 31 - 1)):
        assert gated(lib, **kw) == INVALID, kw
        assert gated8(lib, **kw) == INVALID, kw
    for kw in (dict(tb=2), dict(tb=-1), dict(A=P + 2), dict(Bg=2 * P + 1), dict(Bu=3 * P + 2), dict(form=-2), dict(form=8),
               dict(form=sg.GATED_PRODUCTS), dict(form=sg.GATED_PRODUCTS, ws=6 * P, ws_bytes=2 * 8 * 8 * 4 - 16),
               # a tile whose offsets would not fit in 32 bits
               dict(form=0, lda=1 << 23), dict(form=2, tb=1, ldg=1 << 23), dict(form=1, ldu=1 << 26)):
        assert gated(lib, **kw) == INVALID, kw
    for kw in (dict(sa=8 * P + 2), dict(sgate=9 * P + 1), dict(su=10 * P + 2), dict(C=8 * P), dict(C=9 * P), dict(C=10 * P),
               dict(ws=8 * P, ws_bytes=64), dict(ws=10 * P, ws_bytes=64)):
        assert gated8(lib, **kw) == INVALID, kw
    assert lib.sgemm_f32_gated(0, 8, 8, 8, P, 8, 2 * P, 8, 3 * P, 8, 4 * P, 8, None, 0, 0, -1, 0) == INVALID
    assert lib.sgemm_e4m3_gated(8, 8, 8, P, 8, None, 2 * P, 8, None, 3 * P, 8, None, 4 * P, 8, None, 0, 0, 0) == INVALID
    # the workspace must keep clear of what the gate reads and stores
    for e in (gate(bias_up=6 * P), gate(pre_up=6 * P, ld_pre_up=8)):
        assert gated(lib, e, ws=6 * P, ws_bytes=64) == INVALID
        assert gated8(lib, e, ws=6 * P, ws_bytes=64) == INVALID
    # nothing to do is no error, whatever the pointers
    assert gated(lib, M=0, A=0, Bg=0, Bu=0, C=0) == 0
    assert gated8(lib, N=0, A=0, Bg=0, Bu=0, C=0) == 0
    n = ctypes.c_size_t()
    assert lib.sgemm_f32_gated_workspace(0, -1, 8, 8, P, 8, P, 8, P, 8, ctypes.byref(n)) == INVALID
    assert lib.sgemm_f32_gated_workspace(0, 8, 8, 8, P, 8, P, 8, P, 8, None) == INVALID
    assert lib.sgemm_f32_gated_workspace(1, 8, 8, 8, P, 8, P, 8, P, 7, ctypes.byref(n)) == INVALID
    assert lib.sgemm_e4m3_gated_workspace(1, 1, -1, ctypes.byref(n)) == INVALID
    assert lib.sgemm_e4m3_gated_workspace(1, 1, 1, None) == INVALID


def pair(lib, tb=0, M=8, N=8, K=8, A1=P, A2=2 * P, lda=8, B1=3 * P, ldb1=8, B2=4 * P, ldb2=8, C=5 * P, ldc=8, ws=0,
         ws_bytes=0):
    return lib.sgemm_f32_pair(tb, M, N, K, A1, A2, lda, B1, ldb1, B2, ldb2, C, ldc, ws, ws_bytes, 0)


def test_pairs_refused(lib):
    for kw in (dict(tb=2), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=7), dict(ldb1=7), dict(ldb2=7), dict(ldc=7), dict(A1=0),
               dict(A2=0), dict(B1=0), dict(B2=0), dict(C=0), dict(A2=2 * P + 2), dict(B2=4 * P + 1), dict(C=5 * P + 2),
               dict(C=P), dict(C=2 * P), dict(C=3 * P), dict(C=4 * P), dict(ws=5 * P, ws_bytes=64), dict(ws=2 * P, ws_bytes=64),
               dict(ws=4 * P, ws_bytes=64), dict(ws=6 * P + 4, ws_bytes=64), dict(ldb2=2 ** 31 - 1)):
        assert pair(lib, **kw) == INVALID, kw
    assert pair(lib, M=0, A1=0, A2=0, B1=0, B2=0, C=0) == 0
    n = ctypes.c_size_t()
    assert lib.sgemm_f32_pair_workspace(0, 8, 8, 8, P, P, 7, P, 8, P, 8, ctypes.byref(n)) == INVALID
    assert lib.sgemm_f32_pair_workspace(0, 8, 8, 8, P, P, 8, P, 8, P, 8, None) == INVALID


def gate_grad(lib, M=40, N=8, act=4, dY=P, ldy=8, G=2 * P, ldg=8, U=3 * P, ldu=8, dG=4 * P, lddg=8, dU=5 * P, lddu=8, bg=6 * P,
              bu=8 * P, ws=7 * P, ws_bytes=1 << 18):
    return lib.sgemm_f32_gated_grad(M, N, act, dY, ldy, G, ldg, U, ldu, dG, lddg, dU, lddu, bg, bu, ws, ws_bytes, 0)


def test_gate_gradients_refused(lib):
    M = 4000
    need = workspace(lib.sgemm_f32_gated_grad_workspace, M, 8)
    assert need > 0
    for kw in (dict(M=-1), dict(N=-1), dict(act=5), dict(act=-1), dict(dY=0), dict(G=0), dict(U=0), dict(ldy=7), dict(ldg=7),
               dict(ldu=7), dict(lddg=7), dict(lddu=7), dict(dG=4 * P + 2), dict(dU=5 * P + 2), dict(bg=6 * P + 2),
               dict(bu=8 * P + 1), dict(dG=P, lddg=9), dict(dG=P + 32), dict(dU=2 * P + 32), dict(dU=3 * P, lddu=9),
               dict(dG=5 * P), dict(dG=P, dU=P), dict(bg=P), dict(bg=4 * P), dict(bu=5 * P), dict(bu=6 * P), dict(bu=2 * P),
               dict(ws=0, ws_bytes=0), dict(ws_bytes=need - 1), dict(ws=7 * P + 8), dict(ws=P), dict(ws=3 * P), dict(ws=4 * P),
               dict(ws=5 * P), dict(ws=6 * P), dict(ws=8 * P)):
        assert gate_grad(lib, **{"M": M, **kw}) == INVALID, kw
    assert gate_grad(lib, N=0, dY=0) == 0
    assert gate_grad(lib, dG=None, dU=None, bg=None, bu=None, ws=0, ws_bytes=0) == 0  # nothing asked for
    n = ctypes.c_size_t()
    assert lib.sgemm_f32_gated_grad_workspace(-1, 8, ctypes.byref(n)) == INVALID
    assert lib.sgemm_f32_gated_grad_workspace(8, 8, None) == INVALID


# ---- layer norm ------------------------------------------------------------------------------------

def row(lib, rows=4, D=8, X=P, ldx=8, R=2 * P, ldr=8, w=3 * P, b=7 * P, eps=1e-6, S=4 * P, lds=8, Y=5 * P, ldy=8):
    return lib.sgemm_layernorm_f32(rows, D, X, ldx, R, ldr, w, b, eps, S, lds, Y, ldy, 0)


def row8(lib, rows=4, D=8, X=P, ldx=8, R=2 * P, ldr=8, w=3 * P, b=7 * P, eps=1e-6, S=4 * P, lds=8, Q=5 * P, ldq=8,
         scale=6 * P):
    return lib.sgemm_layernorm_e4m3(rows, D, X, ldx, R, ldr, w, b, eps, S, lds, Q, ldq, scale, 0)


def test_layer_norms_refused(lib):
    for kw in (dict(rows=-1), dict(D=0), dict(D=-3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(X=0), dict(X=P + 2), dict(ldx=7), dict(ldr=7), dict(R=2 * P + 1), dict(w=3 * P + 1),
               dict(b=7 * P + 2), dict(lds=7), dict(ldx=2 ** 31 - 1), dict(rows=2 ** 31 - 1), dict(D=2 ** 31 - 1),
               dict(S=P + 32), dict(S=P, ldx=9), dict(S=2 * P, ldr=9), dict(S=3 * P), dict(S=7 * P),
               dict(S=P, ldx=16, lds=16, D=9)):
        if kw.get("D") == 9:  # the same memory with the same stride is in place, 4 columns on it is not
            kw = dict(S=P + 16, ldx=16, lds=16, D=9, ldr=9, ldy=9, ldq=9)
            kw8 = {k: v for k, v in kw.items() if k != "ldy"}
            kw = {k: v for k, v in kw.items() if k != "ldq"}
            assert row(lib, **kw) == INVALID and row8(lib, **kw8) == INVALID
            continue
        assert row(lib, **kw) == INVALID, kw
        assert row8(lib, **kw) == INVALID, kw
    for kw in (dict(Y=0), dict(Y=5 * P + 2), dict(ldy=7), dict(Y=4 * P), dict(Y=3 * P), dict(Y=7 * P), dict(Y=P + 4),
               dict(Y=P, ldx=9), dict(Y=P, S=P), dict(Y=2 * P, S=2 * P)):
        assert row(lib, **kw) == INVALID, kw
    for kw in (dict(Q=0), dict(ldq=7), dict(Q=P), dict(Q=2 * P), dict(Q=4 * P), dict(Q=6 * P), dict(Q=7 * P),
               dict(scale=0), dict(scale=6 * P + 2), dict(scale=P), dict(scale=3 * P), dict(scale=4 * P),
               dict(scale=7 * P)):
        assert row8(lib, **kw) == INVALID, kw
    assert row(lib, rows=0, X=0, Y=0) == 0


def grad(lib, rows=4, D=8, dY=P, ldy=8, S=2 * P, lds=8, w=3 * P, eps=1e-6, dS=4 * P, ldds=8, dX=5 * P, lddx=8, dw=6 * P,
         db=8 * P, ws=7 * P, ws_bytes=1 << 16):
    return lib.sgemm_layernorm_f32_grad(rows, D, dY, ldy, S, lds, w, eps, dS, ldds, dX, lddx, dw, db, ws, ws_bytes, 0)


def workspace(fn, *args):
    n = ctypes.c_size_t()
    assert fn(*args, ctypes.byref(n)) == 0
    return n.value


def test_layer_norm_gradients_refused(lib):
    rows = 40
    need = workspace(lib.sgemm_layernorm_f32_grad_workspace, rows, 8)
    assert need > 0
    for kw in (dict(rows=-1), dict(D=0), dict(eps=-1.0), dict(dY=0), dict(S=0), dict(dX=0), dict(ldy=7), dict(lds=7),
               dict(ldds=7), dict(lddx=7), dict(dw=6 * P + 2), dict(db=8 * P + 2), dict(w=2), dict(dX=P), dict(dX=2 * P),
               dict(dX=3 * P), dict(dX=4 * P, ldds=9), dict(dw=P), dict(dw=5 * P), dict(dw=3 * P), dict(db=P),
               dict(db=5 * P), dict(db=6 * P), dict(db=6 * P + 16), dict(ws=0, ws_bytes=0), dict(ws_bytes=need - 1),
               dict(ws=7 * P + 4), dict(ws=P), dict(ws=5 * P), dict(ws=6 * P), dict(ws=8 * P)):
        assert grad(lib, **{"rows": rows, **kw}) == INVALID, kw
    # one of the sums alone still needs the workspace
    assert grad(lib, rows=rows, dw=0, ws=0, ws_bytes=0) == INVALID
    assert grad(lib, rows=rows, db=0, ws=0, ws_bytes=0) == INVALID
    n = ctypes.c_size_t()
    assert lib.sgemm_layernorm_f32_grad_workspace(-1, 8, ctypes.byref(n)) == INVALID
    assert lib.sgemm_layernorm_f32_grad_workspace(1, 0, ctypes.byref(n)) == INVALID
    assert lib.sgemm_layernorm_f32_grad_workspace(1, 8, None) == INVALID
    assert workspace(lib.sgemm_layernorm_f32_grad_workspace, 0, 8) == 0


# ---- norms over many tensors ---------------------------------------------------------------------------

def tensors(*entries):
    return (sg.SgemmTensor * max(len(entries), 1))(*[sg.SgemmTensor(*e) for e in entries])


GOOD = (P, 2 * P, 4, 8, 8, 8)
BAD_LISTS = {
    "negative rows": [(P, 2 * P, -1, 8, 8, 8)],
    "negative columns": [(P, 2 * P, 4, -8, 8, 8)],
    "no input": [(0, 2 * P, 4, 8, 8, 8)],
    "no output": [(P, 0, 4, 8, 8, 8)],
    "misaligned input": [(P + 2, 2 * P, 4, 8, 8, 8)],
    "misaligned output": [(P, 2 * P + 1, 4, 8, 8, 8)],
    "short input rows": [(P, 2 * P, 4, 8, 7, 8)],
    "short output rows": [(P, 2 * P, 4, 8, 8, 7)],
    "too many rows": [(P, P, 2 ** 31, 1, 1, 1)],
    "rows too long": [(P, P, 2, 2 ** 31, 2 ** 31, 2 ** 31)],
    "a run too long": [(P, P, 1, 2 ** 41, 0, 0)],
    "output half over its input": [(P, P + 16, 4, 8, 8, 8)],
    "output on its input with another stride": [(P, P, 4, 8, 8, 9)],
    "output over another's input": [GOOD, (3 * P, P, 4, 8, 8, 8)],
    "output over another's output": [GOOD, (3 * P, 2 * P + 64, 4, 8, 8, 8)],
    "a tensor twice in place": [(P, P, 4, 8, 8, 8), (P, P, 4, 8, 8, 8)],
    "columns that meet": [(P, P, 4, 8, 16, 16), (P + 28, P + 28, 4, 8, 16, 16)],
    "columns that wrap": [(P, P, 4, 8, 16, 16), (P + 64 * 2 - 4, P + 64 * 2 - 4, 2, 8, 16, 16)],
    "inside the workspace": [(P, 7 * P, 4, 8, 8, 8)],
    "input in the workspace": [(7 * P + 64, 2 * P, 4, 8, 8, 8)],
    "over the norm": [(P, 6 * P, 4, 8, 8, 8)],
    "input is the norm": [(6 * P, 2 * P, 1, 1, 1, 1)],
}


def clip(lib, entries, max_norm=1.0, eps=1e-6, norm=6 * P, ws=7 * P, ws_bytes=1 << 17, count=None):
    return lib.sgemm_clip_f32(len(entries) if count is None else count, tensors(*entries), max_norm, eps, norm, ws,
                              ws_bytes, 0)


@pytest.mark.parametrize("what", BAD_LISTS)
def test_lists_refused(lib, what):
    assert clip(lib, BAD_LISTS[what]) == INVALID


def test_clipping_refused(lib):
    need = workspace(lib.sgemm_clip_f32_workspace, 1)
    assert need > 0 and workspace(lib.sgemm_clip_f32_workspace, 1000) > need
    nan, inf = float("nan"), float("inf")
    for kw in (dict(max_norm=-1.0), dict(max_norm=nan), dict(max_norm=inf), dict(eps=-1.0), dict(eps=nan),
               dict(eps=inf), dict(norm=6 * P + 2), dict(ws=0, ws_bytes=0), dict(ws=7 * P + 8), dict(ws_bytes=need - 1),
               dict(count=-1), dict(norm=7 * P)):
        assert clip(lib, [GOOD], **kw) == INVALID, kw
    many = [(P + 256 * i, P + 256 * i, 4, 8, 8, 8) for i in range(100)]
    assert clip(lib, many, ws_bytes=need) == INVALID  # the table of a long list needs room
    norm = lambda entries, out=6 * P, ws=7 * P, n=1 << 17: lib.sgemm_norm_f32(len(entries), tensors(*entries), out, ws, n, 0)  # noqa: E731
    for bad in (norm([GOOD], out=0), norm([GOOD], out=P), norm([GOOD], ws=P), norm([GOOD], n=need - 1),
                norm([(0, 0, 4, 8, 8, 8)]), norm([(P, 0, 4, 8, 7, 8)])):
        assert bad == INVALID
    n = ctypes.c_size_t()
    assert lib.sgemm_clip_f32_workspace(-1, ctypes.byref(n)) == INVALID
    assert lib.sgemm_clip_f32_workspace(1, None) == INVALID


# ---- the binding ------------------------------------------------------------------------------------------

def test_host_tensors_and_types_are_refused():
    torch = pytest.importorskip("torch")
    x, q = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.uint8).view(torch.float8_e4m3fn)
    for call in (lambda: sg.layernorm(x), lambda: sg.layernorm_e4m3(x), lambda: sg.layernorm_backward(x, x),
                 lambda: sg.sgemm_gated(x, x, x), lambda: sg.gated_grad(x, x, x),
                 lambda: sg.sgemm_gated_backward(x, x, x, x, pre_gate=x, pre_up=x),
                 lambda: sg.gemm_e4m3_gated(q, None, q, None, q, None), lambda: sg.grad_norm([x]), lambda: sg.clip_grad_norm([x], 1.0), lambda: sg.grad_norm([]),
                 lambda: sg.clip_grad_norm([], 1.0)):
        with pytest.raises(ValueError):
            call()


def test_planes():
    """A tensor of any shape is one run if contiguous; else only rows with unit
    column stride are taken."""
    torch = pytest.importorskip("torch")
    from fp32_gemm_sgemm_amd import layers
    assert layers._plane(torch.zeros(3, 4, 5), "x") == (1, 60, 0)
    assert layers._plane(torch.zeros(()), "x") == (1, 1, 0)
    assert layers._plane(torch.zeros(4, 10)[:, :5], "x") == (4, 5, 10)
    for bad in (torch.zeros(4, 10).T, torch.zeros(4, 10, 6)[:, :, :3], torch.zeros(10)[::2], torch.zeros(1, 4).expand(3, 4)):
        with pytest.raises(ValueError):
            layers._plane(bad, "x")
    with pytest.raises(TypeError):
        layers._plane(torch.zeros(4, dtype=torch.float64), "x")
    host = torch.device("cpu")
    a, b = torch.zeros(4, 10)[:, :5], torch.zeros(4, 5)
    t = layers._tensor_list([a, b], [b, a], host)
    assert [(e.rows, e.cols, e.ldx, e.ldy) for e in t] == [(4, 5, 10, 5), (4, 5, 5, 10)]
    assert (t[0].x, t[0].y) == (a.data_ptr(), b.data_ptr())
    with pytest.raises(ValueError, match="shapes"):
        layers._tensor_list([a], [torch.zeros(5, 4)], host)


# ---- the reference itself ------------------------------------------------------------------------------------

def test_reference_layer_norm_gradient_is_the_derivative():
    rng = np.random.default_rng(0)
    s, w, b, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal(7), rng.standard_normal((3, 7))

    def f(s, w, b):
        return float((ref.layernorm(s, w, b, 1e-3)[0] * dy).sum())
    dx, dw, db, *_ = ref.layernorm_grad(dy, s, w, 1e-3)
    h = 1e-6
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(s)
            e[i, j] = h
            assert abs((f(s + e, w, b) - f(s - e, w, b)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros(7)
        e[j] = h
        assert abs((f(s, w + e, b) - f(s, w - e, b)) / (2 * h) - dw[j]) < 1e-7
        assert abs((f(s, w, b + e) - f(s, w, b - e)) / (2 * h) - db[j]) < 1e-7


def test_reference_gated_gradient_is_the_derivative():
    rng = np.random.default_rng(1)
    A, Bg, Bu, dy = (rng.standard_normal(s) for s in ((3, 4), (4, 5), (4, 5), (3, 5)))
    bg, bu = rng.standard_normal(5), rng.standard_normal(5)
    for name in ref.ref.ACTS:
        def f(A, Bg, Bu, bg, bu):
            return float((ref.gated(A, Bg, Bu, 4, bg, bu, name)[0] * dy).sum())
        _, G, U, *_ = ref.gated(A, Bg, Bu, 4, bg, bu, name)
        _, _, dbg, dbu, *_ = ref.gated_grad(dy, G, U, name)
        dA, dBg, dBu, *_ = ref.gated_backward(dy, A, Bg, Bu, G, U, name)
        h = 1e-6
        for k, want in enumerate((dA, dBg, dBu, dbg, dbu)):
            for i in np.ndindex(want.shape):
                args = [A, Bg, Bu, bg, bu]
                e = np.zeros_like(args[k])
                e[i] = h
                up, down = list(args), list(args)
                up[k], down[k] = args[k] + e, args[k] - e
                assert abs((f(*up) - f(*down)) / (2 * h) - want[i]) < 1e-6, (name, k, i)


# ---- the sizes that stand for the gated 8-bit kernels ---------------------------------------------------------

def test_gated_8_bit_cases_reach_their_kernels(tmp_path):
    planner = layers_cases.Planner(str(tmp_path))
    cases = layers_cases.E4M3_GATED
    plans = planner.plans([(m, n, k, al, ws) for _, m, n, k, al, ws, _ in cases])
    for case, (kernel, splits, _) in zip(cases, plans):
        assert (kernel, splits) == (case[0], case[6]), case
    for name, reg in planner.kernels():
        for aligned in (True, False) if reg else (True,):
            mine = [c for c in cases if c[0] == name and c[4] == aligned]
            assert mine, (name, aligned)
            if name in e4m3_cases.SKINNY:
                assert all(c[1] <= int(name[4:]) for c in mine)
                continue
            ks = [c[3] for c in mine if c[6] == 1]
            assert any(c[6] > 1 for c in mine) and any(k % 16 for k in ks), (name, aligned)
            assert min(ks) <= e4m3_cases.SLICE[name], (name, aligned)
            assert max(ks) > e4m3_cases.SLICE[name] * e4m3_cases.STAGES[name], (name, aligned)
