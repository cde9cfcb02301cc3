"""What a model's layer needs next to its products, for torch tensors: the C
ABI of include/sgemm_layers.h, argument marshalling only (the work is the
library's HIP kernels, and nothing falls back to another implementation).

Conventions are those of ops.py: 2-D float32 device tensors with unit column
stride and any row stride, 8-bit matrices as torch.float8_e4m3fn, one GPU a
call (not necessarily the current one), work enqueued on `stream` or on torch's
current one, no synchronisation.
"""
import ctypes
import functools

from .binding import GATED_AUTO, SgemmGate, SgemmTensor, _check, load
from .ops import (_MAX_DIM, _activation, _elsewhere, _empty, _empty_codes, _gpu_of, _handle, _matrix, _norm_inputs,
                  _rows, _same_gpu, _scratch, _supplied, _torch, _vector)


@functools.lru_cache(maxsize=256)
def _bytes_of(lib, name, index, *sizes):
    """The workspace that an entry point wants for these sizes on GPU `index`
    (the current one).  Kept: a call costs a microsecond, a tenth of a small one."""
    nbytes = ctypes.c_size_t(0)
    _check(getattr(lib, name)(*sizes, ctypes.byref(nbytes)), name)
    return nbytes.value


def _workspace(name, device, *sizes):
    """(tensor or None, address, bytes) of that workspace."""
    nbytes = _bytes_of(load(), name, device.index, *sizes)
    return (*_scratch(nbytes, device), nbytes)


# ---- the gated feed-forward block ------------------------------------------------------------

def _gate(device, M, N, activation, bias_gate, bias_up, pre_gate, pre_up):
    """SgemmGate of tensors that match an M x N output."""
    g = SgemmGate(activation=_activation(activation))
    if bias_gate is not None:
        g.bias_gate = _vector(bias_gate, N, device, "bias_gate")
    if bias_up is not None:
        g.bias_up = _vector(bias_up, N, device, "bias_up")
    if pre_gate is not None:
        g.ld_pre_gate, g.pre_gate = _matrix(pre_gate, M, N, device, "pre_gate"), pre_gate.data_ptr()
    if pre_up is not None:
        g.ld_pre_up, g.pre_up = _matrix(pre_up, M, N, device, "pre_up"), pre_up.data_ptr()
    return g


def _weights(B_gate, B_up, transb, device):
    """(K, N, row strides) of a gated block's weights."""
    _same_gpu(device, B_gate, "B_gate")
    _same_gpu(device, B_up, "B_up")
    rows, cols, ldg = _rows(B_gate, "B_gate")
    r, c, ldu = _rows(B_up, "B_up")
    if (r, c) != (rows, cols):
        raise ValueError(f"B_gate and B_up must have one shape, got {(rows, cols)} and {(r, c)}")
    return (cols, rows, ldg, ldu) if transb else (rows, cols, ldg, ldu)


def sgemm_gated(A, B_gate, B_up, *, bias_gate=None, bias_up=None, activation="silu", pre_gate=None, pre_up=None,
                out=None, transb=False, workspace=True, stream=None, form=GATED_AUTO):
    """act(A @ op(B_gate) + bias_gate) * (A @ op(B_up) + bias_up): both
    projections of a gated feed-forward block, the activation and the product in
    one call.

    A is M x K, the weights are K x N each, or N x K with `transb` (one row per
    output); they may be the two halves of one tensor.  `activation` is a name of
    ACTIVATIONS.  `pre_gate` and `pre_up`, if given, receive the two projections
    with their biases, which sgemm_gated_backward() needs.  `workspace` as for
    sgemm(), `form` a forced form (GATED_* of sgemm_layers.h).
    """
    torch = _torch()
    device = _gpu_of(A, "A")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return sgemm_gated(A, B_gate, B_up, bias_gate=bias_gate, bias_up=bias_up, activation=activation,
                               pre_gate=pre_gate, pre_up=pre_up, out=out, transb=transb, workspace=workspace,
                               form=form)
    M, K, lda = _rows(A, "A")
    K2, N, ldg, ldu = _weights(B_gate, B_up, transb, device)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    tb = 1 if transb else 0
    if out is None:
        out, ldc = _empty((M, N), device), max(N, 1)
    else:
        ldc = _matrix(out, M, N, device, "out")
    g = _gate(device, M, N, activation, bias_gate, bias_up, pre_gate, pre_up)
    operands = (tb, M, N, K, A.data_ptr(), lda, B_gate.data_ptr(), ldg, B_up.data_ptr(), ldu)
    ws, ws_ptr, ws_bytes = None, None, 0
    if isinstance(workspace, torch.Tensor):
        ws_ptr, ws_bytes = _supplied(workspace, device)
    elif workspace:
        nbytes = ctypes.c_size_t(0)
        _check(load().sgemm_f32_gated_workspace(*operands, ctypes.byref(nbytes)), "sgemm_f32_gated_workspace")
        ws_bytes = nbytes.value
        ws, ws_ptr = _scratch(ws_bytes, device)
    code = load().sgemm_f32_gated(*operands, out.data_ptr(), ldc, ctypes.byref(g), ws_ptr, ws_bytes, form,
                                  _handle(device))
    del ws
    _check(code, "sgemm_f32_gated")
    return out


def gated_grad(grad, pre_gate, pre_up, activation="silu", *, out_gate=None, out_up=None, dbias_gate=None,
               dbias_up=None, stream=None):
    """(dG, dU, dbias_gate, dbias_up) from the gradient of act(G) * U, G and U as
    sgemm_gated() stored them: dG = grad * U * act'(G), dU = grad * act(G) and
    their column sums, in one pass.

    `out_gate`, `out_up`: a tensor to write (any of the three inputs for in
    place), None for a new one, or False for none.  `dbias_gate`, `dbias_up`: a
    tensor of N values, None for a new one, or False for none.
    """
    device = _gpu_of(grad, "grad")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gated_grad(grad, pre_gate, pre_up, activation, out_gate=out_gate, out_up=out_up,
                              dbias_gate=dbias_gate, dbias_up=dbias_up)
    M, N, ldy = _rows(grad, "grad")
    act = _activation(activation)
    ldg, ldu = _matrix(pre_gate, M, N, device, "pre_gate"), _matrix(pre_up, M, N, device, "pre_up")
    outs, sums = [], []
    for name, t in (("out_gate", out_gate), ("out_up", out_up)):
        if t is False:
            outs.append((None, None, 0))
        elif t is None:
            t = _empty((M, N), device)
            outs.append((t, t.data_ptr(), max(N, 1)))
        else:
            outs.append((t, t.data_ptr(), _matrix(t, M, N, device, name)))
    for name, t in (("dbias_gate", dbias_gate), ("dbias_up", dbias_up)):
        if t is False:
            sums.append((None, None))
        else:
            t = _empty((N,), device) if t is None else t
            sums.append((t, _vector(t, N, device, name)))
    _gate_grad(M, N, act, grad, ldy, pre_gate, ldg, pre_up, ldu, *outs[0][1:], *outs[1][1:], sums[0][1], sums[1][1],
               device)
    return outs[0][0], outs[1][0], sums[0][0], sums[1][0]


def _gate_grad(M, N, act, grad, ldy, pre_gate, ldg, pre_up, ldu, dg, lddg, du, lddu, bias_gate, bias_up, device):
    """The call with checked tensors and the outputs' addresses."""
    ws, ws_ptr, nbytes = None, None, 0
    if bias_gate is not None or bias_up is not None:
        ws, ws_ptr, nbytes = _workspace("sgemm_f32_gated_grad_workspace", device, M, N)
    code = load().sgemm_f32_gated_grad(M, N, act, grad.data_ptr(), ldy, pre_gate.data_ptr(), ldg, pre_up.data_ptr(),
                                       ldu, dg, lddg, du, lddu, bias_gate, bias_up, ws_ptr, nbytes, _handle(device))
    del ws
    _check(code, "sgemm_f32_gated_grad")


def _products(batch, ta, tb, M, N, K, x, ldx, sx, y, ldy, sy, out, ldo, so, workspace, device):
    """out = op(X) op(Y) over a batch, of checked operands' addresses."""
    ws, ws_ptr, ws_bytes = None, None, 0
    if isinstance(workspace, _torch().Tensor):
        ws_ptr, ws_bytes = _supplied(workspace, device)
    elif workspace and M and N and K:
        ws, ws_ptr, ws_bytes = _workspace("sgemm_f32_workspace_size", device, ta, tb, M, N, K, ldx, ldy, ldo, batch)
    code = load().sgemm_f32_ex(ta, tb, M, N, K, 1.0, x, ldx, sx, y, ldy, sy, 0.0, out, ldo, so, batch, ws_ptr,
                               ws_bytes, _handle(device), None)
    del ws
    _check(code, "sgemm_f32_ex")


def _pair(tb, M, N, K, x1, x2, ldx, y1, ldy1, y2, ldy2, out, ldo, workspace, device):
    """out = X1 op(Y1) + X2 op(Y2) of checked operands' addresses."""
    operands = (tb, M, N, K, x1, x2, ldx, y1, ldy1, y2, ldy2)
    ws, ws_ptr, ws_bytes = None, None, 0
    if isinstance(workspace, _torch().Tensor):
        ws_ptr, ws_bytes = _supplied(workspace, device)
    elif workspace:
        nbytes = ctypes.c_size_t(0)
        _check(load().sgemm_f32_pair_workspace(*operands, ctypes.byref(nbytes)), "sgemm_f32_pair_workspace")
        ws_bytes = nbytes.value
        ws, ws_ptr = _scratch(ws_bytes, device)
    code = load().sgemm_f32_pair(*operands, out, ldo, ws_ptr, ws_bytes, _handle(device))
    del ws
    _check(code, "sgemm_f32_pair")


def sgemm_gated_backward(grad, A, B_gate, B_up, *, pre_gate, pre_up, activation="silu", transb=False,
                         need=("A", "B", "bias"), workspace=True, stream=None):
    """Gradients of y = act(A @ op(B_gate) + bias_gate) * (A @ op(B_up) + bias_up)
    from y's: (dA, dB_gate, dB_up, dbias_gate, dbias_up), None for those `need`
    does not name.

    `pre_gate` and `pre_up` hold what sgemm_gated() stored there.  Where the
    weights are the two halves of one tensor (side by side, or with `transb` one
    below the other; the gate's first or second), dB_gate and dB_up are the
    halves of one tensor too, in the same order.
    `workspace` as for sgemm(): one given as a tensor is used by the products,
    one after the other.
    """
    device = _gpu_of(grad, "grad")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return sgemm_gated_backward(grad, A, B_gate, B_up, pre_gate=pre_gate, pre_up=pre_up,
                                        activation=activation, transb=transb, need=need, workspace=workspace)
    _same_gpu(device, A, "A")
    M, K, lda = _rows(A, "A")
    K2, N, ldg, ldu = _weights(B_gate, B_up, transb, device)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    ldy = _matrix(grad, M, N, device, "grad")
    ldpg, ldpu = _matrix(pre_gate, M, N, device, "pre_gate"), _matrix(pre_up, M, N, device, "pre_up")
    act, tb = _activation(activation), 1 if transb else 0
    torch = _torch()
    # one tensor of both weights: its products are single ones of twice the size
    apart = B_up.data_ptr() - B_gate.data_ptr()
    merged = ldg == ldu and abs(apart) == 4 * N * (ldg if transb else 1) and (transb or ldg >= 2 * N)
    swapped = merged and apart < 0  # (the gate's half is the second)
    # dG and dU side by side in the weights' order; halves that products read one by one start 16-byte aligned
    half = N if merged else (N + 3) & ~3
    ld = max((2 * half + 3) & ~3, 4)
    dA = dB = dB_gate = dB_up = dbias_gate = dbias_up = dz = z = dg = du = bias = None
    if "A" in need or "B" in need:
        dz = torch.empty_strided((M, 2 * half), (ld, 1), dtype=torch.float32, device=device)
        z = dz.data_ptr()
        dg, du = (z + 4 * half, z) if swapped else (z, z + 4 * half)
    if "bias" in need:
        dbias_gate, dbias_up = _empty((N,), device), _empty((N,), device)
        bias = dbias_gate.data_ptr(), dbias_up.data_ptr()
    _gate_grad(M, N, act, grad, ldy, pre_gate, ldpg, pre_up, ldpu, dg, ld, du, ld, *(bias or (None, None)), device)
    a, k = A.data_ptr(), max(K, 1)
    if "A" in need:
        dA = _empty((M, K), device)
        if merged:
            both = (B_up if swapped else B_gate).data_ptr()
            _products(1, 0, 1 - tb, M, K, 2 * N, z, ld, 0, both, ldg, 0, dA.data_ptr(), k, 0, workspace, device)
        else:
            _pair(1 - tb, M, K, N, dg, du, ld, B_gate.data_ptr(), ldg, B_up.data_ptr(), ldu, dA.data_ptr(), k, workspace,
                  device)
    if "B" in need:
        if transb:
            dB = _empty((2, N, K), device)
            _products(2, 1, 0, N, K, M, z, ld, half, a, lda, 0, dB.data_ptr(), k, N * K, workspace, device)
        elif merged:
            dB = _empty((K, 2 * N), device)
            _products(1, 1, 0, K, 2 * N, M, a, lda, 0, z, ld, 0, dB.data_ptr(), max(2 * N, 1), 0, workspace, device)
        else:
            dB = _empty((2, K, N), device)
            _products(2, 1, 0, K, N, M, a, lda, 0, z, ld, half, dB.data_ptr(), max(N, 1), K * N, workspace, device)
        halves = (dB[:, :N], dB[:, N:]) if merged and not transb else (dB[0], dB[1])
        dB_gate, dB_up = halves[::-1] if swapped else halves
    return dA, dB_gate, dB_up, dbias_gate, dbias_up


def gemm_e4m3_gated(A, scale_a, B_gate, scale_gate, B_up, scale_up, *, bias_gate=None, bias_up=None,
                    activation="silu", pre_gate=None, pre_up=None, out=None, workspace=True, stream=None):
    """sgemm_gated() for 8-bit A (M x K) and weights (N x K, one row per output),
    in float32: act((scale_a[:, None] * A) @ (scale_gate[:, None] * B_gate).T +
    bias_gate) times the same of B_up.

    Scales are M and N float32 factors, or None for ones.
    """
    torch = _torch()
    device = _gpu_of(A, "A")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemm_e4m3_gated(A, scale_a, B_gate, scale_gate, B_up, scale_up, bias_gate=bias_gate,
                                   bias_up=bias_up, activation=activation, pre_gate=pre_gate, pre_up=pre_up, out=out,
                                   workspace=workspace)
    codes = torch.float8_e4m3fn
    M, K, lda = _rows(A, "A", codes)
    _same_gpu(device, B_gate, "B_gate")
    _same_gpu(device, B_up, "B_up")
    N, K2, ldg = _rows(B_gate, "B_gate", codes)
    r, c, ldu = _rows(B_up, "B_up", codes)
    if (r, c) != (N, K2):
        raise ValueError(f"B_gate and B_up must have one shape, got {(N, K2)} and {(r, c)}")
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    sa = _vector(scale_a, M, device, "scale_a") if scale_a is not None else None
    sg = _vector(scale_gate, N, device, "scale_gate") if scale_gate is not None else None
    su = _vector(scale_up, N, device, "scale_up") if scale_up is not None else None
    if out is None:
        out, ldc = _empty((M, N), device), max(N, 1)
    else:
        ldc = _matrix(out, M, N, device, "out")
    g = _gate(device, M, N, activation, bias_gate, bias_up, pre_gate, pre_up)
    ws, ws_ptr, ws_bytes = None, None, 0
    if isinstance(workspace, torch.Tensor):
        ws_ptr, ws_bytes = _supplied(workspace, device)
    elif workspace:
        ws, ws_ptr, ws_bytes = _workspace("sgemm_e4m3_gated_workspace", device, M, N, K)
    code = load().sgemm_e4m3_gated(M, N, K, A.data_ptr(), lda, sa, B_gate.data_ptr(), ldg, sg, B_up.data_ptr(), ldu,
                                   su, out.data_ptr(), ldc, ctypes.byref(g), ws_ptr, ws_bytes, _handle(device))
    del ws
    _check(code, "sgemm_e4m3_gated")
    return out


# ---- layer norm ----------------------------------------------------------------------------

def layernorm(x, weight=None, bias=None, *, eps=1e-5, residual=None, sum_out=None, out=None, stream=None):
    """(y, s): s = x + residual, y = (s - mean(s)) / sqrt(var(s) + eps) * weight
    + bias, per row (var the mean squared difference from the mean).

    Without `residual`, s is x itself (and lost where `out` is x).  `sum_out`
    receives s (it may be `x` or `residual`, which then holds the residual
    stream updated in place).
    """
    device = _gpu_of(x, "x")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return layernorm(x, weight, bias, eps=eps, residual=residual, sum_out=sum_out, out=out)
    rows, D, ldx, w, r, ldr, s_ptr, lds, s = _norm_inputs(x, weight, residual, sum_out, device)
    b = _vector(bias, D, device, "bias") if bias is not None else None
    if out is None:
        out, ldy = _empty((rows, D), device), D
    else:
        ldy = _matrix(out, rows, D, device, "out")
    _check(load().sgemm_layernorm_f32(rows, D, x.data_ptr(), ldx, r, ldr, w, b, float(eps), s_ptr, lds,
                                      out.data_ptr(), ldy, _handle(device)), "sgemm_layernorm_f32")
    return out, s


def layernorm_e4m3(x, weight=None, bias=None, *, eps=1e-5, residual=None, sum_out=None, stream=None):
    """(q, scale, s): layernorm() with y in 8 bits, q * scale[:, None] standing
    for y; gemm_e4m3() and gemm_e4m3_gated() take q and scale as they are."""
    device = _gpu_of(x, "x")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return layernorm_e4m3(x, weight, bias, eps=eps, residual=residual, sum_out=sum_out)
    rows, D, ldx, w, r, ldr, s_ptr, lds, s = _norm_inputs(x, weight, residual, sum_out, device)
    b = _vector(bias, D, device, "bias") if bias is not None else None
    (q, ldq), scale = _empty_codes(rows, D, device), _empty((rows,), device)
    _check(load().sgemm_layernorm_e4m3(rows, D, x.data_ptr(), ldx, r, ldr, w, b, float(eps), s_ptr, lds,
                                       q.data_ptr(), ldq, scale.data_ptr(), _handle(device)), "sgemm_layernorm_e4m3")
    return q, scale, s


def layernorm_backward(grad, s, weight=None, *, eps=1e-5, dsum=None, out=None, need_weight=True, need_bias=True,
                       stream=None):
    """(dx, dweight, dbias) from layernorm()'s y's gradient; `s` is the sum it
    returned.

    dx is the gradient of x and of the residual.  `dsum`, the gradient that
    reaches s past the norm (down the residual stream), is added to it; `out`
    may be `dsum`.  dweight is None without `weight` or with need_weight false,
    dbias with need_bias false.
    """
    device = _gpu_of(grad, "grad")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return layernorm_backward(grad, s, weight, eps=eps, dsum=dsum, out=out, need_weight=need_weight,
                                      need_bias=need_bias)
    rows, D, ldy = _rows(grad, "grad")
    if D < 1:
        raise ValueError("rows need at least one value")
    lds = _matrix(s, rows, D, device, "s")
    g, ldds = None, 0
    if dsum is not None:
        ldds, g = _matrix(dsum, rows, D, device, "dsum"), dsum.data_ptr()
    w = _vector(weight, D, device, "weight") if weight is not None else None
    if out is None:
        out, lddx = _empty((rows, D), device), D
    else:
        lddx = _matrix(out, rows, D, device, "out")
    dw = _empty((D,), device) if weight is not None and need_weight else None
    db = _empty((D,), device) if need_bias else None
    ws, ws_ptr, nbytes = None, None, 0
    if dw is not None or db is not None:
        ws, ws_ptr, nbytes = _workspace("sgemm_layernorm_f32_grad_workspace", device, rows, D)
    code = load().sgemm_layernorm_f32_grad(
        rows, D, grad.data_ptr(), ldy, s.data_ptr(), lds, w, float(eps), g, ldds, out.data_ptr(), lddx,
        dw.data_ptr() if dw is not None else None, db.data_ptr() if db is not None else None, ws_ptr, nbytes,
        _handle(device))
    del ws
    _check(code, "sgemm_layernorm_f32_grad")
    return out, dw, db


# ---- norms over many tensors ------------------------------------------------------------------

def _plane(t, name):
    """(rows, cols, row stride) of a tensor of any shape whose elements are one
    run, or of a 2-D one with unit column stride."""
    if t.dtype != _torch().float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.is_contiguous():
        return 1, t.numel(), 0
    if t.dim() != 2:
        raise ValueError(f"{name} must be contiguous, or 2-D with unit column stride")
    return _rows(t, name)


def _tensor_list(tensors, out, device):
    """The C array of the tensors (and of what is written for each)."""
    flat, float32, index = [], _torch().float32, device.index
    for i, x in enumerate(tensors):
        # (the common case first: a list of many little tensors is a call's whole time)
        if x.dtype is float32 and x.is_contiguous():
            rows, cols, ldx = 1, x.numel(), 0
        else:
            rows, cols, ldx = _plane(x, "a tensor")
        if x.get_device() != index:
            _same_gpu(device, x, "a tensor")
        ptr = x.data_ptr()
        if out is None:
            flat += (ptr, ptr, rows, cols, ldx, ldx)
            continue
        to = out[i]
        if to.shape != x.shape:
            raise ValueError(f"out must have the tensors' shapes: {tuple(to.shape)} for {tuple(x.shape)}")
        if to.get_device() != index:
            _same_gpu(device, to, "out")
        if to.dtype is float32 and to.is_contiguous():
            orows, ocols, ldy = 1, cols if rows == 1 else to.numel(), 0
        else:
            orows, ocols, ldy = _plane(to, "out")
        if orows != rows or ocols != cols:
            # one of the two is a run and the other has gaps between its rows
            rows, cols = x.shape
            ldx, ldy = ldx or cols, ldy or cols
        flat += (ptr, to.data_ptr(), rows, cols, ldx, ldy)
    return (SgemmTensor * len(tensors)).from_buffer((ctypes.c_longlong * len(flat))(*flat))


def _many(tensors, out, device, call):
    """Runs call(count, array, norm address, workspace address, bytes); the norm
    as a tensor without dimensions."""
    torch = _torch()
    array = _tensor_list(tensors, out, device)
    ws, ws_ptr, nbytes = _workspace("sgemm_clip_f32_workspace", device, len(tensors))
    norm = torch.empty_strided((), (), dtype=torch.float32, device=device)
    call(len(tensors), array, norm.data_ptr(), ws_ptr, nbytes)
    del ws
    return norm


def _list_device(tensors):
    if not tensors:
        raise ValueError("at least one tensor is needed")
    if len(tensors) > _MAX_DIM:
        raise ValueError(f"no more than {_MAX_DIM} tensors")
    return _gpu_of(tensors[0], "a tensor")


def grad_norm(tensors, *, stream=None):
    """The Euclidean norm of all elements of a list of float32 tensors (a
    tensor without dimensions, on the GPU).

    Each is contiguous, of any shape, or 2-D with unit column stride (such as a
    half of a gated layer's weight gradient).
    """
    tensors = list(tensors)
    device = _list_device(tensors)
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return grad_norm(tensors)

    def call(count, array, norm, ws, nbytes):
        _check(load().sgemm_norm_f32(count, array, norm, ws, nbytes, _handle(device)), "sgemm_norm_f32")
    return _many(tensors, None, device, call)


def clip_grad_norm(tensors, max_norm, *, eps=1e-6, out=None, stream=None):
    """Scales a list of float32 tensors by min(1, max_norm / (norm + eps)), norm
    that of all their elements, which is returned (on the GPU, as grad_norm()).

    The tensors are scaled in place, or `out`, a list of tensors of the same
    shapes, receives the scaled ones and they are left as they are.  No two may
    share memory (name a shared tensor once).  Nothing waits for the GPU, so a
    norm that is not finite is the caller's to look at.
    """
    tensors = list(tensors)
    device = _list_device(tensors)
    if out is not None:
        out = list(out)
        if len(out) != len(tensors):
            raise ValueError(f"out must hold {len(tensors)} tensors, got {len(out)}")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return clip_grad_norm(tensors, max_norm, eps=eps, out=out)

    def call(count, array, norm, ws, nbytes):
        _check(load().sgemm_clip_f32(count, array, float(max_norm), float(eps), norm, ws, nbytes, _handle(device)),
               "sgemm_clip_f32")
    return _many(tensors, out, device, call)
