"""The operators around a matrix product for torch tensors: the C ABI of
include/sgemm_ops.h, argument marshalling only (the work is the library's HIP
kernels, and nothing falls back to another implementation).

Matrices are 2-D (a product's may be 3-D batches) float32 device tensors with
unit column stride and any row stride; 8-bit matrices are torch.float8_e4m3fn.
All tensors of a call are on one GPU, which need not be the current one.  Work
is enqueued on `stream` (default: torch's current stream of that GPU) and
nothing synchronises.  What a call allocates (outputs, workspaces) it allocates
on the stream it runs on, as torch does under `torch.cuda.stream(stream)`.
"""
import ctypes

from .binding import (ACTIVATIONS, SgemmEpilogue, _check, load, sgemm_f32_cfg_geometry,
                      sgemm_f32_workspace_size)

E4M3_MAX = 448.0
_MAX_DIM = 2**31 - 1 - 1024  # largest size, row stride or batch the C ABI takes
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _elsewhere(device, stream):
    """None where `device` is the current GPU and `stream` its current stream;
    else the context that makes them so (a call enters it and starts again)."""
    torch = _torch()
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            handle = int(stream)
            stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
        if stream != torch.cuda.current_stream(device):
            return torch.cuda.stream(stream)
    # (the tensors are on a GPU, so torch has set it up: current_device() would look again)
    if torch._C._cuda_getDevice() != device.index:
        return torch.cuda.device(device)
    return None


def _handle(device):
    # (the handle alone: a Stream object costs 2 us, a sixth of a small call)
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _gpu_of(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _same_gpu(device, t, name):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _activation(name):
    if name is None:
        return 0
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _rows(t, name, dtype=None):
    """(rows, cols, row stride) of a 2-D tensor with unit column stride."""
    want = _torch().float32 if dtype is None else dtype
    if t.dtype != want:
        raise TypeError(f"{name} must be {str(want).split('.')[-1]}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name}'s rows must not overlap (row stride {ld}, {cols} columns)")
    if rows > _MAX_DIM or cols > _MAX_DIM or ld > _MAX_DIM:
        raise ValueError(f"{name}'s sizes and row stride must not pass {_MAX_DIM}")
    return rows, cols, ld if ld > 0 else 1


def _matrix(t, rows, cols, device, name):
    """Row stride of a 2-D float32 tensor of the given shape."""
    r, c, ld = _rows(t, name)
    if r != rows or c != cols:
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {(r, c)}")
    _same_gpu(device, t, name)
    return ld


def _vector(t, n, device, name):
    if t.dtype != _torch().float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _same_gpu(device, t, name)
    return t.data_ptr()


def _empty(shape, device):
    torch = _torch()
    # (empty() takes a third longer, 0.4 us of a small call's 8 to 16)
    if len(shape) == 2:
        return torch.empty_strided(shape, (max(shape[1], 1), 1), dtype=torch.float32, device=device)
    if len(shape) == 1:
        return torch.empty_strided(shape, (1,), dtype=torch.float32, device=device)
    return torch.empty(shape, dtype=torch.float32, device=device)


def _empty_codes(rows, cols, device):
    """8-bit rows that start 16-byte aligned, as the product reads fastest;
    (tensor, row stride)."""
    torch = _torch()
    ld = (cols + 15) & ~15
    # (one call: a slice of an empty() costs 1.2 us more, a tenth of a small quantisation)
    return torch.empty_strided((rows, cols), (ld, 1), dtype=torch.float8_e4m3fn, device=device), ld


def _scratch(nbytes, device):
    """(tensor or None, address) of a workspace."""
    if nbytes <= 0:
        return None, None
    torch = _torch()
    ws = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
    return ws, ws.data_ptr()


def _supplied(workspace, device):
    """(address, bytes) of a caller's workspace tensor."""
    if workspace.device != device:
        raise ValueError("workspace must be a device tensor on the operands' GPU")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _batch_view(t, name):
    """(batch, rows, cols, row stride, batch stride) of a 2-D or 3-D float32 tensor."""
    if t.dim() == 2:
        return (1, *_rows(t, name), 0)
    if t.dim() != 3:
        raise ValueError(f"{name} must be 2-D or 3-D")
    n = t.shape[0]
    if n > _MAX_DIM:
        raise ValueError(f"{name} must not have more than {_MAX_DIM} batch entries")
    return (n, *_rows(t[0] if n else t.new_empty(t.shape[1:]), name), t.stride(0) if n > 1 else 0)


def _epilogue(device, batch, M, N, bias, activation, pre, grad_pre, residual):
    """SgemmEpilogue of tensors that match a batch x M x N output (2-D ones are
    shared by the batch, but for `pre`)."""
    e = SgemmEpilogue(activation=_activation(activation))
    if pre is not None and grad_pre is not None:
        raise ValueError("pre and grad_pre exclude each other")
    if bias is not None:
        if bias.dim() == 2 and bias.shape[0] == batch:
            e.stride_bias = bias.stride(0) if batch > 1 else 0
            if batch:
                _vector(bias[0], N, device, "bias")
            e.bias = bias.data_ptr()
        else:
            e.bias = _vector(bias, N, device, "bias")
    for name, t in (("pre", pre), ("grad_pre", grad_pre), ("residual", residual)):
        if t is None:
            continue
        b, rows, cols, ld, stride = _batch_view(t, name)
        if rows != M or cols != N or (b != batch and (b != 1 or name == "pre")):
            raise ValueError(f"{name} must have shape {(M, N)}, got {tuple(t.shape)}")
        _same_gpu(device, t, name)
        setattr(e, name, t.data_ptr())
        setattr(e, "ld_" + name, ld)
        setattr(e, "stride_" + name, stride)
    return e


def sgemm_epilogue(A, B, *, bias=None, activation=None, residual=None, out=None, pre=None, grad_pre=None,
                   alpha=1.0, transa=False, transb=False, workspace=True, stream=None, cfg=None):
    """act(alpha * op(A) @ op(B) + bias) + residual in one product.

    A and B as for sgemm() (2-D) or sgemm_batched() (3-D, batch sizes equal or
    1).  `bias` holds N values (or one row of N per batch entry), `activation`
    is a name of ACTIVATIONS, `residual` has the output's shape and may be
    `out` itself (the product is then added to it in place).  `pre`, if given,
    receives alpha * op(A) @ op(B) + bias, which the gradient needs.  With
    `grad_pre` the product is instead multiplied by act'(grad_pre): the
    gradient that goes on into the layer whose pre-activations it holds.
    `workspace` as for sgemm(), `cfg` a forced configuration.
    """
    torch = _torch()
    device = _gpu_of(A, "A")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return sgemm_epilogue(A, B, bias=bias, activation=activation, residual=residual, out=out, pre=pre,
                                  grad_pre=grad_pre, alpha=alpha, transa=transa, transb=transb,
                                  workspace=workspace, cfg=cfg)
    _same_gpu(device, B, "B")
    batched = A.dim() == 3 or B.dim() == 3
    ba, ra, ca, lda, sa = _batch_view(A, "A")
    bb, rb, cb, ldb, sb = _batch_view(B, "B")
    M, K = (ca, ra) if transa else (ra, ca)
    K2, N = (cb, rb) if transb else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    batch = bb if ba == 1 else ba
    if bb not in (1, batch):
        raise ValueError("batch sizes differ")
    ta, tb = 1 if transa else 0, 1 if transb else 0
    if out is None:
        out, ldc, sc = _empty((batch, M, N) if batched else (M, N), device), max(N, 1), M * N
    else:
        bo, Mo, No, ldc, sc = _batch_view(out, "out")
        if (bo, Mo, No) != (batch, M, N) or (out.dim() == 3) != batched:
            raise ValueError("out has the wrong shape")
        _same_gpu(device, out, "out")
    e = _epilogue(device, batch, M, N, bias, activation, pre, grad_pre, residual)
    ws, ws_ptr, ws_bytes = None, None, 0
    if isinstance(workspace, torch.Tensor):
        ws_ptr, ws_bytes = _supplied(workspace, device)
    elif workspace and M and N and K and batch:
        if cfg is None:
            ws_bytes = sgemm_f32_workspace_size(ta, tb, M, N, K, lda, ldb, ldc, batch)
        elif cfg.splits > 1:
            ws_bytes = sgemm_f32_cfg_geometry(cfg, ta, tb, M, N, K, lda, ldb, ldc, batch).workspace_bytes
        ws, ws_ptr = _scratch(ws_bytes, device)
    code = load().sgemm_f32_epilogue(
        ta, tb, M, N, K, float(alpha), A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, out.data_ptr(), ldc, sc,
        batch, ctypes.byref(e), ws_ptr, ws_bytes, _handle(device), ctypes.byref(cfg) if cfg is not None else None)
    del ws
    _check(code, "sgemm_f32_epilogue")
    return out


def activation_grad(grad, pre=None, activation=None, *, out=None, dbias=None, stream=None):
    """(dZ, dbias) from the gradient of a layer's output: dZ = grad * act'(pre),
    dbias = dZ's column sums, in one pass.

    `out`: a tensor for dZ (`grad` itself for in place), None for a new one, or
    False for none.  `dbias`: a tensor of N values, None for a new one, or
    False for none.  `pre` is read only with an activation.
    """
    device = _gpu_of(grad, "grad")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return activation_grad(grad, pre, activation, out=out, dbias=dbias)
    M, N, ldy = _rows(grad, "grad")
    act = _activation(activation)
    if act and pre is None:
        raise ValueError("an activation's gradient needs `pre`")
    ldz = _matrix(pre, M, N, device, "pre") if act else 0
    if out is None:
        out, ldo = _empty((M, N), device), max(N, 1)
    elif out is False:
        out, ldo = None, 0
    else:
        ldo = _matrix(out, M, N, device, "out")
    ws, ws_ptr, nbytes = None, None, ctypes.c_size_t(0)
    if dbias is False:
        dbias = None
    else:
        if dbias is None:
            dbias = _empty((N,), device)
        else:
            _vector(dbias, N, device, "dbias")
        _check(load().sgemm_f32_activation_grad_workspace(M, N, ctypes.byref(nbytes)),
               "sgemm_f32_activation_grad_workspace")
        ws, ws_ptr = _scratch(nbytes.value, device)
    code = load().sgemm_f32_activation_grad(
        M, N, act, grad.data_ptr(), ldy, pre.data_ptr() if act else None, ldz,
        out.data_ptr() if out is not None else None, ldo, dbias.data_ptr() if dbias is not None else None,
        ws_ptr, nbytes.value, _handle(device))
    del ws
    _check(code, "sgemm_f32_activation_grad")
    return out, dbias


def sgemm_epilogue_backward(grad, A, B, *, pre=None, activation=None, a_pre=None, a_activation=None,
                            alpha=1.0, transa=False, transb=False, need=("A", "B", "bias"),
                            workspace=True, stream=None):
    """Gradients of y = act(alpha * op(A) @ op(B) + bias) + residual (2-D) from
    y's: (dA, dB, dbias), None for those `need` does not name.  The residual's
    gradient is `grad` itself.

    `pre` holds the pre-activations that sgemm_epilogue() stored (needed with
    an activation).  With `a_pre` and `a_activation`, A is taken for the
    activations of a layer below, act_a(a_pre): dA is then the gradient of
    a_pre (that layer's `grad` with no activation left), the product's epilogue
    doing the multiplication.  `workspace` as for sgemm(): one given as a tensor
    is used by the products, one after the other.
    """
    device = _gpu_of(grad, "grad")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return sgemm_epilogue_backward(grad, A, B, pre=pre, activation=activation, a_pre=a_pre,
                                           a_activation=a_activation, alpha=alpha, transa=transa, transb=transb,
                                           need=need, workspace=workspace)
    _same_gpu(device, A, "A")
    _same_gpu(device, B, "B")
    ra, ca, lda = _rows(A, "A")
    rb, cb, ldb = _rows(B, "B")
    M, K = (ca, ra) if transa else (ra, ca)
    K2, N = (cb, rb) if transb else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    ldz = _matrix(grad, M, N, device, "grad")
    act, a_act = _activation(activation), _activation(a_activation)
    below = None
    if a_act:
        if a_pre is None:
            raise ValueError("a_activation needs `a_pre`")
        ld = _matrix(a_pre, ra, ca, device, "a_pre")
        below = SgemmEpilogue(activation=a_act, grad_pre=a_pre.data_ptr(), ld_grad_pre=ld)
    dz, dbias, dA, dB = grad, None, None, None
    products = "A" in need or "B" in need
    if "bias" in need or (act and products):
        dz, dbias = activation_grad(grad, pre, activation, out=None if act and products else False,
                                    dbias=None if "bias" in need else False)
        dz, ldz = (grad, ldz) if dz is None else (dz, max(N, 1))
    a, b, z = (A, lda), (B, ldb), (dz, ldz)
    if "A" in need:
        x, y, tx, ty = (b, z, transb, True) if transa else (z, b, False, not transb)
        dA = _product(x, tx, y, ty, ra, ca, N, alpha, workspace, device, below)
    if "B" in need:
        x, y, tx, ty = (z, a, True, transa) if transb else (a, z, not transa, False)
        dB = _product(x, tx, y, ty, rb, cb, M, alpha, workspace, device)
    return dA, dB, dbias


def _product(x, tx, y, ty, M, N, K, alpha, workspace, device, epilogue=None):
    """alpha * op(X) @ op(Y) (M x N, inner size K) of checked (tensor, row
    stride) pairs, through `epilogue` if given: sgemm()'s product without its
    checks, which cost a small gradient 8 us a product."""
    (X, ldx), (Y, ldy), tx, ty = x, y, 1 if tx else 0, 1 if ty else 0
    out, ldo = _empty((M, N), device), max(N, 1)
    ws, ws_ptr, ws_bytes = None, None, 0
    if isinstance(workspace, _torch().Tensor):
        ws_ptr, ws_bytes = _supplied(workspace, device)
    elif workspace and M and N and K:
        ws_bytes = sgemm_f32_workspace_size(tx, ty, M, N, K, ldx, ldy, ldo)
        ws, ws_ptr = _scratch(ws_bytes, device)
    where = "sgemm_f32_ex" if epilogue is None else "sgemm_f32_epilogue"
    args = (tx, ty, M, N, K, float(alpha), X.data_ptr(), ldx, 0, Y.data_ptr(), ldy, 0)
    to = (out.data_ptr(), ldo, 0, 1)
    if epilogue is None:
        code = load().sgemm_f32_ex(*args, 0.0, *to, ws_ptr, ws_bytes, _handle(device), None)
    else:
        code = load().sgemm_f32_epilogue(*args, *to, ctypes.byref(epilogue), ws_ptr, ws_bytes, _handle(device), None)
    del ws
    _check(code, where)
    return out


def _norm_inputs(x, weight, residual, sum_out, device):
    """(rows, D, ldx, weight address, residual address, ldr, S or None, its
    address, lds, what the caller gets as s)."""
    rows, D, ldx = _rows(x, "x")
    if D < 1:
        raise ValueError("rows need at least one value")
    w = _vector(weight, D, device, "weight") if weight is not None else None
    r, ldr = None, 0
    if residual is not None:
        ldr, r = _matrix(residual, rows, D, device, "residual"), residual.data_ptr()
    if sum_out is not None:
        lds = _matrix(sum_out, rows, D, device, "sum_out")
    elif residual is not None:
        sum_out, lds = _empty((rows, D), device), D
    else:
        return rows, D, ldx, w, r, ldr, None, 0, x
    return rows, D, ldx, w, r, ldr, sum_out.data_ptr(), lds, sum_out


def rmsnorm(x, weight=None, *, eps=1e-6, residual=None, sum_out=None, out=None, stream=None):
    """(y, s): s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, per row.

    Without `residual`, s is x itself (and lost where `out` is x).  `sum_out` receives s (it may be `x` or
    `residual`, which then holds the residual stream updated in place).
    """
    device = _gpu_of(x, "x")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return rmsnorm(x, weight, eps=eps, residual=residual, sum_out=sum_out, out=out)
    rows, D, ldx, w, r, ldr, s_ptr, lds, s = _norm_inputs(x, weight, residual, sum_out, device)
    if out is None:
        out, ldy = _empty((rows, D), device), D
    else:
        ldy = _matrix(out, rows, D, device, "out")
    _check(load().sgemm_rmsnorm_f32(rows, D, x.data_ptr(), ldx, r, ldr, w, float(eps), s_ptr, lds, out.data_ptr(),
                                    ldy, _handle(device)), "sgemm_rmsnorm_f32")
    return out, s


def rmsnorm_e4m3(x, weight=None, *, eps=1e-6, residual=None, sum_out=None, stream=None):
    """(q, scale, s): rmsnorm() with y in 8 bits, q * scale[:, None] standing
    for y; gemm_e4m3() takes q and scale as they are."""
    device = _gpu_of(x, "x")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return rmsnorm_e4m3(x, weight, eps=eps, residual=residual, sum_out=sum_out)
    rows, D, ldx, w, r, ldr, s_ptr, lds, s = _norm_inputs(x, weight, residual, sum_out, device)
    (q, ldq), scale = _empty_codes(rows, D, device), _empty((rows,), device)
    _check(load().sgemm_rmsnorm_e4m3(rows, D, x.data_ptr(), ldx, r, ldr, w, float(eps), s_ptr, lds, q.data_ptr(),
                                     ldq, scale.data_ptr(), _handle(device)), "sgemm_rmsnorm_e4m3")
    return q, scale, s


def quantize_e4m3(x, *, stream=None):
    """(q, scale): the rows of x in 8 bits (e4m3) with one scale a row."""
    device = _gpu_of(x, "x")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return quantize_e4m3(x)
    rows, D, ldx = _rows(x, "x")
    if D < 1:
        raise ValueError("rows need at least one value")
    (q, ldq), scale = _empty_codes(rows, D, device), _empty((rows,), device)
    _check(load().sgemm_quantize_e4m3(rows, D, x.data_ptr(), ldx, q.data_ptr(), ldq, scale.data_ptr(),
                                      _handle(device)), "sgemm_quantize_e4m3")
    return q, scale


def rmsnorm_backward(grad, s, weight=None, *, eps=1e-6, dsum=None, out=None, need_weight=True, stream=None):
    """(dx, dweight) from rmsnorm()'s y's gradient; `s` is the sum it returned.

    dx is the gradient of x and of the residual.  `dsum`, the gradient that
    reaches s past the norm (down the residual stream), is added to it; `out`
    may be `dsum`.  dweight is None without `weight` or with need_weight false.
    """
    device = _gpu_of(grad, "grad")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return rmsnorm_backward(grad, s, weight, eps=eps, dsum=dsum, out=out, need_weight=need_weight)
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
    dw, ws, ws_ptr, nbytes = None, None, None, ctypes.c_size_t(0)
    if weight is not None and need_weight:
        dw = _empty((D,), device)
        _check(load().sgemm_rmsnorm_f32_grad_workspace(rows, D, ctypes.byref(nbytes)),
               "sgemm_rmsnorm_f32_grad_workspace")
        ws, ws_ptr = _scratch(nbytes.value, device)
    code = load().sgemm_rmsnorm_f32_grad(
        rows, D, grad.data_ptr(), ldy, s.data_ptr(), lds, w, float(eps), g, ldds, out.data_ptr(), lddx,
        dw.data_ptr() if dw is not None else None, ws_ptr, nbytes.value, _handle(device))
    del ws
    _check(code, "sgemm_rmsnorm_f32_grad")
    return out, dw


def gemm_e4m3(A, scale_a, B, scale_b, *, bias=None, activation=None, residual=None, pre=None, grad_pre=None,
              out=None, workspace=True, stream=None):
    """act((scale_a[:, None] * A) @ (scale_b[:, None] * B).T + bias) + residual
    for 8-bit A (M x K) and B (N x K, one row per output), in float32.

    Scales are M and N float32 factors, or None for ones.  Other arguments as
    sgemm_epilogue().
    """
    torch = _torch()
    device = _gpu_of(A, "A")
    elsewhere = _elsewhere(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemm_e4m3(A, scale_a, B, scale_b, bias=bias, activation=activation, residual=residual, pre=pre,
                             grad_pre=grad_pre, out=out, workspace=workspace)
    _same_gpu(device, B, "B")
    M, K, lda = _rows(A, "A", torch.float8_e4m3fn)
    N, K2, ldb = _rows(B, "B", torch.float8_e4m3fn)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    sa = _vector(scale_a, M, device, "scale_a") if scale_a is not None else None
    sb = _vector(scale_b, N, device, "scale_b") if scale_b is not None else None
    if out is None:
        out, ldc = _empty((M, N), device), max(N, 1)
    else:
        ldc = _matrix(out, M, N, device, "out")
    e = _epilogue(device, 1, M, N, bias, activation, pre, grad_pre, residual)
    ws, ws_ptr, ws_bytes = None, None, 0
    if isinstance(workspace, torch.Tensor):
        ws_ptr, ws_bytes = _supplied(workspace, device)
    elif workspace:
        nbytes = ctypes.c_size_t(0)
        _check(load().sgemm_e4m3_workspace_size(M, N, K, ctypes.byref(nbytes)), "sgemm_e4m3_workspace_size")
        ws_bytes = nbytes.value
        ws, ws_ptr = _scratch(ws_bytes, device)
    code = load().sgemm_e4m3(M, N, K, A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, out.data_ptr(), ldc,
                             ctypes.byref(e), ws_ptr, ws_bytes, _handle(device))
    del ws
    _check(code, "sgemm_e4m3")
    return out
