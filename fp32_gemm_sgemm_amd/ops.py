"""The operators around a matrix product for torch tensors: the C ABI of
include/sgemm_ops.h, argument marshalling only (the work is the library's HIP
kernels, and nothing falls back to another implementation).

Matrices are 2-D (a product's may be 3-D batches) float32 device tensors with
unit column stride and any row stride; 8-bit matrices are torch.float8_e4m3fn.
All tensors of a call are on one GPU, which need not be the current one.  Work
is enqueued on `stream` (default: torch's current stream of that GPU) and
nothing synchronises.  A tensor that a call allocates is tied to that stream,
and so may be used on it at once.
"""
import ctypes

from .binding import (ACTIVATIONS, SgemmEpilogue, _check, _row_major_view, _stream_handle, _workspace,
                      load, sgemm, sgemm_f32_cfg_geometry, sgemm_f32_workspace_size)

E4M3_MAX = 448.0


def _activation(name):
    if name is None:
        return 0
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _on_gpu(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _gpu_of(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _vector(t, n, name):
    import torch
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _matrix(t, shape, name):
    """Row stride of a 2-D float32 tensor of the given shape."""
    rows, cols, ld = _row_major_view(t, name)
    if (rows, cols) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {(rows, cols)}")
    return ld


def _codes(t, name):
    """(rows, cols, row stride) of an 8-bit matrix."""
    import torch
    if t.dtype != torch.float8_e4m3fn:
        raise TypeError(f"{name} must be float8_e4m3fn, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return rows, cols, max(t.stride(0) if rows > 1 else cols, cols, 1)


class _Call:
    """The GPU and stream of one call, as a context with that GPU current.
    new() allocates the call's outputs: on torch's current stream, as torch
    does, and recorded on the call's own where that is another."""

    def __init__(self, device, stream):
        import torch
        self.device, self._stream = device, stream
        self._guard = torch.cuda.device(device)

    def __enter__(self):
        import torch
        self._guard.__enter__()
        self.stream, self.handle = _stream_handle(self._stream, self.device)
        self._other = self._stream is not None and hasattr(self.stream, "cuda_stream") and \
            self.stream != torch.cuda.current_stream(self.device)
        return self

    def __exit__(self, *exc):
        return self._guard.__exit__(*exc)

    def new(self, shape, dtype=None):
        import torch
        t = torch.empty(shape, dtype=dtype or torch.float32, device=self.device)
        if self._other:
            t.record_stream(self.stream)
        return t

    def new_codes(self, rows, cols):
        """8-bit rows that start 16-byte aligned, as the product reads fastest."""
        import torch
        return self.new((rows, -(-cols // 16) * 16), torch.float8_e4m3fn)[:, :cols]

    def workspace(self, nbytes):
        return _workspace(nbytes, self.device, self.stream)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _supplied(workspace, device):
    """(address, bytes) of a caller's workspace tensor."""
    if not workspace.is_cuda or workspace.device != device:
        raise ValueError("workspace must be a device tensor on the operands' GPU")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _batch_view(t, name):
    """(batch, rows, cols, row stride, batch stride) of a 2-D or 3-D float32 tensor."""
    if t.dim() == 2:
        return (1, *_row_major_view(t, name), 0)
    if t.dim() != 3:
        raise ValueError(f"{name} must be 2-D or 3-D")
    rows, cols, ld = _row_major_view(t[0] if t.shape[0] > 0 else t.new_empty(t.shape[1:]), name)
    return t.shape[0], rows, cols, ld, (t.stride(0) if t.shape[0] > 1 else 0)


def _epilogue(batch, M, N, bias, activation, pre, grad_pre, residual):
    """SgemmEpilogue of tensors that match a batch x M x N output (2-D ones are
    shared by the batch, but for `pre`)."""
    e = SgemmEpilogue(activation=_activation(activation))
    if bias is not None:
        if bias.dim() == 2 and bias.shape[0] == batch:
            e.stride_bias = bias.stride(0) if batch > 1 else 0
            e.bias = bias.data_ptr()
            if batch > 0:
                _vector(bias[0], N, "bias")
        else:
            e.bias = _vector(bias, N, "bias")
    for name, t in (("pre", pre), ("grad_pre", grad_pre), ("residual", residual)):
        if t is None:
            continue
        b, rows, cols, ld, stride = _batch_view(t, name)
        if (rows, cols) != (M, N) or (b != batch and (b != 1 or name == "pre")):
            raise ValueError(f"{name} must have shape {(M, N)}, got {tuple(t.shape)}")
        setattr(e, name, t.data_ptr())
        setattr(e, f"ld_{name}", ld)
        setattr(e, f"stride_{name}", stride)
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
    import torch
    device = _gpu_of(A, "A")
    _on_gpu(device, B=B, bias=bias, residual=residual, out=out, pre=pre, grad_pre=grad_pre)
    batched = A.dim() == 3 or B.dim() == 3
    ba, ra, ca, lda, sa = _batch_view(A, "A")
    bb, rb, cb, ldb, sb = _batch_view(B, "B")
    M, K = (ca, ra) if transa else (ra, ca)
    K2, N = (cb, rb) if transb else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    batch = bb if ba == 1 else ba
    if ba not in (1, batch) or bb not in (1, batch):
        raise ValueError("batch sizes differ")
    ta, tb = int(bool(transa)), int(bool(transb))
    if pre is not None and grad_pre is not None:
        raise ValueError("pre and grad_pre exclude each other")
    with _Call(device, stream) as call:
        if out is None:
            out = call.new((batch, M, N) if batched else (M, N))
        bo, Mo, No, ldc, sc = _batch_view(out, "out")
        if (bo, Mo, No) != (batch, M, N) or (out.dim() == 3) != batched:
            raise ValueError("out has the wrong shape")
        e = _epilogue(batch, M, N, bias, activation, pre, grad_pre, residual)
        ws, ws_ptr, ws_bytes = None, 0, 0
        if isinstance(workspace, torch.Tensor):
            ws_ptr, ws_bytes = _supplied(workspace, device)
        elif workspace and M and N and K and batch:
            if cfg is None:
                ws_bytes = sgemm_f32_workspace_size(ta, tb, M, N, K, lda, ldb, ldc, batch)
            elif cfg.splits > 1:
                ws_bytes = sgemm_f32_cfg_geometry(cfg, ta, tb, M, N, K, lda, ldb, ldc, batch).workspace_bytes
            ws = call.workspace(ws_bytes)
            ws_ptr = _ptr(ws)
        code = load().sgemm_f32_epilogue(
            ta, tb, M, N, K, float(alpha), A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, out.data_ptr(), ldc, sc,
            batch, ctypes.byref(e), ws_ptr, ws_bytes, call.handle,
            ctypes.byref(cfg) if cfg is not None else None)
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
    M, N, ldy = _row_major_view(grad, "grad")
    act = _activation(activation)
    ldz = 0
    if act:
        if pre is None:
            raise ValueError("an activation's gradient needs `pre`")
        ldz = _matrix(pre, (M, N), "pre")
        _on_gpu(device, pre=pre)
    with _Call(device, stream) as call:
        if out is None:
            out = call.new((M, N))
        if dbias is None:
            dbias = call.new((N,))
        out = None if out is False else out
        dbias = None if dbias is False else dbias
        _on_gpu(device, out=out, dbias=dbias)
        ldo = _matrix(out, (M, N), "out") if out is not None else 0
        if dbias is not None:
            _vector(dbias, N, "dbias")
        nbytes = ctypes.c_size_t(0)
        if dbias is not None:
            _check(load().sgemm_f32_activation_grad_workspace(M, N, ctypes.byref(nbytes)),
                   "sgemm_f32_activation_grad_workspace")
        ws = call.workspace(nbytes.value)
        code = load().sgemm_f32_activation_grad(
            M, N, act, grad.data_ptr(), ldy, _ptr(pre) if act else None, ldz, _ptr(out), ldo, _ptr(dbias),
            _ptr(ws), nbytes.value if ws is not None else 0, call.handle)
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
    doing the multiplication.
    """
    device = _gpu_of(grad, "grad")
    _on_gpu(device, A=A, B=B, pre=pre, a_pre=a_pre)
    ra, ca, _ = _row_major_view(A, "A")
    rb, cb, _ = _row_major_view(B, "B")
    M, K = (ca, ra) if transa else (ra, ca)
    K2, N = (cb, rb) if transb else (rb, cb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    _matrix(grad, (M, N), "grad")
    act, a_act = _activation(activation), _activation(a_activation)
    if a_act and a_pre is None:
        raise ValueError("a_activation needs `a_pre`")
    if a_pre is not None and tuple(a_pre.shape) != tuple(A.shape):
        raise ValueError("a_pre must have A's shape")
    dz, dbias, dA, dB = grad, None, None, None
    need_products = "A" in need or "B" in need
    if "bias" in need or (act and need_products):
        dz, dbias = activation_grad(grad, pre, activation, out=None if act and need_products else False,
                                    dbias=None if "bias" in need else False, stream=stream)
        dz = grad if dz is None else dz
    kw = {"alpha": alpha, "workspace": workspace, "stream": stream}
    if "A" in need:
        left = (B, dz, transb, True) if transa else (dz, B, False, not transb)
        if a_act:
            dA = sgemm_epilogue(left[0], left[1], transa=left[2], transb=left[3], activation=a_activation,
                                grad_pre=a_pre, **kw)
        else:
            dA = _product(*left, device, **kw)
    if "B" in need:
        dB = _product(*((dz, A, True, transa) if transb else (A, dz, not transa, False)), device, **kw)
    return dA, dB, dbias


def _product(X, Y, tx, ty, device, alpha, workspace, stream):
    """sgemm() with its output tied to the stream it runs on."""
    with _Call(device, stream) as call:
        out = call.new((X.shape[1] if tx else X.shape[0], Y.shape[0] if ty else Y.shape[1]))
    return sgemm(X, Y, out=out, transa=tx, transb=ty, alpha=alpha, workspace=workspace, stream=stream)


def _norm_inputs(x, weight, residual, sum_out):
    device = _gpu_of(x, "x")
    rows, D, ldx = _row_major_view(x, "x")
    if D < 1:
        raise ValueError("rows need at least one value")
    _on_gpu(device, weight=weight, residual=residual, sum_out=sum_out)
    if weight is not None:
        _vector(weight, D, "weight")
    ldr = _matrix(residual, (rows, D), "residual") if residual is not None else 0
    return device, rows, D, ldx, ldr


def _sum_tensor(call, x, residual, sum_out):
    """(tensor for S or None, what the caller gets as S)."""
    if residual is None and sum_out is None:
        return None, x
    s = call.new(tuple(x.shape)) if sum_out is None else sum_out
    return s, s


def rmsnorm(x, weight=None, *, eps=1e-6, residual=None, sum_out=None, out=None, stream=None):
    """(y, s): s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, per row.

    Without `residual`, s is x itself.  `sum_out` receives s (it may be `x` or
    `residual`, which then holds the residual stream updated in place).
    """
    device, rows, D, ldx, ldr = _norm_inputs(x, weight, residual, sum_out)
    with _Call(device, stream) as call:
        _on_gpu(device, out=out)
        y = call.new((rows, D)) if out is None else out
        ldy = _matrix(y, (rows, D), "out")
        s, s_result = _sum_tensor(call, x, residual, sum_out)
        lds = _matrix(s, (rows, D), "sum_out") if s is not None else 0
        code = load().sgemm_rmsnorm_f32(rows, D, x.data_ptr(), ldx, _ptr(residual), ldr, _ptr(weight), float(eps),
                                        _ptr(s), lds, y.data_ptr(), ldy, call.handle)
    _check(code, "sgemm_rmsnorm_f32")
    return y, s_result


def rmsnorm_e4m3(x, weight=None, *, eps=1e-6, residual=None, sum_out=None, stream=None):
    """(q, scale, s): rmsnorm() with y in 8 bits, q * scale[:, None] standing
    for y; gemm_e4m3() takes q and scale as they are."""
    import torch
    device, rows, D, ldx, ldr = _norm_inputs(x, weight, residual, sum_out)
    with _Call(device, stream) as call:
        q, scale = call.new_codes(rows, D), call.new((rows,))
        s, s_result = _sum_tensor(call, x, residual, sum_out)
        lds = _matrix(s, (rows, D), "sum_out") if s is not None else 0
        code = load().sgemm_rmsnorm_e4m3(rows, D, x.data_ptr(), ldx, _ptr(residual), ldr, _ptr(weight), float(eps),
                                         _ptr(s), lds, q.data_ptr(), -(-D // 16) * 16, scale.data_ptr(),
                                         call.handle)
    _check(code, "sgemm_rmsnorm_e4m3")
    return q, scale, s_result


def quantize_e4m3(x, *, stream=None):
    """(q, scale): the rows of x in 8 bits (e4m3) with one scale a row."""
    device = _gpu_of(x, "x")
    rows, D, ldx = _row_major_view(x, "x")
    if D < 1:
        raise ValueError("rows need at least one value")
    with _Call(device, stream) as call:
        q, scale = call.new_codes(rows, D), call.new((rows,))
        code = load().sgemm_quantize_e4m3(rows, D, x.data_ptr(), ldx, q.data_ptr(), -(-D // 16) * 16,
                                          scale.data_ptr(), call.handle)
    _check(code, "sgemm_quantize_e4m3")
    return q, scale


def rmsnorm_backward(grad, s, weight=None, *, eps=1e-6, dsum=None, out=None, need_weight=True, stream=None):
    """(dx, dweight) from rmsnorm()'s y's gradient; `s` is the sum it returned.

    dx is the gradient of x and of the residual.  `dsum`, the gradient that
    reaches s past the norm (down the residual stream), is added to it; `out`
    may be `dsum`.  dweight is None without `weight` or with need_weight false.
    """
    device = _gpu_of(grad, "grad")
    rows, D, ldy = _row_major_view(grad, "grad")
    if D < 1:
        raise ValueError("rows need at least one value")
    _on_gpu(device, s=s, weight=weight, dsum=dsum, out=out)
    lds = _matrix(s, (rows, D), "s")
    ldds = _matrix(dsum, (rows, D), "dsum") if dsum is not None else 0
    if weight is not None:
        _vector(weight, D, "weight")
    with _Call(device, stream) as call:
        dx = call.new((rows, D)) if out is None else out
        lddx = _matrix(dx, (rows, D), "out")
        dw = call.new((D,)) if weight is not None and need_weight else None
        nbytes = ctypes.c_size_t(0)
        if dw is not None:
            _check(load().sgemm_rmsnorm_f32_grad_workspace(rows, D, ctypes.byref(nbytes)),
                   "sgemm_rmsnorm_f32_grad_workspace")
        ws = call.workspace(nbytes.value)
        code = load().sgemm_rmsnorm_f32_grad(
            rows, D, grad.data_ptr(), ldy, s.data_ptr(), lds, _ptr(weight), float(eps), _ptr(dsum), ldds,
            dx.data_ptr(), lddx, _ptr(dw), _ptr(ws), nbytes.value if ws is not None else 0, call.handle)
    del ws
    _check(code, "sgemm_rmsnorm_f32_grad")
    return dx, dw


def gemm_e4m3(A, scale_a, B, scale_b, *, bias=None, activation=None, residual=None, pre=None, grad_pre=None,
              out=None, workspace=True, stream=None):
    """act((scale_a[:, None] * A) @ (scale_b[:, None] * B).T + bias) + residual
    for 8-bit A (M x K) and B (N x K, one row per output), in float32.

    Scales are M and N float32 factors, or None for ones.  Other arguments as
    sgemm_epilogue().
    """
    import torch
    device = _gpu_of(A, "A")
    _on_gpu(device, B=B, scale_a=scale_a, scale_b=scale_b, bias=bias, residual=residual, pre=pre,
            grad_pre=grad_pre, out=out)
    M, K, lda = _codes(A, "A")
    N, K2, ldb = _codes(B, "B")
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    sa = _vector(scale_a, M, "scale_a") if scale_a is not None else None
    sb = _vector(scale_b, N, "scale_b") if scale_b is not None else None
    if pre is not None and grad_pre is not None:
        raise ValueError("pre and grad_pre exclude each other")
    with _Call(device, stream) as call:
        if out is None:
            out = call.new((M, N))
        ldc = _matrix(out, (M, N), "out")
        e = _epilogue(1, M, N, bias, activation, pre, grad_pre, residual)
        ws, ws_ptr, ws_bytes = None, 0, 0
        if isinstance(workspace, torch.Tensor):
            ws_ptr, ws_bytes = _supplied(workspace, device)
        elif workspace:
            nbytes = ctypes.c_size_t(0)
            _check(load().sgemm_e4m3_workspace_size(M, N, K, ctypes.byref(nbytes)), "sgemm_e4m3_workspace_size")
            ws_bytes = nbytes.value
            ws = call.workspace(ws_bytes)
            ws_ptr = _ptr(ws)
        code = load().sgemm_e4m3(M, N, K, A.data_ptr(), lda, sa, B.data_ptr(), ldb, sb, out.data_ptr(), ldc,
                                 ctypes.byref(e), ws_ptr, ws_bytes, call.handle)
    del ws
    _check(code, "sgemm_e4m3")
    return out
