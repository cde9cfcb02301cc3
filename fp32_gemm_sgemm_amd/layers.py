"""What a model's layer needs next to its products, for torch tensors: the C
ABI of include/sgemm_layers.h, argument marshalling only (the work is the
library's HIP kernels, and nothing falls back to another implementation).

Conventions are those of ops.py: 2-D float32 device tensors with unit column
stride and any row stride, 8-bit matrices as torch.float8_e4m3fn, one GPU a
call (not necessarily the current one), work enqueued on `stream` or on torch's
current one, no synchronisation.
"""
import ctypes

from .binding import SgemmTensor, _check, load
from .ops import (_MAX_DIM, _elsewhere, _empty, _empty_codes, _gpu_of, _handle, _matrix, _norm_inputs, _rows,
                  _same_gpu, _scratch, _torch, _vector)


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
    ws, ws_ptr, nbytes = None, None, ctypes.c_size_t(0)
    if dw is not None or db is not None:
        _check(load().sgemm_layernorm_f32_grad_workspace(rows, D, ctypes.byref(nbytes)),
               "sgemm_layernorm_f32_grad_workspace")
        ws, ws_ptr = _scratch(nbytes.value, device)
    code = load().sgemm_layernorm_f32_grad(
        rows, D, grad.data_ptr(), ldy, s.data_ptr(), lds, w, float(eps), g, ldds, out.data_ptr(), lddx,
        dw.data_ptr() if dw is not None else None, db.data_ptr() if db is not None else None, ws_ptr, nbytes.value,
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
    flat = []
    for i, x in enumerate(tensors):
        rows, cols, ldx = _plane(x, "a tensor")
        _same_gpu(device, x, "a tensor")
        ptr = x.data_ptr()
        y, ldy = ptr, ldx
        if out is not None:
            to = out[i]
            if to.shape != x.shape:
                raise ValueError(f"out must have the tensors' shapes: {tuple(to.shape)} for {tuple(x.shape)}")
            _same_gpu(device, to, "out")
            y = to.data_ptr()
            orows, ocols, ldy = _plane(to, "out")
            if (orows, ocols) != (rows, cols):
                # one of the two is a run and the other has gaps between its rows
                rows, cols = x.shape
                ldx, ldy = ldx or cols, ldy or cols
        flat += (ptr, y, rows, cols, ldx, ldy)
    return (SgemmTensor * len(tensors)).from_buffer((ctypes.c_longlong * max(len(flat), 1))(*flat)) if flat else None


def _many(tensors, out, device, call):
    """Runs call(count, array, norm address, workspace address, bytes); the norm
    as a tensor without dimensions."""
    torch = _torch()
    array = _tensor_list(tensors, out, device)
    nbytes = ctypes.c_size_t(0)
    _check(load().sgemm_clip_f32_workspace(len(tensors), ctypes.byref(nbytes)), "sgemm_clip_f32_workspace")
    ws, ws_ptr = _scratch(nbytes.value, device)
    norm = torch.empty((), dtype=torch.float32, device=device)
    call(len(tensors), array, norm.data_ptr(), ws_ptr, nbytes.value)
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
    shapes, receives the scaled ones and they are left as they are.  Nothing
    waits for the GPU, so a norm that is not finite is the caller's to look at.
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
