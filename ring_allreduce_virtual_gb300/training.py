"""The operators of a data-parallel training step around the AllReduce, on
torch tensors: layer norm (forward, backward, and as a differentiable call), the
norm of a list of gradients, and clipping by it. Everything is computed by the
kernels of libvr.so (include/vr.h states the formulas and the rules); this
module checks the tensors, allocates outputs and workspaces, and passes
addresses. There is no CPU fallback.

    from ring_allreduce_virtual_gb300 import training
    y = training.layer_norm(x, weight, bias)            # differentiable
    ...                                                 # backward, all_reduce of the gradients
    grads = training.TensorList([p.grad for p in params])
    norm = training.clip_grad_norm(grads, 1.0, scale=1 / n_ranks)   # in place

Calls are asynchronous on the current torch stream of the tensors' device (which
need not be the current device), or on `stream` of that device; outputs and
workspaces are allocated there, so that they may be freed at any time. As with
any torch operation, tensors that were made or are freed on another stream
need the caller's own ordering (wait_stream, record_stream). Tensors that are
given to be written (out, dx, dweight, dbias, outs, gradients clipped in place)
count as changed in place: autograd refuses a backward pass that saved them.
"""
import functools

import torch
from torch.autograd.graph import increment_version as _written

import ring_allreduce_virtual_gb300 as vr

_CODE = {torch.float16: vr.DTYPES["float16"], torch.bfloat16: vr.DTYPES["bfloat16"],
         torch.float32: vr.DTYPES["float32"], torch.float64: vr.DTYPES["float64"]}
_NORM_CODE = {t: _CODE[t] for t in (torch.float16, torch.bfloat16, torch.float32)}
_F32 = torch.float32

# The current stream's handle. torch's own getter of the raw handle takes 0.1 us, a
# Stream object 2 us, a tenth of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


# The library launches on the device that is current. Where that is not the tensors',
# a call makes it so for its duration.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_device(index, f, *args):
    with torch.cuda.device(index):
        return f(*args)


def _on(stream, index, f, *args):
    """f(*args) on `stream` of the tensors' device: allocations go to that
    stream's pool too."""
    if stream.device_index != index:
        raise ValueError("the stream is not on the tensors' device")
    with torch.cuda.stream(stream):
        return f(*args)


# ------------------------------------------------------------ layer norm
def _rows(t, what):
    """(rows, row stride) of a tensor seen as a matrix of its last axis. The
    last axis has to be dense and the leading ones one row stride apart."""
    cols = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // cols, cols
    rows, stride = 1, None
    if cols != 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the last axis must be dense")
    for size, step in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = step
        elif step != stride * rows:
            raise ValueError(f"{what}: the leading axes must be one row stride apart")
        rows *= size
    stride = cols if stride is None else stride
    if rows and stride < cols:
        raise ValueError(f"{what}: rows overlap")
    return rows, stride


def _has_rows(t):
    """Whether _rows takes t as it is."""
    if t.is_contiguous():
        return True
    try:
        _rows(t, "t")
    except ValueError:
        return False
    return True


def _bad_x(x):
    if x.dtype not in _NORM_CODE:
        raise ValueError(f"unsupported dtype {x.dtype}")
    raise ValueError("x must be a CUDA tensor with a last axis of at least one element")


def _check_x(x):
    """(columns, type code, device index)"""
    code = _NORM_CODE.get(x.dtype)
    if code is None or not x.is_cuda or not x.dim() or not x.shape[-1]:
        _bad_x(x)
    return x.shape[-1], code, x.get_device()


def _check_param(p, x, cols, device, other=None):
    """A weight or bias: a dense vector of x's columns, of x's type or float32,
    and of `other`'s."""
    if p.get_device() != device or p.dim() != 1 or p.shape[0] != cols or not p.is_contiguous():
        raise ValueError("weight and bias must be dense vectors of x's last axis, on its device")
    t = p.dtype
    if (t != _F32 and t != x.dtype) or (other is not None and other.dtype != t):
        raise ValueError("weight and bias must have one type: x's or float32")


def _check_like(t, x, device, what):
    if t.get_device() != device or t.dtype != x.dtype or t.shape != x.shape:
        raise ValueError(f"{what} must have x's shape, type and device")


def _dense_like(x):
    return torch.empty_like(x) if x.is_contiguous() else \
        torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, stats=True, out=None, stream=None):
    """(y, mean, rstd): layer norm over x's last axis; mean and rstd (float32,
    x's leading shape) are what the backward pass needs, None with
    stats=False. `out`: a tensor of x's shape and type for y, x itself allowed.
    Tensors of x's shape, here and in the backward pass, have a dense last axis
    and leading axes that are one row stride apart."""
    if stream is not None:
        return _on(stream, x.get_device(), layer_norm_forward, x, weight, bias, eps, stats, out)
    cols, code, device = _check_x(x)
    if device != _current_device():
        return _on_device(device, layer_norm_forward, x, weight, bias, eps, stats, out)
    wcode = code
    if weight is not None:
        _check_param(weight, x, cols, device)
        wcode = _NORM_CODE[weight.dtype]
    if bias is not None:
        _check_param(bias, x, cols, device, weight)
        wcode = _NORM_CODE[bias.dtype]
    rows, xs = _rows(x, "x")
    if out is None:
        y, ys = _dense_like(x), cols
    else:
        _check_like(out, x, device, "out")
        y, ys = out, _rows(out, "out")[1]
    mean = rstd = None
    if stats:
        mean = torch.empty(x.shape[:-1], dtype=_F32, device=x.device)
        rstd = torch.empty_like(mean)
    rc = vr.lib().vrLayerNormForward(x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(),
                                     _ptr(mean), _ptr(rstd), rows, cols, xs, ys, eps, code, wcode,
                                     _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrLayerNormForward")
    if out is not None:
        _written(out)
    return y, mean, rstd


@functools.lru_cache(maxsize=256)
def _backward_workspace(rows, cols, code):
    return vr.vrLayerNormBackwardWorkspace(rows, cols, code)


def layer_norm_backward(dy, x, mean, rstd, weight=None, dx=True, dweight=True, dbias=True,
                        stream=None):
    """(dx, dweight, dbias) of layer_norm_forward. dx, dweight and dbias may
    each be False (not wanted, None is returned) or a tensor to write to, such as
    a view of the flat bucket that the AllReduce takes. The parameters'
    gradients have the weight's type (x's without a weight, or the given
    tensors')."""
    if stream is not None:
        return _on(stream, x.get_device(), layer_norm_backward, dy, x, mean, rstd, weight, dx,
                   dweight, dbias)
    cols, code, device = _check_x(x)
    if device != _current_device():
        return _on_device(device, layer_norm_backward, dy, x, mean, rstd, weight, dx, dweight,
                          dbias)
    given = [t for t in (dx, dweight, dbias) if isinstance(t, torch.Tensor)]
    rows, xs = _rows(x, "x")
    _check_like(dy, x, device, "dy")
    dys = _rows(dy, "dy")[1]
    for t in (mean, rstd):
        if t.dtype != _F32 or t.get_device() != device or t.numel() != rows or \
                not t.is_contiguous():
            raise ValueError("mean and rstd must be the forward pass's")
    wt = weight
    if weight is not None:
        _check_param(weight, x, cols, device)
    grads = [dweight, dbias]
    for i, t in enumerate(grads):
        if isinstance(t, torch.Tensor):
            _check_param(t, x, cols, device, wt)
            wt = t
        elif not t:
            grads[i] = None
    wt = x.dtype if wt is None else wt.dtype
    dxs = cols
    if dx is True:
        dx = _dense_like(x)
    elif isinstance(dx, torch.Tensor):
        _check_like(dx, x, device, "dx")
        dxs = _rows(dx, "dx")[1]
    else:
        dx = None
    ws, nbytes = None, 0
    if grads[0] is not None or grads[1] is not None:
        nbytes = _backward_workspace(rows, cols, code)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        for i in (0, 1):
            if grads[i] is True:
                grads[i] = torch.empty_like(weight) if weight is not None else \
                    torch.empty(cols, dtype=wt, device=x.device)
    elif dx is None:
        return None, None, None
    dw, db = grads
    rc = vr.lib().vrLayerNormBackward(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(),
                                      rstd.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db), rows, cols,
                                      dys, xs, dxs, code, _NORM_CODE[wt], _ptr(ws), nbytes,
                                      _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrLayerNormBackward")
    if given:
        _written(given)
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        if x.dim() and x.shape[-1] and not _has_rows(x):
            x = x.contiguous()
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps, any(ctx.needs_input_grad))
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.bias_type = None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        db = need[2]
        if db and weight is None:  # the bias alone says the gradient's type
            db = torch.empty(x.shape[-1], dtype=ctx.bias_type, device=x.device)
        dx, dw, db = layer_norm_backward(dy.contiguous(), x, mean, rstd, weight, need[0],
                                         need[1] and weight is not None, db)
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over x's last axis, differentiable once with respect to x,
    weight and bias. An x whose last axis is not dense, or whose leading axes are
    not one row stride apart (x[:, 1:] of three axes, an expanded one), is copied
    first."""
    return _LayerNorm.apply(x, weight, bias, eps)


# ------------------------------------------------- gradient norm, clipping
class TensorList:
    """A list of gradients (or outputs) whose addresses have been checked and
    marshalled once, about 0.75 us a tensor; it keeps the tensors alive. Make it
    for buffers that stay where they are from step to step. It does not follow
    tensors that are replaced or moved: after zero_grad(set_to_none=True), which
    gives every parameter a new gradient, it still names the old ones, and a
    tensor given other memory (.data, resize_, set_) needs a new list. A plain
    sequence of tensors works wherever a TensorList does and is marshalled for
    the call."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        if not self.tensors:
            raise ValueError("an empty list of tensors")
        self.device = self.tensors[0].device
        for t in self.tensors:
            if not t.is_cuda or t.device != self.device or not t.is_contiguous():
                raise ValueError("tensors must be contiguous CUDA tensors of one device")
            if t.dtype not in _CODE:
                raise ValueError(f"unsupported dtype {t.dtype}")
        self.arrays = vr.tensor_arrays([t.data_ptr() for t in self.tensors],
                                       [t.numel() for t in self.tensors],
                                       [_CODE[t.dtype] for t in self.tensors])
        self.workspace_bytes = vr.vrGradNormWorkspace(len(self.tensors))
        self.index = self.tensors[0].get_device()
        self.shape = bytes(self.arrays[1]) + bytes(self.arrays[2])  # counts and types

    def __len__(self):
        return len(self.tensors)

    @functools.cached_property
    def bases(self):
        """What the tensors are views of, each once: views share its version."""
        each = (t if t._base is None else t._base for t in self.tensors)
        return list({id(t): t for t in each}.values())


def _list(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def grad_norm(grads, scale=1.0, per_tensor=False, stream=None):
    """The 2-norm of all elements of `grads` (a TensorList or a sequence of
    tensors) times |scale|, a float32 scalar tensor; with per_tensor also the
    norms of the single tensors, a float32 vector."""
    grads = _list(grads)
    if stream is not None:
        return _on(stream, grads.index, grad_norm, grads, scale, per_tensor)
    if grads.index != _current_device():
        return _on_device(grads.index, grad_norm, grads, scale, per_tensor)
    device, nbytes = grads.device, grads.workspace_bytes
    norm = torch.empty((), dtype=_F32, device=device)
    norms = torch.empty(len(grads), dtype=_F32, device=device) if per_tensor else None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ptrs, counts, types = grads.arrays
    rc = vr.lib().vrGradNorm(ptrs, counts, types, len(ptrs), scale, norm.data_ptr(), _ptr(norms),
                             ws.data_ptr(), nbytes, _raw_stream(grads.index))
    if rc:
        raise vr.VrError(rc, "vrGradNorm")
    return (norm, norms) if per_tensor else norm


def clip_grad_norm(grads, max_norm, scale=1.0, outs=None, stream=None):
    """Multiply `grads` (a TensorList or a sequence of tensors) by `scale` and,
    where the norm of the result exceeds max_norm, by max_norm over that norm; in
    place, or into `outs`, as many tensors of the same sizes and types. Returns
    that norm, a float32 scalar tensor. If an element is infinite or NaN, so is
    the norm, and only `scale` is applied; a norm that leaves the range of
    float32 alone is returned as infinity and clipped by in 64 bits."""
    given, grads = grads, _list(grads)
    if stream is not None:
        return _on(stream, grads.index, clip_grad_norm, grads, max_norm, scale, outs)
    if grads.index != _current_device():
        return _on_device(grads.index, clip_grad_norm, grads, max_norm, scale, outs)
    to = grads if outs is None else _list(outs)
    kept = to is outs or to is given
    device, nbytes = grads.device, grads.workspace_bytes
    if to is not grads and (to.device != device or to.shape != grads.shape):
        raise ValueError("outs must match grads in number, sizes, types and device")
    norm = torch.empty((), dtype=_F32, device=device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ptrs, counts, types = grads.arrays
    rc = vr.lib().vrClipGradNorm(ptrs, to.arrays[0], counts, types, len(ptrs), scale, max_norm,
                                 norm.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(grads.index))
    if rc:
        raise vr.VrError(rc, "vrClipGradNorm")
    _written(to.bases if kept else to.tensors)
    return norm
