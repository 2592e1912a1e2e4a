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

Calls are asynchronous on the current torch stream, or on `stream`; outputs and
workspaces are allocated there, so that they may be freed at any time. As with
any torch operation, tensors that were made or are freed on another stream
need the caller's own ordering (wait_stream, record_stream).
"""
import contextlib

import torch

import ring_allreduce_virtual_gb300 as vr

_CODE = {torch.float16: vr.DTYPES["float16"], torch.bfloat16: vr.DTYPES["bfloat16"],
         torch.float32: vr.DTYPES["float32"], torch.float64: vr.DTYPES["float64"]}
_NORM_TYPES = (torch.float16, torch.bfloat16, torch.float32)


def _on(stream):
    """Allocations go to `stream`'s pool too."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


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


def _check_params(x, weight, bias):
    if x.dtype not in _NORM_TYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if not x.is_cuda or x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be a CUDA tensor with a last axis of at least one element")
    wt = None
    for p in (weight, bias):
        if p is None:
            continue
        if p.device != x.device or p.dim() != 1 or p.shape[0] != x.shape[-1] or \
                not p.is_contiguous():
            raise ValueError("weight and bias must be dense vectors of x's last axis, on its device")
        if p.dtype not in (x.dtype, torch.float32) or wt not in (None, p.dtype):
            raise ValueError("weight and bias must have one type: x's or float32")
        wt = p.dtype
    return wt or x.dtype


def _ptr(t):
    return None if t is None else t.data_ptr()


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, stats=True, out=None, stream=None):
    """(y, mean, rstd): layer norm over x's last axis; mean and rstd (float32,
    x's leading shape) are what the backward pass needs, None with
    stats=False. `out`: a tensor of x's shape and type for y, x itself allowed."""
    wt = _check_params(x, weight, bias)
    rows, xs = _rows(x, "x")
    with _on(stream):
        if out is None:
            y, ys = torch.empty(x.shape, dtype=x.dtype, device=x.device), x.shape[-1]
        else:
            if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
                raise ValueError("out must have x's shape, type and device")
            y, ys = out, _rows(out, "out")[1]
        mean = rstd = None
        if stats:
            mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
            rstd = torch.empty_like(mean)
        vr.vrLayerNormForward(x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(mean),
                              _ptr(rstd), rows, x.shape[-1], xs, ys, eps, _CODE[x.dtype],
                              _CODE[wt], _raw_stream(x.device))
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, dx=True, dweight=True, dbias=True,
                        stream=None):
    """(dx, dweight, dbias) of layer_norm_forward. dx, dweight and dbias may
    each be False (not wanted, None is returned) or a tensor to write to, such as
    a view of the flat bucket that the AllReduce takes. The parameters'
    gradients have the weight's type (x's without a weight, or the given
    tensors')."""
    given = [t for t in (dweight, dbias) if isinstance(t, torch.Tensor)]
    wt = _check_params(x, weight if weight is not None else (given or [None])[0], None)
    cols = x.shape[-1]
    rows, xs = _rows(x, "x")
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != x.device:
        raise ValueError("dy must have x's shape, type and device")
    dys = _rows(dy, "dy")[1]
    for t in (mean, rstd):
        if t.dtype != torch.float32 or t.device != x.device or t.numel() != rows or \
                not t.is_contiguous():
            raise ValueError("mean and rstd must be the forward pass's")
    with _on(stream):
        dxs = cols
        if dx is True:
            dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        elif isinstance(dx, torch.Tensor):
            if dx.shape != x.shape or dx.dtype != x.dtype or dx.device != x.device:
                raise ValueError("dx must have x's shape, type and device")
            dxs = _rows(dx, "dx")[1]
        params = []
        for t in (dweight, dbias):
            if t is True:
                t = torch.empty(cols, dtype=wt, device=x.device)
            elif isinstance(t, torch.Tensor):
                if t.numel() != cols or t.dtype != wt or t.device != x.device or \
                        not t.is_contiguous():
                    raise ValueError("dweight and dbias must be dense vectors of the weight's type")
            else:
                t = None
            params.append(t)
        dx = None if dx is False else dx
        ws, nbytes = None, 0
        if params[0] is not None or params[1] is not None:
            nbytes = vr.vrLayerNormBackwardWorkspace(rows, cols, _CODE[x.dtype])
            ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        if dx is not None or ws is not None:
            vr.vrLayerNormBackward(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(),
                                   rstd.data_ptr(), _ptr(dx), _ptr(params[0]), _ptr(params[1]),
                                   rows, cols, dys, xs, dxs, _CODE[x.dtype], _CODE[wt], _ptr(ws),
                                   nbytes, _raw_stream(x.device))
    return dx, params[0], params[1]


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
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
    weight and bias; x's last axis is dense."""
    return _LayerNorm.apply(x, weight, bias, eps)


# ------------------------------------------------- gradient norm, clipping
class TensorList:
    """A list of gradients (or outputs) whose addresses have been checked and
    marshalled once; it keeps the tensors alive. Make it for buffers that stay
    where they are from step to step; a plain sequence of tensors works wherever
    a TensorList does and is marshalled for the call."""

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

    def __len__(self):
        return len(self.tensors)

    def like(self, other):
        """Same element counts and types."""
        return bytes(self.arrays[1]) == bytes(other.arrays[1]) and \
            bytes(self.arrays[2]) == bytes(other.arrays[2])


def _list(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def grad_norm(grads, scale=1.0, per_tensor=False, stream=None):
    """The 2-norm of all elements of `grads` (a TensorList or a sequence of
    tensors) times |scale|, a float32 scalar tensor; with per_tensor also the
    norms of the single tensors, a float32 vector."""
    grads = _list(grads)
    with _on(stream):
        norm = torch.empty((), dtype=torch.float32, device=grads.device)
        norms = torch.empty(len(grads), dtype=torch.float32, device=grads.device) \
            if per_tensor else None
        ws = torch.empty(grads.workspace_bytes, dtype=torch.uint8, device=grads.device)
        vr.vrGradNorm(grads.arrays, scale, norm.data_ptr(), _ptr(norms), ws.data_ptr(),
                      grads.workspace_bytes, _raw_stream(grads.device))
    return (norm, norms) if per_tensor else norm


def clip_grad_norm(grads, max_norm, scale=1.0, outs=None, stream=None):
    """Multiply `grads` (a TensorList or a sequence of tensors) by `scale` and,
    where the norm of the result exceeds max_norm, by max_norm over that norm; in
    place, or into `outs`, as many tensors of the same sizes and types. Returns
    that norm, a float32 scalar tensor. If it is not finite, only `scale` is
    applied."""
    grads = _list(grads)
    to = grads if outs is None else _list(outs)
    if to is not grads and (to.device != grads.device or not to.like(grads)):
        raise ValueError("outs must match grads in number, sizes, types and device")
    with _on(stream):
        norm = torch.empty((), dtype=torch.float32, device=grads.device)
        ws = torch.empty(grads.workspace_bytes, dtype=torch.uint8, device=grads.device)
        vr.vrClipGradNorm(grads.arrays, to.arrays[0], scale, max_norm, norm.data_ptr(),
                          ws.data_ptr(), grads.workspace_bytes, _raw_stream(grads.device))
    return norm
