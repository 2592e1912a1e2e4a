"""The operators of a data-parallel training step around the AllReduce, on
torch tensors: layer norm, dropout, the norm and rotation of query and key heads,
and the losses of policies and preferences (each forward, backward, and as a
differentiable call), the norm of a list of gradients, and clipping by it.
Everything is computed by the kernels of libvr.so (include/vr.h states the
formulas and the rules); this module checks the tensors, allocates outputs and
workspaces, and passes addresses. There is no CPU fallback.

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


# ----------------------------------------------------------------- dropout
def _seed(seed, x, device):
    """(seed, address of the seed) of a number or of a CUDA tensor of one int64."""
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.get_device() != device:
            raise ValueError("seed must be an integer or one int64 on x's device")
        return 0, seed.data_ptr()
    if not 0 <= seed < 1 << 64:
        raise ValueError("seed must be in [0, 2^64)")
    return seed, None


def dropout_forward(x, p, seed, offset=0, residual=None, out=None, stream=None):
    """x / (1 - p) where an element stays, 0 where it is dropped (probability p), plus
    `residual` (of x's shape and type). Whether element i of x, counted along its
    shape, stays is a function of `seed` and of offset + i alone: no mask is kept, and
    a rank that gives the number of its part's first element as `offset` drops what
    one rank would with the whole batch. `seed`: an integer of [0, 2^64), or a CUDA
    tensor of one int64, read when the kernel runs, so that a captured graph draws
    anew once that tensor is changed. `out`: a tensor of x's shape and type, x and
    residual themselves allowed. Tensors of x's shape have a dense last axis and
    leading axes that are one row stride apart."""
    if stream is not None:
        return _on(stream, x.get_device(), dropout_forward, x, p, seed, offset, residual, out)
    cols, code, device = _check_x(x)
    if device != _current_device():
        return _on_device(device, dropout_forward, x, p, seed, offset, residual, out)
    if not 0 <= p <= 1:
        raise ValueError("p must be in [0, 1]")
    if not 0 <= offset < 1 << 64:
        raise ValueError("offset must be in [0, 2^64)")
    seed, at = _seed(seed, x, device)
    rows, xs = _rows(x, "x")
    rs = cols
    if residual is not None:
        _check_like(residual, x, device, "residual")
        rs = _rows(residual, "residual")[1]
    if out is None:
        y, ys = _dense_like(x), cols
    else:
        _check_like(out, x, device, "out")
        y, ys = out, _rows(out, "out")[1]
    rc = vr.lib().vrDropout(x.data_ptr(), _ptr(residual), y.data_ptr(), rows, cols, xs, rs, ys, p,
                            seed, at, offset, code, _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrDropout")
    if out is not None:
        _written(out)
    return y


def dropout_backward(dy, p, seed, offset=0, out=None, stream=None):
    """The gradient of dropout_forward's x from that of its result, with the same p,
    seed and offset (the residual's gradient is dy). `out`: dy itself allowed."""
    return dropout_forward(dy, p, seed, offset, None, out, stream)


def _as_rows(t):
    return t if not t.dim() or not t.shape[-1] or _has_rows(t) else t.contiguous()


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, offset, residual):
        tensor = isinstance(seed, torch.Tensor)
        ctx.save_for_backward(*([seed] if tensor else []))
        ctx.args = (p, None if tensor else seed, offset)
        return dropout_forward(_as_rows(x), p, seed, offset,
                               None if residual is None else _as_rows(residual))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        p, seed, offset = ctx.args
        if ctx.saved_tensors:
            seed, = ctx.saved_tensors
        dx = dropout_backward(_as_rows(dy), p, seed, offset) if ctx.needs_input_grad[0] else None
        return dx, None, None, None, dy if ctx.needs_input_grad[4] else None


def dropout(x, p, seed, offset=0, residual=None):
    """dropout_forward, differentiable once with respect to x and residual; tensors of
    other layouts are copied first. A seed tensor has to hold its value until the
    backward pass; autograd refuses one that was changed in place."""
    return _Dropout.apply(x, p, seed, offset, residual)


# ---------------------------------------------- norm and rotation of heads
@functools.lru_cache(maxsize=1024)
def _head_layout(shape, strides):
    """(batch, tokens, heads, dim, batch, token and head strides) of a tensor of (tokens,
    heads, dim) or (batch, tokens, heads, dim)."""
    n = len(shape)
    if n != 3 and n != 4:
        raise ValueError("heads must be (tokens, heads, dim) or (batch, tokens, heads, dim)")
    if strides[-1] != 1 and shape[-1] != 1:
        raise ValueError("the last axis of heads must be dense")
    batch, stride = (shape[0], strides[0]) if n == 4 else (1, 0)
    return (batch, *shape[-3:], vr.strides3(stride, strides[-3], strides[-2]))


def _heads(t, shape, dtype, device, what):
    """The strides of a tensor that has to have this shape, type and device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{what} does not match in shape, type or device")
    return _head_layout(shape, t.stride())[4]


def _keys(k, q, batch, tokens, dim, device):
    """(heads, strides) of the keys that go with q."""
    b, t, heads, d, strides = _head_layout(k.shape, k.stride())
    if b != batch or t != tokens or d != dim or k.dtype is not q.dtype or k.get_device() != device:
        raise ValueError("k does not match q in batch, tokens, dim, type or device")
    return heads, strides


def _rotation(cos, sin, positions, batch, tokens, dim, device):
    """The arguments that describe the rotation, of the forward and the backward pass."""
    if cos is None:
        if sin is not None:
            raise ValueError("cos and sin go together")
        return None, None, 0, None, 4, 0, 0
    if sin is None or positions is None:
        raise ValueError("a rotation needs cos, sin and positions")
    shape = cos.shape
    if sin.shape != shape or len(shape) != 2 or 2 * shape[1] > dim or cos.dtype is not _F32 or \
            sin.dtype is not _F32 or not cos.is_contiguous() or not sin.is_contiguous() or \
            cos.get_device() != device or sin.get_device() != device:
        raise ValueError("cos and sin must be dense float32 (positions, rotary / 2) on q's device")
    kind = _POSITION.get(positions.dtype)
    if kind is None or positions.get_device() != device:
        raise ValueError("positions must be int32 or int64 on q's device")
    at, strides = positions.shape, positions.stride()
    if at == (batch, tokens) and (tokens <= 1 or strides[1] == 1):
        step = strides[0]
    elif at == (tokens,) and (tokens <= 1 or strides[0] == 1):
        step = 0
    else:
        raise ValueError("positions must be (tokens,) or (batch, tokens), dense along tokens")
    return cos.data_ptr(), sin.data_ptr(), shape[0], positions.data_ptr(), kind, step, 2 * shape[1]


_POSITION = {torch.int32: vr.DTYPES["int32"], torch.int64: vr.DTYPES["int64"]}


def _head_weights(q, dim, device, *weights):
    """The type code of the given weights, one type for all."""
    first = None
    for w in weights:
        if w is None:
            continue
        _check_param(w, q, dim, device, first)
        first = w
    return _NORM_CODE[q.dtype if first is None else first.dtype]


def qk_norm_rope_forward(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                         eps=1e-6, interleaved=False, q_out=None, k_out=None, stream=None):
    """(q', k'): the root-mean-square norm of each head of q and k over its last axis,
    times the weight, rotated by its token's position. q: (batch, tokens, heads, dim) or
    (tokens, heads, dim), of any strides with a dense last axis, such as views of one
    projection's output or of (batch, heads, tokens, dim); k the same with heads of its
    own, or None. Weights: dense vectors of dim elements, shared by the heads. cos, sin:
    float32 tables of (positions, rotary / 2), rotary <= dim elements are rotated, in
    pairs of halves or, interleaved, of neighbours; None: no rotation. positions: int32
    or int64, (batch, tokens) or (tokens,). q_out and k_out: tensors of q's and k's
    shape, q and k themselves allowed."""
    if stream is not None:
        return _on(stream, q.get_device(), qk_norm_rope_forward, q, k, q_weight, k_weight, cos, sin,
                   positions, eps, interleaved, q_out, k_out)
    _, code, device = _check_x(q)
    if device != _current_device():
        return _on_device(device, qk_norm_rope_forward, q, k, q_weight, k_weight, cos, sin, positions,
                          eps, interleaved, q_out, k_out)
    batch, tokens, heads, dim, qs = _head_layout(q.shape, q.stride())
    dtype = q.dtype
    wcode = _head_weights(q, dim, device, q_weight, k_weight)
    kheads, ks, yk, yks = 0, None, None, None
    if k is not None:
        kheads, ks = _keys(k, q, batch, tokens, dim, device)
        yk = torch.empty_like(k) if k_out is None else k_out
        yks = _heads(yk, k.shape, dtype, device, "k_out")
    yq = torch.empty_like(q) if q_out is None else q_out
    yqs = _heads(yq, q.shape, dtype, device, "q_out")
    c, s, table, at, kind, step, rot = _rotation(cos, sin, positions, batch, tokens, dim, device)
    rc = vr.lib().vrQkNormRopeForward(
        q.data_ptr(), heads, qs, _ptr(k), kheads, ks, _ptr(q_weight), _ptr(k_weight), yq.data_ptr(),
        yqs, _ptr(yk), yks, c, s, table, at, kind, step, batch, tokens, dim, rot, interleaved, eps,
        code, wcode, _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrQkNormRopeForward")
    for t in (q_out, k_out if k is not None else None):
        if t is not None:
            _written(t)
    return yq, yk


@functools.lru_cache(maxsize=256)
def _qk_workspace(dim):
    return vr.vrQkNormRopeBackwardWorkspace(dim)


def qk_norm_rope_backward(dq, dk, q, k, q_weight=None, k_weight=None, cos=None, sin=None,
                          positions=None, eps=1e-6, interleaved=False, dq_weight=True,
                          dk_weight=True, dq_in=None, dk_in=None, stream=None):
    """(dq, dk, dq_weight, dk_weight): the gradients of qk_norm_rope_forward's inputs from
    those of its results. dq_weight and dk_weight may each be False (not wanted, None is
    returned) or a tensor to write to, such as a view of the flat bucket that the AllReduce
    takes; they have the weights' type (q's without). dq_in and dk_in: tensors for the
    gradients of q and k, such as views of one projection's gradient; dq and dk themselves
    allowed. With k None, dk and dk_in are not examined, and a tensor given as dk_weight
    is filled with zeros."""
    if stream is not None:
        return _on(stream, q.get_device(), qk_norm_rope_backward, dq, dk, q, k, q_weight, k_weight,
                   cos, sin, positions, eps, interleaved, dq_weight, dk_weight, dq_in, dk_in)
    _, code, device = _check_x(q)
    if device != _current_device():
        return _on_device(device, qk_norm_rope_backward, dq, dk, q, k, q_weight, k_weight, cos, sin,
                          positions, eps, interleaved, dq_weight, dk_weight, dq_in, dk_in)
    batch, tokens, heads, dim, qs = _head_layout(q.shape, q.stride())
    dtype = q.dtype
    given = [t for t in (dq_weight, dk_weight, dq_in, None if k is None else dk_in)
             if isinstance(t, torch.Tensor)]
    wcode = _head_weights(q, dim, device, q_weight, k_weight, *[
        t for t in (dq_weight, dk_weight) if isinstance(t, torch.Tensor)])
    dqs = _heads(dq, q.shape, dtype, device, "dq")
    dq_in = torch.empty_like(q) if dq_in is None else dq_in
    dqis = _heads(dq_in, q.shape, dtype, device, "dq_in")
    kheads, ks, dks, dkis = 0, None, None, None
    if k is not None:
        kheads, ks = _keys(k, q, batch, tokens, dim, device)
        dks = _heads(dk, k.shape, dtype, device, "dk")
        dk_in = torch.empty_like(k) if dk_in is None else dk_in
        dkis = _heads(dk_in, k.shape, dtype, device, "dk_in")
    else:
        dk, dk_in = None, None
        if not isinstance(dk_weight, torch.Tensor):  # a given one becomes zeros
            dk_weight = False
    grads = [dq_weight, dk_weight]
    for i in (0, 1):
        if grads[i] is True:
            like = (q_weight, k_weight)[i]
            grads[i] = torch.empty(dim, dtype=_TYPE[wcode], device=q.device) if like is None else \
                torch.empty_like(like)
        elif not isinstance(grads[i], torch.Tensor):
            grads[i] = None
    ws, nbytes = None, 0
    if grads[0] is not None or grads[1] is not None:
        nbytes = _qk_workspace(dim)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    c, s, table, at, kind, step, rot = _rotation(cos, sin, positions, batch, tokens, dim, device)
    rc = vr.lib().vrQkNormRopeBackward(
        dq.data_ptr(), dqs, _ptr(dk), dks, q.data_ptr(), heads, qs, _ptr(k), kheads, ks,
        _ptr(q_weight), _ptr(k_weight), dq_in.data_ptr(), dqis, _ptr(dk_in), dkis, _ptr(grads[0]),
        _ptr(grads[1]), c, s, table, at, kind, step, batch, tokens, dim, rot, interleaved, eps, code,
        wcode, _ptr(ws), nbytes, _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrQkNormRopeBackward")
    if given:
        _written(given)
    return dq_in, dk_in, grads[0], grads[1]


_TYPE = {c: t for t, c in _CODE.items()}


def _as_heads(t):
    return t if t is None or not t.dim() or t.shape[-1] == 1 or t.stride(-1) == 1 else t.contiguous()


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
        q, k = _as_heads(q), _as_heads(k)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.args = eps, interleaved
        ctx.set_materialize_grads(False)
        return qk_norm_rope_forward(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dq is None and dk is None:
            return (None,) * 9
        dq = torch.zeros_like(q) if dq is None else _as_heads(dq)
        if k is not None:
            dk = torch.zeros_like(k) if dk is None else _as_heads(dk)
        dq, dk, dqw, dkw = qk_norm_rope_backward(
            dq, dk, q, k, q_weight, k_weight, cos, sin, positions, *ctx.args,
            need[2] and q_weight is not None, need[3] and k_weight is not None)
        return (dq if need[0] else None, dk if need[1] else None, dqw, dkw, None, None, None, None,
                None)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6,
                 interleaved=False):
    """qk_norm_rope_forward, differentiable once with respect to q, k and the weights.
    Heads whose last axis is not dense are copied first."""
    return _QkNormRope.apply(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)


# ------------------------------------------------------------------ losses
def _check_logits(logits, targets):
    """(columns, type code, device index, rows, row stride) of a matrix of logits and its
    targets."""
    shape = logits.shape
    code = _NORM_CODE.get(logits.dtype)
    if code is None or not logits.is_cuda or not shape or not shape[-1]:
        _bad_x(logits)
    device = logits.get_device()
    if targets.dtype is not torch.int64 or targets.get_device() != device or \
            targets.shape != shape[:-1] or not targets.is_contiguous():
        raise ValueError("targets must be dense int64 of the logits' leading axes, on their device")
    rows, stride = (targets.numel(), shape[-1]) if logits.is_contiguous() else _rows(logits, "logits")
    return shape[-1], code, device, rows, stride


def _row_vectors(device, shape, *tensors):
    """The addresses of dense float32 vectors with a number for each row; None stays None."""
    at = []
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        if t.dtype is not _F32 or t.get_device() != device or t.shape != shape or not t.is_contiguous():
            raise ValueError("numbers of rows must be dense float32 of the targets' shape, on their device")
        at.append(t.data_ptr())
    return at


def _gradient_of(logits, out, device, cols):
    """(a tensor for the logits' gradient, its row stride)"""
    if out is None:
        return _dense_like(logits), cols
    _check_like(out, logits, device, "out")
    return out, _rows(out, "out")[1]


def token_logprobs_forward(logits, targets, rest=False, stream=None):
    """(logp, lse): the log probability of each row's target, and the logarithm of the sum
    of the row's exponentials (what the backward pass needs), float32. logits: (...,
    vocabulary), a dense last axis and leading axes that are one row stride apart;
    targets: int64 of the leading axes. A row of a negative target is not read: it gives 0.
    rest=True: (logp, lse, rest), with what lse lost by being rounded, for gradients of
    rows whose logits are all large (of 2^10 lse alone leaves them an error of 2^-14)."""
    if stream is not None:
        return _on(stream, logits.get_device(), token_logprobs_forward, logits, targets, rest)
    cols, code, device, rows, xs = _check_logits(logits, targets)
    if device != _current_device():
        return _on_device(device, token_logprobs_forward, logits, targets, rest)
    logp = torch.empty_like(targets, dtype=_F32)
    lse = torch.empty_like(logp)
    rest = torch.empty_like(logp) if rest else None
    rc = vr.lib().vrTokenLogProbsForward(logits.data_ptr(), targets.data_ptr(), logp.data_ptr(),
                                         lse.data_ptr(), _ptr(rest), rows, cols, xs, code,
                                         _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrTokenLogProbsForward")
    return (logp, lse) if rest is None else (logp, lse, rest)


def token_logprobs_backward(dlogp, logits, targets, lse, rest=None, gain=None, out=None,
                            stream=None):
    """The gradient of the logits from that by logp, times `gain` (a float32 scalar
    tensor, such as a loss's gradient). Rows of dlogp 0 or of a negative target are 0
    whatever their logits hold. `out`: a tensor of the logits' shape and type, logits
    themselves allowed."""
    if stream is not None:
        return _on(stream, logits.get_device(), token_logprobs_backward, dlogp, logits, targets, lse,
                   rest, gain, out)
    cols, code, device, rows, xs = _check_logits(logits, targets)
    if device != _current_device():
        return _on_device(device, token_logprobs_backward, dlogp, logits, targets, lse, rest, gain, out)
    if gain is not None and (gain.dtype != _F32 or gain.numel() != 1 or gain.get_device() != device):
        raise ValueError("gain must be one float32 on the logits' device")
    if dlogp is None or lse is None:
        raise ValueError("the gradient needs dlogp and lse")
    c, s, r = _row_vectors(device, targets.shape, dlogp, lse, rest)
    dx, ds = _gradient_of(logits, out, device, cols)
    rc = vr.lib().vrTokenLogProbsBackward(c, _ptr(gain), logits.data_ptr(), targets.data_ptr(), s,
                                          r, dx.data_ptr(), rows, cols, xs, ds, code,
                                          _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrTokenLogProbsBackward")
    if out is not None:
        _written(out)
    return dx


def _policy(logits, targets, old_logp, advantages, weights, ref_logp, clip_low, clip_high, kl_coef,
            scale, gradient, out):
    """(loss, logp, lse, dlogp, rest), or (loss, logp, dlogits) of the gradient in one pass"""
    cols, code, device, rows, xs = _check_logits(logits, targets)
    if device != _current_device():
        return _on_device(device, _policy, logits, targets, old_logp, advantages, weights, ref_logp,
                          clip_low, clip_high, kl_coef, scale, gradient, out)
    if old_logp is None or advantages is None:
        raise ValueError("a policy loss needs old_logp and advantages")
    vectors = _row_vectors(device, targets.shape, old_logp, advantages, weights, ref_logp)
    dx, ds = _gradient_of(logits, out, device, cols) if gradient else (None, 0)
    loss = torch.empty((), dtype=_F32, device=logits.device)
    logp = torch.empty_like(old_logp)
    kept, n, at = _row_buffers(logits, rows, 8 * rows)
    rc = vr.lib().vrPolicyLoss(logits.data_ptr(), targets.data_ptr(), *vectors, loss.data_ptr(),
                               logp.data_ptr(), at, at + 8 * n, at + 4 * n, _ptr(dx), rows, cols, xs,
                               ds, clip_low, clip_high, kl_coef, scale, code, at + 12 * n, 8 * rows,
                               _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrPolicyLoss")
    if gradient:
        if out is not None:
            _written(out)
        return loss, logp, dx
    return loss, logp, *_kept_rows(kept, n, targets)


def _row_buffers(logits, rows, extra):
    """(tensor, n, address): one allocation for what a call keeps of its rows, three times n
    floats (lse, dlogp, rest), and `extra` bytes behind them."""
    n = (rows + 3) // 4 * 4
    kept = torch.empty(3 * n + extra // 4, dtype=_F32, device=logits.device)
    return kept, n, kept.data_ptr()


def _kept_rows(kept, n, targets):
    """(lse, dlogp, rest)"""
    rows = targets.numel()
    return tuple(kept[i * n: i * n + rows].view(targets.shape) for i in range(3))


def policy_loss_forward(logits, targets, old_logp, advantages, weights=None, ref_logp=None,
                        clip_low=0.2, clip_high=0.2, kl_coef=0.0, scale=1.0, stream=None):
    """(loss, logp, lse, dlogp): the clipped policy loss of the rows of `logits`, whose
    tokens `targets` were sampled by a policy that gave them old_logp:
        scale sum(weights (-min(ratio A, clip(ratio, 1 - clip_low, 1 + clip_high) A)
                           + kl_coef (exp(ref_logp - logp) - (ref_logp - logp) - 1)))
    with ratio = exp(logp - old_logp). old_logp, advantages (A), weights and ref_logp are
    float32 of the targets' shape; without weights a row's is 1, without ref_logp the
    second term is left out. Rows of weight 0 or of a negative target count for nothing,
    whatever they hold. For a mean give weights, or a scale, of 1 over the tokens that
    count, of all ranks. dlogp is the loss's gradient by logp: token_logprobs_backward
    makes the logits' of it."""
    if stream is not None:
        return _on(stream, logits.get_device(), policy_loss_forward, logits, targets, old_logp,
                   advantages, weights, ref_logp, clip_low, clip_high, kl_coef, scale)
    return _policy(logits, targets, old_logp, advantages, weights, ref_logp, clip_low, clip_high,
                   kl_coef, scale, False, None)[:4]


def policy_loss_gradient(logits, targets, old_logp, advantages, weights=None, ref_logp=None,
                         clip_low=0.2, clip_high=0.2, kl_coef=0.0, scale=1.0, out=None,
                         stream=None):
    """(loss, logp, dlogits) of policy_loss_forward's loss and its gradient by the logits in
    one pass over them: for a step that goes on with logits.backward(dlogits). `out`: a
    tensor of the logits' shape and type for the gradient, logits themselves allowed."""
    if stream is not None:
        return _on(stream, logits.get_device(), policy_loss_gradient, logits, targets, old_logp,
                   advantages, weights, ref_logp, clip_low, clip_high, kl_coef, scale, out)
    return _policy(logits, targets, old_logp, advantages, weights, ref_logp, clip_low, clip_high,
                   kl_coef, scale, True, out)


def _preference(logits, targets, ref_logps, starts, beta, label_smoothing, scale, gradient, out):
    """(loss, logps, lse, dlogp, rest), or (loss, logps, dlogits)"""
    cols, code, device, rows, xs = _check_logits(logits, targets)
    if device != _current_device():
        return _on_device(device, _preference, logits, targets, ref_logps, starts, beta,
                          label_smoothing, scale, gradient, out)
    if starts is not None:
        if starts.dtype != torch.int64 or starts.dim() != 1 or starts.shape[0] < 3 or \
                starts.shape[0] % 2 == 0 or not starts.is_contiguous() or \
                starts.get_device() != device:
            raise ValueError("starts must be a dense int64 vector of 2 pairs + 1, on the logits' device")
        pairs = starts.shape[0] // 2
    elif logits.dim() < 3 or logits.shape[0] < 2 or logits.shape[0] % 2:
        raise ValueError("without starts, logits must be (2 pairs, tokens, vocabulary)")
    else:
        pairs = logits.shape[0] // 2
    if ref_logps is not None and (ref_logps.dtype is not _F32 or ref_logps.shape != (2, pairs) or
                                  not ref_logps.is_contiguous() or ref_logps.get_device() != device):
        raise ValueError("ref_logps must be dense float32 (2, pairs), on the logits' device")
    dx, ds = _gradient_of(logits, out, device, cols) if gradient else (None, 0)
    loss = torch.empty((), dtype=_F32, device=logits.device)
    logps = torch.empty((2, pairs), dtype=_F32, device=logits.device)
    n = (rows + 3) // 4 * 4  # the tokens' logp and a workspace
    kept, n, at = _row_buffers(logits, rows, 4 * n + 16 * pairs)
    rc = vr.lib().vrPreferenceLoss(logits.data_ptr(), targets.data_ptr(), _ptr(ref_logps),
                                   _ptr(starts), loss.data_ptr(), logps.data_ptr(), at + 12 * n, at,
                                   at + 8 * n, at + 4 * n, _ptr(dx), pairs, rows, cols, xs, ds, beta,
                                   label_smoothing, scale, code, at + 16 * n, 16 * pairs,
                                   _raw_stream(device))
    if rc:
        raise vr.VrError(rc, "vrPreferenceLoss")
    if gradient:
        if out is not None:
            _written(out)
        return loss, logps, dx
    return loss, logps, *_kept_rows(kept, n, targets)


def preference_loss_forward(logits, targets, ref_logps=None, starts=None, beta=0.1,
                            label_smoothing=0.0, scale=1.0, stream=None):
    """(loss, logps, lse, dlogp): the loss of preferences between pairs of sequences by the
    ratio of their probabilities under the policy to those under a reference,
        h = beta ((logps - ref_logps)[0] - (logps - ref_logps)[1])
        scale sum over pairs ((1 - label_smoothing) log(1 + exp(-h)) + label_smoothing log(1 + exp(h)))
    with logps (2, pairs) the sums of the sequences' log probabilities, row 0 of the chosen
    ones, row 1 of the rejected ones. The sequences are the rows of `logits` in that order:
    (2 pairs, tokens, vocabulary), or packed with starts, int64, of 2 pairs + 1 rows where
    sequences begin and end, none smaller than the one before. Tokens of negative targets (prompts, padding) count for nothing.
    ref_logps: float32 (2, pairs), None: zeros. dlogp is the loss's gradient by the tokens'
    log probabilities: token_logprobs_backward makes the logits' of it."""
    if stream is not None:
        return _on(stream, logits.get_device(), preference_loss_forward, logits, targets, ref_logps,
                   starts, beta, label_smoothing, scale)
    return _preference(logits, targets, ref_logps, starts, beta, label_smoothing, scale, False,
                       None)[:4]


def preference_loss_gradient(logits, targets, ref_logps=None, starts=None, beta=0.1,
                             label_smoothing=0.0, scale=1.0, out=None, stream=None):
    """(loss, logps, dlogits) of preference_loss_forward's loss and its gradient by the
    logits, for a step that goes on with logits.backward(dlogits). `out`: a tensor of the
    logits' shape and type for the gradient, logits themselves allowed."""
    if stream is not None:
        return _on(stream, logits.get_device(), preference_loss_gradient, logits, targets, ref_logps,
                   starts, beta, label_smoothing, scale, out)
    return _preference(logits, targets, ref_logps, starts, beta, label_smoothing, scale, True, out)


class _TokenLogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets):
        logits, targets = _as_rows(logits), targets.contiguous()
        logp, lse, rest = token_logprobs_forward(logits, targets, True)
        ctx.save_for_backward(logits, targets, lse, rest)
        return logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dlogp):
        return token_logprobs_backward(dlogp.contiguous(), *ctx.saved_tensors), None


class _Loss(torch.autograd.Function):
    """A loss of rows of logits, of which forward keeps the gradient by each row's logp."""

    @staticmethod
    def forward(ctx, logits, targets, loss, *args):
        logits, targets = _as_rows(logits), targets.contiguous()
        value, logp, lse, dlogp, rest = loss(logits, targets, *args, False, None)
        ctx.save_for_backward(logits, targets, lse, dlogp, rest)
        ctx.mark_non_differentiable(logp)
        ctx.rest = len(args)
        return value, logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gain, _):
        logits, targets, lse, dlogp, rest = ctx.saved_tensors
        d = token_logprobs_backward(dlogp, logits, targets, lse, rest, gain.contiguous())
        return (d, None, None) + (None,) * ctx.rest


def token_logprobs(logits, targets):
    """The log probability of each row's target, float32, differentiable once with respect
    to the logits; logits of layouts other than token_logprobs_forward's are copied first."""
    return _TokenLogProbs.apply(logits, targets)


def policy_loss(logits, targets, old_logp, advantages, weights=None, ref_logp=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, scale=1.0):
    """(loss, logp) of policy_loss_forward, the loss differentiable once with respect to the
    logits. It reads the logits forward and again backward; policy_loss_gradient does
    both in one pass."""
    return _Loss.apply(logits, targets, _policy, old_logp, advantages, weights, ref_logp,
                       clip_low, clip_high, kl_coef, scale)


def preference_loss(logits, targets, ref_logps=None, starts=None, beta=0.1, label_smoothing=0.0,
                    scale=1.0):
    """(loss, logps) of preference_loss_forward, the loss differentiable once with respect to
    the logits."""
    return _Loss.apply(logits, targets, _preference, ref_logps, starts, beta,
                       label_smoothing, scale)
