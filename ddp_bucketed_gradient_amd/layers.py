"""Python front end of the operators beside a model's matrix products
(``include/ddpb.h``, "Beside the matrix products"): layer norm, dropout and the
embedding, each with its backward pass.

As elsewhere, PyTorch supplies device memory and streams and every step runs in
the native library. The functions work like torch's own: on the current stream
of the tensors' device, with outputs and workspaces from torch's allocator, so
they can be captured into graphs. They record nothing for autograd: the backward
passes are called by name and write the parameters' gradients where they are
told to, such as the tensors a Reducer is bound to. Where autograd is recording,
inputs that require a gradient are therefore refused: their results would not.
"""
from __future__ import annotations

import math as _math
from typing import NamedTuple, Optional

from . import _abi
from .optim import _code


_torch = None


def _t():
    """torch, imported with the first call."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


class Drop:
    """Which elements a dropout keeps: a function of the seed, the offset and an
    element's index, so that nothing is stored for the backward pass, which
    takes the same Drop. Two dropouts with one seed have one mask where their
    offsets, the counters included, are equal: no two, of any step, may be. With
    a counter of steps that is ``Drop(p, seed, offset=site << 32, counter=step)``,
    site numbering the dropouts of a step.

    ``p``: the share that is dropped, rounded to a multiple of 2^-16 (what is
    kept is scaled by just that share). ``counter``: None, or a 1-element int64
    CUDA tensor that is added to the offset when a call runs, so that a replayed
    graph drops anew once the counter has moved (behind the backward pass); it
    has to live as long as such a graph.
    """
    __slots__ = ("p", "seed", "offset", "counter", "active", "_c")

    def __init__(self, p: float, seed: int, offset: int = 0, counter=None):
        p = float(p)
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1]")
        at = None
        if counter is not None:
            import torch
            if not isinstance(counter, torch.Tensor) or counter.dtype != torch.int64 or not counter.is_cuda \
                    or counter.numel() != 1:
                raise ValueError("counter must be a 1-element int64 CUDA tensor")
            at = counter.data_ptr()
        m = (1 << 64) - 1
        self.p, self.seed, self.offset, self.counter = p, int(seed), int(offset), counter
        self.active = p * 65536 >= 0.5
        self._c = _abi.DropStruct(p, self.seed & m, self.offset & m, at)

    def _on(self, device):
        if self.counter is not None and self.counter.device != device:
            raise ValueError(f"the dropout's counter must be on {device}")
        return self._c

    def __repr__(self):
        return f"Drop(p={self.p}, seed={self.seed}, offset={self.offset}, counter={self.counter})"


class Normed(NamedTuple):
    """What layer_norm returns: y; h, the input of the norm (x itself without
    residual and dropout); stats, fp32, mean and 1 / deviation of each row."""
    y: object
    h: object
    stats: object


class NormGrads(NamedTuple):
    """What layer_norm_backward returns: the gradient of x, and that of h, which
    is the residual's (the same tensor without a dropout)."""
    dx: object
    dh: object


def _rows(t, what: str, like=None):
    """(rows, cols, stride) of a CUDA tensor whose rows, of its last dimension,
    lie at equal distances. ``like``: a tensor of the same shape, type and device."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{what} must have shape {tuple(like.shape)} and type {like.dtype} on {like.device}")
    if t.dim() == 0:
        raise ValueError(f"{what} must have at least one dimension")
    cols, n = t.shape[-1], t.numel()
    if t.is_contiguous():
        return (n // cols if cols else _math.prod(t.shape[:-1])), cols, cols
    if t.dim() == 2 and (cols == 1 or t.stride(1) == 1):
        return n // cols, cols, t.stride(0)
    if cols != 1 and t.stride(-1) != 1:
        raise ValueError(f"the elements of a row of {what} must be consecutive")
    stride = size = None
    for n_d, s_d in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n_d == 1:
            continue
        if stride is None:
            stride, size = s_d, n_d
        elif s_d != stride * size:
            raise ValueError(f"the rows of {what} must lie at equal distances: call contiguous() first")
        else:
            size *= n_d
    return n // cols, cols, cols if stride is None else stride


def _vector(t, what: str, n: int, device, dtype=None):
    """The address of an optional contiguous tensor of n elements."""
    if t is None:
        return 0
    if not t.is_cuda or t.device != device or not t.is_contiguous() or t.numel() != n or \
            (dtype is not None and t.dtype != dtype):
        kind = "" if dtype is None else f"{dtype} "
        raise ValueError(f"{what} must be a contiguous {kind}CUDA tensor of {n} elements on {device}")
    return t.data_ptr()


def _wanted(t):
    return t is not None and t.requires_grad


def _unrecorded():
    """Refuses inputs that require a gradient, which would be lost without a word."""
    if _t().is_grad_enabled():
        raise ValueError("an input requires a gradient, and autograd records nothing of this call: make it under "
                         "torch.no_grad() and call the backward pass by name, or pass a detached tensor")


def _call(device, f, *args):
    """f(*args, stream) on the current stream of ``device``."""
    torch = _t()
    i = device.index
    stream = torch._C._cuda_getCurrentRawStream(i)   # current_stream(device).cuda_stream without its Stream object
    if torch.cuda.current_device() == i:
        return f(*args, stream)
    with torch.cuda.device(device):
        return f(*args, stream)


def _like(t):
    """A new contiguous tensor of t's shape, type and device."""
    return _t().empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _wrote(*ts):
    """The gradients were written in place, through their addresses: autograd
    counts writes by tensor."""
    for t in ts:
        if t is not None:
            _t().autograd.graph.increment_version(t)


def _lib(lib):
    return lib if lib is not None else _abi.lib()


def dropout(x, drop: Drop, residual=None, lib: Optional[_abi.Lib] = None):
    """``x`` with a share of its elements dropped and the others scaled, plus
    ``residual``: a new contiguous tensor of x's type (fp32, bf16 or fp16). Where
    nothing is dropped or added that is x itself, as it lies, and no copy."""
    code = _code(x.dtype, "x")
    if residual is None and not drop.active:
        if not x.is_cuda:
            raise ValueError("x must be a CUDA tensor")
        return x
    if x.requires_grad or _wanted(residual):
        _unrecorded()
    rows, cols, stride = _rows(x, "x")
    rs = 0 if residual is None else _rows(residual, "residual", x)[2]
    y = _like(x)
    _call(x.device, _lib(lib).dropout, rows, cols, code, x.data_ptr(), stride,
          0 if residual is None else residual.data_ptr(), rs, drop._on(x.device), y.data_ptr())
    return y


def dropout_backward(dy, drop: Drop, lib: Optional[_abi.Lib] = None):
    """The gradient of dropout's x (the residual's is dy): dy itself where nothing
    is dropped."""
    return dropout(dy, drop, lib=lib)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, residual=None, drop: Optional[Drop] = None,
               lib: Optional[_abi.Lib] = None) -> Normed:
    """Layer norm over the last dimension of ``h = residual + dropout(x)``, in
    one pass. ``weight`` and ``bias``: one type, which may differ from x's."""
    if x.requires_grad or _wanted(weight) or _wanted(bias) or _wanted(residual):
        _unrecorded()
    code, dev = _code(x.dtype, "x"), x.device
    rows, cols, stride = _rows(x, "x")
    rs = 0 if residual is None else _rows(residual, "residual", x)[2]
    wt = weight.dtype if weight is not None else bias.dtype if bias is not None else x.dtype
    w, b = _vector(weight, "weight", cols, dev, wt), _vector(bias, "bias", cols, dev, wt)
    y = _like(x)
    fused = residual is not None or (drop is not None and drop.active)
    h = _like(x) if fused else x
    stats = x.new_empty(x.shape[:-1] + (2,), dtype=_t().float32)
    _call(dev, _lib(lib).layer_norm, rows, cols, code, x.data_ptr(), stride,
          0 if residual is None else residual.data_ptr(), rs, None if drop is None else drop._on(dev), w, b,
          _code(wt, "weight and bias"), eps, y.data_ptr(), h.data_ptr() if fused else 0, stats.data_ptr())
    return Normed(y, h, stats)


def _norm_backward(dy, h, stats, weight, dweight, dbias, grad_h, drop, accumulate, lib):
    """layer_norm_backward in steps: the checks here return the device, the bytes of the
    workspace and prepare(workspace, check), which allocates the outputs, has the library
    check the call as well, if so asked, and returns it. All but the call itself writes nothing."""
    torch = _t()
    if dy.requires_grad or h.requires_grad or _wanted(grad_h):
        _unrecorded()
    code, dev = _code(dy.dtype, "dy"), dy.device
    rows, cols, stride = _rows(dy, "dy")
    hs = _rows(h, "h", dy)[2]
    gs = 0 if grad_h is None else _rows(grad_h, "grad_h", dy)[2]
    st = _vector(stats, "stats", 2 * rows, dev, torch.float32)
    w = _vector(weight, "weight", cols, dev)
    wc = code if weight is None else _code(weight.dtype, "weight")
    gt = dweight.dtype if dweight is not None else dbias.dtype if dbias is not None else torch.float32
    dw, db = _vector(dweight, "dweight", cols, dev, gt), _vector(dbias, "dbias", cols, dev, gt)
    gc = _code(gt, "dweight and dbias")
    dropped = drop is not None and drop.active
    spec = drop._on(dev) if dropped else None
    lib = _lib(lib)
    nbytes = lib.layer_norm_backward_workspace_bytes(rows, cols) if dw or db else 0

    def prepare(ws, check):
        dh = _like(dy)
        dx = _like(dy) if dropped else dh
        args = (rows, cols, code, dy.data_ptr(), stride, h.data_ptr(), hs, st,
                0 if grad_h is None else grad_h.data_ptr(), gs, spec, w, wc, dh.data_ptr(),
                dx.data_ptr() if dropped else 0, dw, db, gc, accumulate, 0 if ws is None else ws.data_ptr(), nbytes)
        if check:
            lib.layer_norm_backward_check(*args)

        def run():
            _call(dev, lib.layer_norm_backward, *args)
            _wrote(dweight, dbias)
            return NormGrads(dx, dh)
        return run
    return dev, nbytes, prepare


def _workspace(device, nbytes):
    return _t().empty(nbytes, dtype=_t().uint8, device=device) if nbytes else None


def _alone(device, nbytes, prepare):
    """A backward pass by itself."""
    ws = _workspace(device, nbytes)
    return prepare(ws, False)()


def _together(passes):
    """The calls of several backward passes, all of them with their memory and checked
    by the library, and the workspaces, which have to be kept until they have been made.
    Passes on one device share one: they run one after the other on one stream."""
    most = {}
    for device, nbytes, _ in passes:
        most[device] = max(most.get(device, 0), nbytes)
    ws = {device: _workspace(device, nbytes) for device, nbytes in most.items()}
    return [prepare(ws[device], True) for device, _, prepare in passes], ws


def layer_norm_backward(dy, h, stats, weight=None, dweight=None, dbias=None, grad_h=None,
                        drop: Optional[Drop] = None, accumulate: bool = False,
                        lib: Optional[_abi.Lib] = None) -> NormGrads:
    """The gradients of layer_norm. ``h``, ``stats``: what it returned; ``drop``:
    the one it was called with. ``dweight``, ``dbias`` (any of them None if not
    wanted; one type): written, or with ``accumulate`` added to. ``grad_h``: a
    gradient that reaches h from elsewhere, as where h itself goes on as the
    next residual."""
    return _alone(*_norm_backward(dy, h, stats, weight, dweight, dbias, grad_h, drop, accumulate, lib))


def _tokens(tokens, device):
    """(count, address, bytes) of a tensor of tokens."""
    torch = _t()
    size = {torch.int64: 8, torch.int32: 4}.get(tokens.dtype)
    if size is None or not tokens.is_cuda or tokens.device != device or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous int64 or int32 CUDA tensor on {device}")
    return tokens.numel(), tokens.data_ptr(), size


def _table(t, what: str):
    if t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor of two dimensions")
    return t.shape[0], t.shape[1], _code(t.dtype, what)


def embedding(tokens, table, scale: float = 1.0, residual=None, dtype=None, lib: Optional[_abi.Lib] = None):
    """``scale * table[tokens] + residual``, of the table's type or ``dtype``. A
    token outside of the table gives a row of zeros."""
    if table.requires_grad or _wanted(residual):
        _unrecorded()
    vocab, cols, tc = _table(table, "table")
    dev = table.device
    n, at, size = _tokens(tokens, dev)
    dtype = table.dtype if dtype is None else dtype
    code = _code(dtype, "dtype")
    y = table.new_empty(tokens.shape + (cols,), dtype=dtype)
    rs = 0 if residual is None else _rows(residual, "residual", y)[2]
    _call(dev, _lib(lib).embedding, n, at, size, vocab, cols, table.data_ptr(), tc, scale,
          0 if residual is None else residual.data_ptr(), rs, y.data_ptr(), code)
    return y


def _embedding_backward(dy, tokens, dtable, scale, accumulate, lib):
    """embedding_backward in the steps of _norm_backward."""
    if dy.requires_grad:
        _unrecorded()
    vocab, cols, gc = _table(dtable, "dtable")
    dev = dtable.device
    n, at, size = _tokens(tokens, dev)
    if dy.device != dev or dy.shape != tokens.shape + (cols,):
        raise ValueError(f"dy must have shape {tuple(tokens.shape) + (cols,)} on {dev}")
    stride = _rows(dy, "dy")[2]
    code = _code(dy.dtype, "dy")
    lib = _lib(lib)
    nbytes = lib.embedding_backward_workspace_bytes(n, vocab, cols)

    def prepare(ws, check):
        args = (n, at, size, vocab, cols, dy.data_ptr(), stride, code, scale, dtable.data_ptr(), gc, accumulate,
                ws.data_ptr(), nbytes)
        if check:
            lib.embedding_backward_check(*args)

        def run():
            _call(dev, lib.embedding_backward, *args)
            _wrote(dtable)
            return dtable
        return run
    return dev, nbytes, prepare


def embedding_backward(dy, tokens, dtable, scale: float = 1.0, accumulate: bool = False,
                       lib: Optional[_abi.Lib] = None):
    """The gradient of embedding's table (the residual's is dy): row v of
    ``dtable`` becomes ``scale`` times the sum of dy over the places of token v,
    in their order; with ``accumulate`` that is added to it. Tokens outside of the
    table are left out. Returns dtable."""
    return _alone(*_embedding_backward(dy, tokens, dtable, scale, accumulate, lib))
