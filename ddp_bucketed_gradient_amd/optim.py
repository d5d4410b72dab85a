"""Python front end of what follows a synchronisation: the global gradient norm
and the AdamW step (``include/ddpb.h``, "After the synchronisation").

As for the reducer, PyTorch supplies device memory and streams and every step
of the operators runs in the native library. The objects keep references to the
tensors they were given; these must keep their storage (no resize or set_).
"""
from __future__ import annotations

import sys as _sys
from numbers import Real as _Real
from typing import Optional, Sequence, Union

from . import _abi

_TYPES = None


def _types():
    global _TYPES
    if _TYPES is None:
        import torch
        _TYPES = {torch.float32: _abi.F32, torch.bfloat16: _abi.BF16, torch.float16: _abi.F16}
    return _TYPES


def _code(dtype, what: str) -> int:
    c = _types().get(dtype)
    if c is None:
        raise ValueError(f"{what} must be fp32, bf16 or fp16, not {dtype}")
    return c


def _device(ts, what: str):
    """The device of a list of tensors: the first one's, which is a GPU."""
    import torch
    if not ts:
        return torch.device("cuda", torch.cuda.current_device())
    if ts[0] is None or not ts[0].is_cuda:
        raise ValueError(f"{what}[0] must be a CUDA tensor")
    return ts[0].device


def _check(ts, what: str, numels, dtype, device) -> list:
    """Addresses of contiguous CUDA tensors of one dtype and device."""
    if len(ts) != len(numels):
        raise ValueError(f"{what}: {len(ts)} tensors for {len(numels)} variables")
    ptrs = []
    for v, (t, n) in enumerate(zip(ts, numels)):
        if t is None or t.dtype != dtype or t.device != device or not t.is_contiguous() or t.numel() != n:
            raise ValueError(f"{what}[{v}] must be a contiguous {dtype} CUDA tensor of {n} elements on {device}")
        ptrs.append(t.data_ptr())
    return ptrs


class _Handle:
    """A native handle with its workspace, bound to one stream of one device.

    A graph that captured its calls uses its memory: the object has to live as
    long as the graph is replayed."""
    _destroy = ""

    def _open(self, lib, h, device, stream, reducer):
        import torch
        self.lib, self.h, self.device, self._reducer = lib, h, device, reducer
        if reducer is not None:
            if getattr(reducer, "compute_stream", None) is None:
                raise _abi.DdpbError(_abi.E_STATE, "the reducer is not bound to tensors")
            if stream is not None and stream != reducer.compute_stream:
                raise ValueError("with a reducer the stream is its compute stream")
            stream = reducer.compute_stream
        self.stream = stream if stream is not None else torch.cuda.current_stream(device)
        if self.stream.device != device:
            raise ValueError(f"the stream belongs to {self.stream.device}, the tensors to {device}")
        # what the caller has enqueued on the tensors so far comes first
        if not torch.cuda.is_current_stream_capturing():
            self.stream.wait_stream(torch.cuda.current_stream(device))
        # allocated for the stream that uses it, so that freeing it needs no wait
        with torch.cuda.device(device), torch.cuda.stream(self.stream):
            self.workspace = torch.empty(self._workspace_bytes(), dtype=torch.uint8, device=device)

    def _red(self):
        """The reducer's handle for a call, or None."""
        if self._reducer is None:
            return None
        if not self._reducer.h:
            raise _abi.DdpbError(_abi.E_STATE, "the reducer was closed")
        return self._reducer.h

    def close(self):
        """Release the handle. Work that is still enqueued finishes: no tensor's
        memory is given to another one before it."""
        if self.h:
            getattr(self.lib, self._destroy)(self.h)
            self.h = None
            # The caller's tensors may have been allocated for other streams than
            # the one they are used on; the allocator has to know that one before
            # the last reference goes. Nothing happens where it is the same.
            for t in self._keep or ():
                t.record_stream(self.stream)
            self._keep = None

    def __del__(self):
        try:
            if _sys.is_finalizing():
                return
            self.close()
        except BaseException:
            pass


class GradNorm(_Handle):
    """Global norm of a list of gradients, with its clip coefficient.

    ``grads``: contiguous fp32, bf16 or fp16 CUDA tensors, also mixed. Work runs
    on ``stream`` (default: the current one), or on the compute stream of
    ``reducer``, whose state is then checked before each call.

    ``norm`` and ``coef`` are fp32 device scalars that each compute() rewrites.
    """
    _destroy = "norm_destroy"

    def __init__(self, grads: Sequence, stream=None, reducer=None, lib: Optional[_abi.Lib] = None):
        import torch
        self.h = self._keep = None
        lib = lib if lib is not None else _abi.lib()
        grads = list(grads)
        dev = _device(grads, "grads")
        ptrs = []
        for v, t in enumerate(grads):
            if t is None or t.device != dev or not t.is_contiguous():
                raise ValueError(f"grads[{v}] must be a contiguous CUDA tensor on {dev}")
            ptrs.append(t.data_ptr())
        h = lib.norm_create([t.numel() for t in grads], [_code(t.dtype, "gradients") for t in grads])
        self._open(lib, h, dev, stream, reducer)
        self._keep = grads
        with torch.cuda.device(dev):
            lib.norm_bind(h, ptrs, self.workspace.data_ptr(), self.workspace.numel(), self.stream.cuda_stream,
                          self._red())
        head = self.workspace[:16]
        self.norm, self.coef = head.view(torch.float32)[0], head.view(torch.float32)[1]
        self.skipped = head.view(torch.int32)[2]
        self._result = self.workspace.data_ptr()

    def _workspace_bytes(self):
        return self.lib.norm_workspace_bytes(self.h)

    def compute(self, max_norm: float = float("inf"), grad_scale: float = 1.0, skip_nonfinite: bool = False):
        """Enqueue the norm of ``grads * grad_scale`` and its coefficient
        (max_norm / norm above max_norm, else 1); returns ``norm``. With
        ``skip_nonfinite`` a step that is given this norm does nothing when it
        is infinite or NaN."""
        self.lib.norm_compute(self.h, max_norm, grad_scale, 1 if skip_nonfinite else 0, self._red())
        return self.norm


class AdamW(_Handle):
    """AdamW over all tensors in one launch per step.

    ``params``: one tensor for each variable, or R rows of them (the replicas:
    every row receives the new values, row 0 is read). ``grads``: one tensor
    for each variable. ``state``: "f32", or "f8" for 8-bit states (e4m3 codes
    of m and of sqrt(v) with an e8m0 scale for every 64 elements, rounded
    stochastically from ``seed``). ``master``: fp32 copies for 16-bit
    parameters, or True to make them from ``params``. ``weight_decay`` and
    ``lr_scale``: a number, or one for each variable. ``states``: the state to
    go on from (a dict of lists as ``exp_avg`` and its like below) after
    ``step`` steps; by default zeros. Work runs on ``stream`` (default: the
    current one) or the compute stream of ``reducer``.

    Attributes: ``exp_avg`` and ``exp_avg_sq`` (fp32) or ``exp_avg``,
    ``exp_avg_root`` (float8_e4m3fn), ``avg_scale``, ``root_scale``
    (float8_e8m0fnu); ``master``; ``lr`` (a float, or a 1-element fp32 CUDA
    tensor that the step reads when it runs, behind what the current stream has
    enqueued; it has to live as long as a graph that captured the step).
    """
    _destroy = "adamw_destroy"

    def __init__(self, params: Sequence, grads: Sequence, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: Union[float, Sequence[float]] = 0.01, state: str = "f32", master=None,
                 lr_scale: Union[None, float, Sequence[float]] = None, states: Optional[dict] = None, step: int = 0,
                 seed: int = 0, stream=None, reducer=None, lib: Optional[_abi.Lib] = None):
        import torch
        self.h = self._keep = None
        lib = lib if lib is not None else _abi.lib()
        params, grads = list(params), list(grads)
        rows = [list(r) for r in params] if params and isinstance(params[0], (list, tuple)) else [params]
        P = len(grads)
        if state not in ("f32", "f8"):
            raise ValueError('state must be "f32" or "f8"')
        f8 = state == "f8"
        dev = _device(grads, "grads")
        if any(t is None for ts in [grads] + rows for t in ts):
            raise ValueError("every variable needs a parameter and a gradient tensor")
        numel = [t.numel() for t in grads]
        pt = rows[0][0].dtype if P and rows[0] else torch.float32
        gt = grads[0].dtype if P else torch.float32
        pc, gc = _code(pt, "parameters"), _code(gt, "gradients")
        pp = [a for r, row in enumerate(rows) for a in _check(row, f"params[{r}]", numel, pt, dev)]
        gp = _check(grads, "grads", numel, gt, dev)
        every = lambda x: [float(x)] * P if isinstance(x, _Real) else [float(y) for y in x]  # noqa: E731
        self._options = {"betas": (float(betas[0]), float(betas[1])), "eps": float(eps),
                         "weight_decay": every(weight_decay), "lr_scale": None if lr_scale is None else every(lr_scale),
                         "state": state, "seed": int(seed)}
        h = lib.adamw_create(numel, len(rows), pc, gc, _abi.STATE_F8 if f8 else _abi.STATE_F32,
                             _abi.ADAMW_MASTER if master is not None and master is not False else 0,
                             *self._options["betas"], self._options["eps"], self._options["weight_decay"],
                             self._options["lr_scale"], seed)
        self._open(lib, h, dev, stream, reducer)
        with torch.cuda.device(dev), torch.cuda.stream(self.stream):
            self.master = None
            if master is True:
                self.master = self._flat(numel, torch.float32)
                for w, p in zip(self.master, rows[0]):
                    w.copy_(p.detach().reshape(-1))
            elif master is not None and master is not False:
                self.master = list(master)
            blocks = [-(-n // _abi.STATE_BLOCK) for n in numel]
            kinds = {"exp_avg": (numel, torch.float8_e4m3fn), "exp_avg_root": (numel, torch.float8_e4m3fn),
                     "avg_scale": (blocks, torch.float8_e8m0fnu), "root_scale": (blocks, torch.float8_e8m0fnu)} if f8 \
                else {"exp_avg": (numel, torch.float32), "exp_avg_sq": (numel, torch.float32)}
            if states is not None and set(states) != set(kinds):
                raise ValueError(f"states must hold {sorted(kinds)}")
            self._state = {k: self._flat(*kinds[k]) if states is None else list(states[k]) for k in kinds}
        at = {k: _check(ts, k, *kinds[k], dev) for k, ts in self._state.items()}
        mp = None if self.master is None else _check(self.master, "master", numel, torch.float32, dev)
        self.lr = lr
        self.params, self.grads = rows, grads
        # The step writes through addresses; autograd counts writes by tensor, to
        # refuse a backward that needs the values from before.
        self._count_write = torch.autograd.graph.increment_version
        self._written = [t for row in (*rows, self.master or ()) for t in row]
        self._keep = [t for ts in (*rows, grads, self.master or (), *self._state.values()) for t in ts]
        with torch.cuda.device(dev):
            lib.adamw_bind(h, pp, gp, mp, at["exp_avg"], at["exp_avg_root" if f8 else "exp_avg_sq"],
                           at.get("avg_scale"), at.get("root_scale"), step, self.workspace.data_ptr(),
                           self.workspace.numel(), self.stream.cuda_stream, self._red())

    def _workspace_bytes(self):
        return self.lib.adamw_workspace_bytes(self.h)

    def _flat(self, numel, dtype):
        """Zeroed tensors in one allocation, each on a 256-byte boundary."""
        import torch
        size = torch.empty(0, dtype=dtype).element_size()
        off, at = [], 0
        for n in numel:
            off.append(at)
            at += -(-n * size // 256) * 256
        flat = torch.zeros(max(at, 1), dtype=torch.uint8, device=self.device)
        return [flat[o:o + n * size].view(dtype) for o, n in zip(off, numel)]

    def __getattr__(self, name):
        s = self.__dict__.get("_state")
        if s is not None and name in s:
            return s[name]
        raise AttributeError(name)

    def step(self, lr=None, grad_scale: float = 1.0, clip: Optional[GradNorm] = None):
        """Enqueue one step. ``lr`` (default: the attribute) and ``grad_scale``
        (the factor that takes a loss scale out) as in the class; ``clip``: a
        GradNorm on the same stream whose compute() was called before.
        Parameters and masters count as written in place for autograd, by the
        call; replays of a graph that captured it are not seen."""
        lr = self.lr if lr is None else lr
        at = 0
        if type(lr) is not float and not isinstance(lr, _Real):
            import torch
            if not isinstance(lr, torch.Tensor) or lr.dtype != torch.float32 or not lr.is_cuda or lr.device != self.device or lr.numel() != 1:
                raise ValueError("lr must be a number or a 1-element fp32 CUDA tensor on the parameters' device")
            # read when the step runs, behind what the current stream wrote; in a
            # capture the caller has ordered the streams (or they are the same)
            now = torch.cuda.current_stream(self.device)
            if now != self.stream and not torch.cuda.is_current_stream_capturing():
                self.stream.wait_stream(now)
            lr.record_stream(self.stream)
            at, lr = lr.data_ptr(), 0.0
        result = 0
        if clip is not None:
            if clip.stream != self.stream:
                raise ValueError("clip must run on the same stream as the step")
            result = clip._result
        self.lib.adamw_step(self.h, lr, at, grad_scale, result, self._red())
        self._count_write(self._written)

    @property
    def states(self) -> dict:
        """The state's tensors, as the argument ``states`` takes them."""
        return {k: list(v) for k, v in self._state.items()}

    @property
    def options(self) -> dict:
        """Every argument but the tensors to update and the count of steps:
        rate, betas, eps, weight decay, rate factors, state type and seed, with
        the state and the masters as they stand. A new AdamW on the same
        parameters, or on copies after a restart or with gradients that have
        moved, goes on bit for bit when it is made with
        ``step=old.steps_done, **old.options``. (The tensors are shared, not
        copied: wait for the stream before saving them, and leave the old handle
        alone afterwards.)"""
        return {**self._options, "lr": self.lr, "states": self.states,
                "master": None if self.master is None else list(self.master)}

    @property
    def steps_done(self) -> int:
        """Steps that counted (waits for the stream)."""
        return self.lib.adamw_get_step(self.h)

    @steps_done.setter
    def steps_done(self, n: int):
        self.lib.adamw_set_step(self.h, n)
