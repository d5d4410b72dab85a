"""Autograd records nothing of layer norm, dropout and the embedding: inputs that
require a gradient are refused while it is recording. On the CPU, through the
host-only library."""
import os

import pytest
import torch

import ddp_bucketed_gradient_amd as D
from ddp_bucketed_gradient_amd import _abi, layers
from test_host_layers_reducer import cuda


@pytest.fixture
def lib(monkeypatch):
    if not os.path.exists(D.HOSTONLY_LIB):
        from ddp_bucketed_gradient_amd import build
        build.build_hostonly()
    monkeypatch.setattr(layers, "_call", lambda device, f, *args: None)
    return _abi.Lib(D.HOSTONLY_LIB)


N, H = 5, 8
DROP = D.Drop(0.5, 1)


def t():
    return cuda(N, dtype=torch.int64)


# every call, with the place that the input p takes in it
CALLS = {
    "norm x": lambda p, lib: D.layer_norm(p, lib=lib).y,
    "norm weight": lambda p, lib: D.layer_norm(cuda(N, H), p[0], lib=lib).y,
    "norm bias": lambda p, lib: D.layer_norm(cuda(N, H), None, p[0], lib=lib).y,
    "norm residual": lambda p, lib: D.layer_norm(cuda(N, H), residual=p, lib=lib).y,
    "dropout x": lambda p, lib: D.dropout(p, DROP, lib=lib),
    "dropout residual": lambda p, lib: D.dropout(cuda(N, H), D.Drop(0.0, 1), p, lib=lib),
    "dropout backward": lambda p, lib: D.dropout_backward(p, DROP, lib=lib),
    "table": lambda p, lib: D.embedding(t(), p, lib=lib),
    "lookup residual": lambda p, lib: D.embedding(t(), cuda(3, H), residual=p, lib=lib),
    "norm dy": lambda p, lib: D.layer_norm_backward(p, cuda(N, H), cuda(N, 2), lib=lib).dh,
    "norm h": lambda p, lib: D.layer_norm_backward(cuda(N, H), p, cuda(N, 2), lib=lib).dh,
    "norm grad_h": lambda p, lib: D.layer_norm_backward(cuda(N, H), cuda(N, H), cuda(N, 2), grad_h=p, lib=lib).dh,
    "lookup dy": lambda p, lib: D.embedding_backward(p, t(), cuda(3, H), lib=lib),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused_while_autograd_is_recording(lib, name):
    p = cuda(N, H).requires_grad_()
    with pytest.raises(ValueError, match="no_grad"):
        CALLS[name](p, lib)
    with torch.no_grad():
        assert not CALLS[name](p, lib).requires_grad
    assert not CALLS[name](p.detach(), lib).requires_grad


def test_not_refused_where_nothing_is_lost(lib):
    p = cuda(N, H).requires_grad_()
    assert D.dropout(p, D.Drop(0.0, 1), lib=lib) is p              # still p's own gradient
    w = cuda(H).requires_grad_()                                   # its gradient is what is being written
    D.layer_norm_backward(cuda(N, H), cuda(N, H), cuda(N, 2), w, cuda(H), lib=lib)


def test_inside_a_function_of_autograd(lib):
    """As a model wraps them: forward and backward run without recording."""
    class Dropped(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return D.dropout(x, DROP, lib=lib)

        @staticmethod
        def backward(ctx, dy):
            return D.dropout_backward(dy.as_subclass(type(cuda(1))), DROP, lib=lib)
    x = cuda(N, H).requires_grad_()
    y = Dropped.apply(x)
    assert y.requires_grad
    y.backward(cuda(N, H))
    assert x.grad.shape == x.shape
