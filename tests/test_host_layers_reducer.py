"""The reducer's backward passes on the CPU, through the host-only library, which
checks calls and enqueues nothing: what is refused, and when."""
import os
from types import SimpleNamespace

import pytest
import torch

import ddp_bucketed_gradient_amd as D
from ddp_bucketed_gradient_amd import _abi, layers

V, H, R, N = 50, 8, 3, 400


class Cuda(torch.Tensor):
    """A CPU tensor that passes for one of the GPU."""
    is_cuda = True


def cuda(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Cuda)


@pytest.fixture
def red(monkeypatch):
    if not os.path.exists(D.HOSTONLY_LIB):
        from ddp_bucketed_gradient_amd import build
        build.build_hostonly()
    r = D.Reducer([(V, H), (H,), (H,)], R, 0, lib=_abi.Lib(D.HOSTONLY_LIB))
    r._grads = [[cuda(V, H), cuda(H), cuda(H)] for _ in range(R)]
    r.bind_ptrs([t.data_ptr() for row in r._grads for t in row])
    r.compute_stream = SimpleNamespace(device=torch.device("cpu"), cuda_stream=0)
    r.calls = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: r.compute_stream)

    def call(device, f, *args):
        r.calls.append(f.__name__)
        return f(*args, 0)
    monkeypatch.setattr(layers, "_call", call)
    empty = torch.empty

    def aligned(n, **kw):                                  # as the GPU's allocator does
        t = empty(n + 256, **kw)
        return t[-t.data_ptr() % 256:][:n]
    monkeypatch.setattr(torch, "empty", aligned)
    yield r
    r.close()


@pytest.fixture
def norm(red):
    g = red._grads[0]
    h = red.lib.norm_create([t.numel() for t in g], [D.F32] * 3)
    ws = 1 << 45
    red.lib.norm_bind(h, [t.data_ptr() for t in g], ws, red.lib.norm_workspace_bytes(h), 0, red.h)

    def averaged():
        try:
            red.lib.norm_compute(h, 1.0, reducer=red.h)
        except D.DdpbError as e:
            assert e.code == D.E_STATE
            return False
        return True
    yield averaged
    red.lib.norm_destroy(h)


def rows():
    return [cuda(N, H) for _ in range(R)]


def stats():
    return [cuda(N, 2) for _ in range(R)]


def tokens():
    return [cuda(N, dtype=torch.int64) for _ in range(R)]


def over(t):
    """A tensor of N rows that begins inside the storage of t."""
    return torch.as_strided(t.view(-1), (N, H), (0, 1), t.storage_offset()).as_subclass(Cuda)


def test_a_replica_that_the_library_refuses_leaves_the_others_unwritten(red, norm):
    for bad in range(R):
        dy = rows()
        dy[bad] = over(red._grads[bad][0])          # reads the gradient that the call writes
        with pytest.raises(D.DdpbError, match="overlaps") as e:
            red.embedding_backward(0, dy, tokens())
        assert e.value.code == D.E_ARG
        h = rows()
        h[bad] = over(red._grads[bad][1])
        with pytest.raises(D.DdpbError, match="overlaps"):
            red.layer_norm_backward(1, 2, rows(), h, stats())
    assert red.calls == [] and norm()                      # nothing enqueued: the averages stand
    red.layer_norm_backward(1, 2, rows(), rows(), stats())
    red.embedding_backward(0, rows(), tokens())
    assert red.calls == ["layer_norm_backward"] * R + ["embedding_backward"] * R
    red.finalize()
    assert norm()


def test_no_memory_leaves_every_replica_unwritten(red, norm, monkeypatch):
    made = []

    def like(t):
        made.append(t)
        if len(made) == R:
            raise torch.cuda.OutOfMemoryError("out of memory")
        return torch.empty_like(t)
    monkeypatch.setattr(layers, "_like", like)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        red.layer_norm_backward(1, 2, rows(), rows(), stats())
    assert red.calls == [] and norm()


@pytest.mark.parametrize("local", [False, True])
def test_a_pass_that_fails_half_way_leaves_gradients_that_are_not_averaged(red, norm, monkeypatch, local):
    if local:
        red.set_sync(False)
    real = layers._call
    runs = []

    def call(device, f, *args):
        runs.append(f)
        if len(runs) == 2:
            raise D.DdpbError(D.E_HIP, "launch")
        return real(device, f, *args)
    monkeypatch.setattr(layers, "_call", call)
    assert norm()
    with pytest.raises(D.DdpbError):
        red.embedding_backward(0, rows(), tokens())
    assert not norm()
    red.set_sync(True)
    red.embedding_backward(0, rows(), tokens())            # written anew, no hook has run
    red.layer_norm_backward(1, 2, rows(), rows(), stats())
    red.finalize()
    assert norm()


def test_begin_writes(red, norm):
    lib = red.lib
    for vs, code in (([0, 3], D.E_INDEX), ([-1], D.E_INDEX)):
        with pytest.raises(D.DdpbError) as e:
            lib.begin_writes(red.h, vs)
        assert e.value.code == code and norm()
    lib.begin_writes(red.h, [])
    assert norm()
    red.mark_ready(1)
    with pytest.raises(D.DdpbError) as e:
        lib.begin_writes(red.h, [0, 1])
    assert e.value.code == D.E_DOUBLE_READY
    red.mark_ready_many([0, 2])
    red.finalize()
    assert norm()
    lib.begin_writes(red.h, [0, 1, 2])
    assert not norm()
    assert lib.dll.ddpb_begin_writes(None, None, 0) == D.E_ARG
    assert lib.dll.ddpb_begin_writes(red.h, None, 1) == D.E_ARG
    assert lib.dll.ddpb_begin_writes(red.h, None, -1) == D.E_ARG


def test_the_checks_are_those_of_the_calls(red):
    from test_host_layers import LOOK_B, NORM_B
    lib = red.lib
    for name, args, bad in (("layer_norm_backward_check", NORM_B, {"dh": NORM_B["dy"]}),
                            ("embedding_backward_check", LOOK_B, {"workspace": 0})):
        f = getattr(lib, name)
        f(*list(args.values())[:-1])
        for change in (bad, {"dtype": 9}):
            with pytest.raises(D.DdpbError) as e:
                f(*list({**args, **change}.values())[:-1])
            assert e.value.code == D.E_ARG
