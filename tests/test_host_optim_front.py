"""The norm's and AdamW's Python front end on the CPU, with stand-ins for
tensors and streams where a GPU would be needed."""
import os

import pytest
import torch

import ddp_bucketed_gradient_amd as D


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a, **kw: self.calls.append((name, a))


class FakeTensor:
    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


def _handle(cls, **attrs):
    x = cls.__new__(cls)
    x.__dict__.update(lib=FakeLib(), h=object(), stream=object(), _reducer=None, _keep=None, **attrs)
    return x


def test_tensors_let_go_by_close_are_known_on_the_stream_that_uses_them():
    """Memory of a tensor that was allocated for another stream must not be
    handed out while a step that was enqueued before close() still uses it."""
    for cls, destroy in ((D.GradNorm, "norm_destroy"), (D.AdamW, "adamw_destroy")):
        for drop in (lambda x: x.close(), lambda x: x.__del__()):
            x, ts = _handle(cls), [FakeTensor() for _ in range(3)]
            x._keep = list(ts)
            drop(x)
            assert [c[0] for c in x.lib.calls] == [destroy]
            assert all(t.streams == [x.stream] for t in ts)
            x.close()                                    # once only
            assert all(len(t.streams) == 1 for t in ts) and len(x.lib.calls) == 1


class FakeStream:
    def __init__(self):
        self.waited = []

    def wait_stream(self, s):
        self.waited.append(s)


class FakeRate(torch.Tensor):
    is_cuda, device = True, "gpu"

    def record_stream(self, s):
        self.__dict__.setdefault("streams", []).append(s)


@pytest.mark.parametrize("elsewhere,capturing", [(False, False), (True, False), (True, True), (False, True)])
def test_a_rate_in_device_memory_is_read_behind_what_wrote_it(monkeypatch, elsewhere, capturing):
    """The step reads it on the handle's stream: behind what the current one has
    enqueued so far, and its memory stays. In a capture the caller has ordered
    the two streams (a wait would draw the handle's stream into the capture)."""
    own, other = FakeStream(), FakeStream()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: other if elsewhere else own)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    x = _handle(D.AdamW, device="gpu", _state={}, _written=[], _count_write=lambda ts: None)
    x.stream = own
    lr = torch.ones(1).as_subclass(FakeRate)
    x.step(lr=lr)
    assert x.lib.calls[-1][0] == "adamw_step" and x.lib.calls[-1][1][2] == lr.data_ptr()
    assert own.waited == ([other] if elsewhere and not capturing else [])
    assert lr.streams == [own]
    x.step(lr=1e-3)                                      # a number needs neither
    assert own.waited == ([other] if elsewhere and not capturing else []) and lr.streams == [own]


def test_a_reducer_without_a_stream_is_refused():
    """Unbound, or bound to raw addresses only: no stream to run on is known."""
    if not os.path.exists(D.HOSTONLY_LIB):
        from ddp_bucketed_gradient_amd import build
        build.build_hostonly()
    red = D.Reducer([(10,)], 2, 0, lib=D.Lib(D.HOSTONLY_LIB))
    for bind in (lambda: None, lambda: red.bind_ptrs([0x1000, 0x2000])):
        bind()
        x = _handle(D.GradNorm)
        with pytest.raises(D.DdpbError) as e:
            x._open(x.lib, x.h, torch.device("cuda", 0), None, red)
        assert e.value.code == D.E_STATE
    red.close()
