"""The norm's and AdamW's Python front end on the CPU, with stand-ins for
tensors and streams where a GPU would be needed."""
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
