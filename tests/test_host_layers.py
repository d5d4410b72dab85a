"""Refusals, workspaces and state checks of layer norm, dropout and the embedding
through the host-only library (nothing is enqueued; addresses are made up), and
the Python front end's own refusals."""
import ctypes as C

import pytest
import torch

import ddp_bucketed_gradient_amd as D
from ddp_bucketed_gradient_amd import _abi

A = [1 << 40, 2 << 40, 3 << 40, 4 << 40, 5 << 40, 6 << 40, 7 << 40, 8 << 40]   # far apart, aligned


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(D.HOSTONLY_LIB):
        from ddp_bucketed_gradient_amd import build
        build.build_hostonly()
    return _abi.Lib(D.HOSTONLY_LIB)


def drop(p=0.1, at=0):
    return _abi.DropStruct(p, 1, 2, at)


NORM = dict(rows=4, cols=8, dtype=D.F32, x=A[0], x_stride=8, residual=0, residual_stride=0, drop=None, weight=A[1],
            bias=A[2], weight_dtype=D.F32, eps=1e-5, y=A[3], h=0, stats=A[4], stream=0)
NORM_B = dict(rows=400, cols=8, dtype=D.F32, dy=A[0], dy_stride=8, h=A[1], h_stride=8, stats=A[2], grad_h=0,
              grad_h_stride=0, drop=None, weight=A[3], weight_dtype=D.F32, dh=A[4], dx=0, dweight=A[5], dbias=A[6],
              grad_dtype=D.F32, accumulate=False, workspace=A[7], ws_bytes=1 << 30, stream=0)
DROP = dict(rows=4, cols=8, dtype=D.F32, x=A[0], x_stride=8, residual=0, residual_stride=0, drop=drop(), y=A[1], stream=0)
LOOK = dict(n=4, tokens=A[0], token_bytes=8, vocab=10, cols=8, table=A[1], table_dtype=D.F32, scale=1.0, residual=0,
            residual_stride=0, y=A[2], dtype=D.F32, stream=0)
LOOK_B = dict(n=4, tokens=A[0], token_bytes=8, vocab=10, cols=8, dy=A[1], dy_stride=8, dtype=D.F32, scale=1.0,
              dtable=A[2], grad_dtype=D.F32, accumulate=False, workspace=A[3], ws_bytes=1 << 30, stream=0)
CALLS = {"layer_norm": NORM, "layer_norm_backward": NORM_B, "dropout": DROP, "embedding": LOOK,
         "embedding_backward": LOOK_B}


@pytest.mark.parametrize("name, change", [
    (n, c) for n in CALLS for c in [{}, {"dtype": D.BF16}, {"dtype": D.F16}]] + [
    ("layer_norm", {"rows": 0, "x": 0, "y": 0, "stats": 0}),
    ("layer_norm", {"weight": 0, "bias": 0}),
    ("layer_norm", {"residual": A[5], "residual_stride": 0, "h": A[6]}),     # one row for all
    ("layer_norm", {"drop": drop(), "h": A[6]}),
    ("layer_norm", {"drop": drop(0.0)}),
    ("layer_norm", {"drop": drop(1.0)}),
    ("layer_norm", {"cols": 1 << 20, "x_stride": 1 << 20}),
    ("layer_norm", {"rows": 1, "x_stride": -5}),                             # no second row
    ("layer_norm", {"residual": A[0], "residual_stride": 8}),                # inputs may coincide
    ("layer_norm_backward", {"dweight": 0, "dbias": 0, "workspace": 0, "ws_bytes": 0}),
    ("layer_norm_backward", {"drop": drop(), "dx": A[7] + (1 << 38)}),
    ("layer_norm_backward", {"rows": 100, "workspace": 0, "ws_bytes": 0}),
    ("layer_norm_backward", {"rows": 0, "dy": 0, "h": 0, "stats": 0, "dh": 0}),
    ("dropout", {"y": A[0]}),                                                # in place
    ("dropout", {"residual": A[1], "residual_stride": 8}),                   # onto the residual
    ("dropout", {"rows": 0}), ("dropout", {"cols": 0}),
    ("embedding", {"n": 0, "tokens": 0, "y": 0}),
    ("embedding", {"vocab": 0, "table": 0}),
    ("embedding", {"token_bytes": 4, "tokens": A[0] + 4}),
    ("embedding_backward", {"n": 0, "tokens": 0, "dy": 0}),
    ("embedding_backward", {"vocab": 0, "dtable": 0}),
])
def test_accepted(lib, name, change):
    getattr(lib, name)(*{**CALLS[name], **change}.values())


@pytest.mark.parametrize("name, change, why", [
    (n, {"dtype": 7}, "dtype") for n in CALLS] + [
    ("layer_norm", {"weight_dtype": 3}, "dtype"),
    ("layer_norm", {"rows": -1}, "rows"),
    ("layer_norm", {"rows": 1 << 31}, "rows"),
    ("layer_norm", {"cols": 0}, "cols"),
    ("layer_norm", {"cols": (1 << 20) + 1}, "cols"),
    ("layer_norm", {"eps": -1e-9}, "eps"),
    ("layer_norm", {"eps": float("nan")}, "eps"),
    ("layer_norm", {"eps": 1e300}, "eps"),
    ("layer_norm", {"x": 0}, "NULL"),
    ("layer_norm", {"x": A[0] + 2}, "misaligned"),
    ("layer_norm", {"x_stride": -8}, "input"),
    ("layer_norm", {"x_stride": 1 << 60}, "spread"),
    ("layer_norm", {"y": 0}, "NULL"),
    ("layer_norm", {"stats": 0}, "NULL"),
    ("layer_norm", {"h": A[6]}, "pass NULL"),
    ("layer_norm", {"drop": drop(0.0), "h": A[6]}, "pass NULL"),
    ("layer_norm", {"weight": A[1] + 1}, "misaligned"),
    ("layer_norm", {"y": A[0]}, "overlap"),
    ("layer_norm", {"y": A[0] + 4 * 31}, "overlap"),                         # the last element
    ("layer_norm", {"stats": A[3]}, "overlap"),
    ("layer_norm", {"y": A[1] + 16}, "overlap"),
    ("layer_norm", {"drop": drop(1.5)}, "p must"),
    ("layer_norm", {"drop": drop(float("nan"))}, "p must"),
    ("layer_norm", {"drop": drop(0.1, 4)}, "offset"),
    ("layer_norm_backward", {"grad_dtype": -1}, "dtype"),
    ("layer_norm_backward", {"ws_bytes": 63}, "workspace"),
    ("layer_norm_backward", {"workspace": 0}, "workspace"),
    ("layer_norm_backward", {"workspace": A[7] + 128}, "workspace"),
    ("layer_norm_backward", {"dh": A[0]}, "overlap"),
    ("layer_norm_backward", {"dh": A[1]}, "overlap"),
    ("layer_norm_backward", {"dweight": A[6]}, "overlap"),
    ("layer_norm_backward", {"workspace": A[4]}, "overlap"),
    ("layer_norm_backward", {"drop": drop()}, "dx goes"),
    ("layer_norm_backward", {"dx": A[7] + (1 << 38)}, "dx goes"),
    ("layer_norm_backward", {"stats": 0}, "NULL"),
    ("layer_norm_backward", {"grad_h": A[4], "grad_h_stride": 8}, "overlap"),
    ("dropout", {"drop": None}, "drop is NULL"),
    ("dropout", {"y": A[0] + 4}, "overlap"),
    ("dropout", {"x_stride": 9, "y": A[0]}, "overlap"),                      # in place needs the same rows
    ("dropout", {"rows": 1 << 30, "cols": 1 << 30}, "2.40"),
    ("dropout", {"rows": 2, "cols": (1 << 33) + 8, "x_stride": (1 << 33) + 9, "y": A[7]}, "contiguous"),
    ("dropout", {"x": 0}, "NULL"),
    ("embedding", {"token_bytes": 2}, "token_bytes"),
    ("embedding", {"tokens": A[0] + 4}, "misaligned"),
    ("embedding", {"n": (1 << 30) + 1}, "2.30"),
    ("embedding", {"vocab": (1 << 31) - 1}, "2.31"),
    ("embedding", {"cols": 0}, "2.20"),
    ("embedding_backward", {"cols": (1 << 20) + 1}, "2.20"),
    ("embedding", {"scale": float("inf")}, "scale"),
    ("embedding", {"scale": 1e39}, "scale"),
    ("embedding", {"y": A[1] + 8}, "overlap"),
    ("embedding", {"table": 0}, "NULL"),
    ("embedding_backward", {"scale": float("nan")}, "scale"),
    ("embedding_backward", {"workspace": 0}, "workspace"),
    ("embedding_backward", {"ws_bytes": 256}, "workspace"),
    ("embedding_backward", {"dtable": A[1] + 4}, "overlap"),
    ("embedding_backward", {"dtable": 0}, "NULL"),
    ("embedding_backward", {"workspace": A[2] + 256}, "overlap"),
])
def test_refused(lib, name, change, why):
    with pytest.raises(D.DdpbError) as e:
        getattr(lib, name)(*{**CALLS[name], **change}.values())
    assert e.value.code == D.E_ARG
    import re
    assert re.search(why, str(e.value)), str(e.value)


@pytest.mark.parametrize("f, args", [("layer_norm_backward_workspace_bytes", a) for a in
                                     [(-1, 4), (1 << 31, 4), (4, 0), (4, (1 << 20) + 1)]] +
                         [("embedding_backward_workspace_bytes", a) for a in
                          [(-1, 4, 4), ((1 << 30) + 1, 4, 1), (4, -1, 4), (4, 4, 0), (1 << 30, 4, 1 << 11)]])
def test_workspace_sizes_refused(lib, f, args):
    with pytest.raises(D.DdpbError) as e:
        getattr(lib, f)(*args)
    assert e.value.code == D.E_ARG


def test_workspaces_stay_in_bounds(lib):
    for rows, cols in [(16384, 1024), ((1 << 31) - 1, 1), (5, 1 << 20), (33, 1024), (129, 128), (5, 2048)]:
        b = lib.layer_norm_backward_workspace_bytes(rows, cols)
        assert 2 * cols * 4 <= b <= 1 << 28 and b % 256 == 0
    for rows, cols in [(0, 1), (0, 1 << 20), (1, 1), (32, 1024), (128, 128), (4, 16384)]:     # one workgroup
        assert lib.layer_norm_backward_workspace_bytes(rows, cols) == 0
    for n, vocab, cols in [(0, 0, 1), (1, 1, 1), (16384, 30522, 1024), (1 << 30, (1 << 31) - 2, 1), (1 << 16, 5, 1 << 20)]:
        b = lib.embedding_backward_workspace_bytes(n, vocab, cols)
        # keys and order twice; histograms of at most 1024 counters for 4096 keys; two partial sums for each unit of
        # 8 or more places, of which there are at most 65536
        units = min(n // 8 + 1, 65536)
        assert 16 * n <= b <= 16 * n + (n // 4096 + 1) * 4096 + units * (8 * cols + 8) + 32768 and b % 256 == 0


def test_null_results(lib):
    assert lib.dll.ddpb_layer_norm_backward_workspace_bytes(4, 4, None) == D.E_ARG
    assert lib.dll.ddpb_embedding_backward_workspace_bytes(4, 4, 4, None) == D.E_ARG
    assert lib.dll.ddpb_check_writable(None, 0) == D.E_ARG


def test_check_writable_follows_the_reducers_state(lib):
    red = D.Reducer([(4, 3), (3,), (3,)], 2, 0, lib=lib)

    def code(v):
        try:
            red.lib.check_writable(red.h, v)
        except D.DdpbError as e:
            return e.code
        return D.OK
    assert code(0) == D.E_STATE                       # not bound
    red.bind_ptrs([A[i % 8] + (i << 20) for i in range(6)])
    assert [code(v) for v in (0, 1, 2, 3, -1)] == [D.OK] * 3 + [D.E_INDEX] * 2
    red.mark_ready(2)
    assert [code(v) for v in (0, 1, 2)] == [D.OK, D.OK, D.E_DOUBLE_READY]
    with pytest.raises(D.DdpbError):
        red.ensure_prior_reduction_finished()
    assert code(0) == D.E_INCOMPLETE
    red.reset()
    red.set_local_used([[True, False, False], [False, False, True]])
    assert [code(v) for v in (0, 1, 2)] == [D.OK, D.E_STATE, D.OK]
    red.mark_ready_many([2, 0])
    red.finalize()
    assert [code(v) for v in (0, 1, 2)] == [D.OK] * 3
    red.set_sync(False)
    red.mark_ready(1)
    red.mark_ready(1)
    assert code(1) == D.OK                            # local steps may write again
    red.set_sync(True)
    red.lib.set_sync_step(red.h, [A[7]] * 6, D.F32, True)
    assert code(1) == D.E_STATE
    red.close()


# ---- the front end --------------------------------------------------------------

def test_drop_refuses():
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError):
            D.Drop(p, 0)
    with pytest.raises(ValueError):
        D.Drop(0.1, 0, counter=torch.zeros(1, dtype=torch.int64))     # not on a GPU
    with pytest.raises(ValueError):
        D.Drop(0.1, 0, counter=3)


def test_drop_is_marshalled():
    d = D.Drop(0.25, -1, 1 << 64)
    assert (d._c.p, d._c.seed, d._c.offset, d._c.offset_device) == (0.25, (1 << 64) - 1, 0, None)
    assert d.active and not D.Drop(0.0, 1).active and not D.Drop(2.0 ** -18, 1).active and D.Drop(2.0 ** -17, 1).active
    assert C.sizeof(_abi.DropStruct) == 32


def test_cpu_tensors_are_refused():
    x, t = torch.zeros(2, 4), torch.zeros(3, dtype=torch.int64)
    d = D.Drop(0.1, 1)
    for f in (lambda: D.dropout(x, d), lambda: D.layer_norm(x), lambda: D.layer_norm_backward(x, x, torch.zeros(2, 2)),
              lambda: D.embedding(t, x), lambda: D.embedding_backward(torch.zeros(3, 4), t, x)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: D.dropout(x.double(), d), lambda: D.layer_norm(x.long())):
        with pytest.raises(ValueError, match="fp32, bf16 or fp16"):
            f()


class Fake:
    """What _rows reads of a CUDA tensor."""
    is_cuda, dtype, device = True, torch.float32, "cuda:0"

    def __init__(self, t):
        self.t = t
        self.shape = t.shape

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("make, want", [
    (lambda: torch.zeros(5), (1, 5, 5)),
    (lambda: torch.zeros(2, 3, 5), (6, 5, 5)),
    (lambda: torch.zeros(0, 5), (0, 5, 5)),
    (lambda: torch.zeros(3, 0), (3, 0, 0)),
    (lambda: torch.zeros(6, 9)[:, 2:7], (6, 5, 9)),
    (lambda: torch.zeros(2, 3, 9)[..., :5], (6, 5, 9)),
    (lambda: torch.zeros(6, 9)[::2, :5], (3, 5, 18)),
    (lambda: torch.zeros(4, 1, 9)[..., :5], (4, 5, 9)),
    (lambda: torch.zeros(1, 5).expand(4, 5), (4, 5, 0)),
    (lambda: torch.zeros(4, 9)[:, :1], (4, 1, 9)),
    (lambda: torch.zeros(9, 4).t()[:, :1], (4, 1, 1)),
    (lambda: torch.zeros(2, 3, 9)[:, :2, :5], None),             # two distances
    (lambda: torch.zeros(5, 4).t(), None),                       # elements of a row apart
    (lambda: torch.zeros(1).expand(4, 5), None),
    (lambda: torch.zeros(()), None),
])
def test_rows_of_a_tensor(make, want):
    from ddp_bucketed_gradient_amd.layers import _rows
    if want is None:
        with pytest.raises(ValueError):
            _rows(Fake(make()), "x")
    else:
        assert _rows(Fake(make()), "x") == want


def test_where_nothing_is_dropped_or_added_x_itself_is_returned():
    """No copy of rows that are cut out of a wider tensor either, in both directions."""
    for x in (torch.zeros(4, 6), torch.zeros(4, 9)[:, :6], torch.zeros(9, 4).t()):
        f = Fake(x)
        assert D.dropout(f, D.Drop(0.0, 1)) is f and D.dropout_backward(f, D.Drop(2.0 ** -18, 1)) is f
    double = Fake(torch.zeros(4, 6))
    double.dtype = torch.float64
    for x in (torch.zeros(4, 6), double):
        with pytest.raises(ValueError):
            D.dropout(x, D.Drop(0.0, 1))


def test_dropouts_used_as_documented_never_share_a_mask():
    """The offset that the documentation gives a place, plus the step's counter, over
    places and steps; and that the masks of such sums differ."""
    import os
    import re

    from oracle import layers as OL
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(here, "README.md")) as f:
        texts = [f.read(), D.Drop.__doc__]
    for text in texts:
        forms = re.findall(r"Drop\([^()]*offset=([^,()]+),\s*counter=step\)", text)
        assert forms
        for form in forms:
            steps = (0, 1, 2, 3, 19, 1 << 20, (1 << 32) - 1)
            at = [eval(form, {"site": site}) + step for site in range(20) for step in steps]
            assert len(set(at)) == len(at)
    masks = {tuple(OL.random16(0, 64, 1, (site << 32) + step) < 6554) for site in range(8) for step in range(8)}
    assert len(masks) == 64


def test_a_drop_is_active_where_the_library_drops(lib):
    """p * 65536 just below 1/2 rounds to 0, of which adding 1/2 makes 1."""
    import math
    for p in (0.5 / 65536, math.nextafter(0.5, 0) / 65536, math.nextafter(0.5, 1) / 65536, 0.0, 5e-324, 1.0):
        d = D.Drop(p, 1)
        args = {**NORM, "drop": d._c, "h": A[6]}       # h is x where nothing is dropped, and then refused
        try:
            lib.layer_norm(*args.values())
            dropped = True
        except D.DdpbError as e:
            assert "pass NULL" in str(e)
            dropped = False
        assert d.active == dropped == (p * 65536 >= 0.5)


def test_workspace_of_many_tiles_stays_in_bounds(lib):
    """Histograms of up to 1024 counters of four bytes for 2048 keys."""
    for n, vocab, cols in [(1 << 20, 1000, 1), (1 << 30, 1000, 1), (1 << 20, 1 << 19, 3), (1 << 24, 1000, 64),
                           (16385, 1023, 9)]:
        b = lib.embedding_backward_workspace_bytes(n, vocab, cols)
        units = min(n // 8 + 1, 65536)
        assert 16 * n <= b <= 16 * n + (n // 2048 + 1) * 4096 + units * (8 * cols + 8) + 32768 and b % 256 == 0
    # the histogram's term is needed: 512 tiles of 1024 counters
    assert lib.embedding_backward_workspace_bytes(1 << 20, 1000, 1) > (16 << 20) + (512 << 12)


@pytest.mark.parametrize("rows, cols", [(1 << 62, 4), (4, 1 << 62), ((1 << 63) - 1, (1 << 63) - 1), (-(1 << 63), 2)])
def test_sizes_whose_product_does_not_fit_are_refused(lib, rows, cols):
    for name in ("layer_norm", "layer_norm_backward", "dropout"):
        with pytest.raises(D.DdpbError) as e:
            getattr(lib, name)(*{**CALLS[name], "rows": rows, "cols": cols}.values())
        assert e.value.code == D.E_ARG
    for name in ("embedding", "embedding_backward"):
        with pytest.raises(D.DdpbError) as e:
            getattr(lib, name)(*{**CALLS[name], "n": rows, "cols": cols}.values())
        assert e.value.code == D.E_ARG
