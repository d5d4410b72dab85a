"""The norm's and AdamW's C ABI on the CPU: what create, bind and the calls
refuse, and the reducer states in which they refuse. The host-only build
enqueues nothing and reads none of the addresses."""
import os

import pytest

import ddp_bucketed_gradient_amd as D

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def host():
    if not os.path.exists(D.HOSTONLY_LIB):
        from ddp_bucketed_gradient_amd import build
        build.build_hostonly()
    return D.Lib(D.HOSTONLY_LIB)


def _code(call):
    with pytest.raises(D.DdpbError) as e:
        call()
    assert str(e.value) and str(e.value) != "E_ARG: "
    return e.value.code


# ---- norm ---------------------------------------------------------------------------

@pytest.mark.parametrize("numel,dtypes", [([-1], [0]), ([4], [3]), ([4], [-1]), ([1 << 41], [0]),
                                          ([1 << 40, 1], [0, 0])])
def test_norm_create_refusals(host, numel, dtypes):
    assert _code(lambda: host.norm_create(numel, dtypes)) == D.E_ARG


def _norm(host, numel=(10, 0, 5000), dtypes=(D.F32, D.BF16, D.F16)):
    n = host.norm_create(list(numel), list(dtypes))
    return n, host.norm_workspace_bytes(n)


GRADS = [0x10000, 0, 0x20000]


def test_norm_bind_and_compute(host):
    n, ws = _norm(host)
    assert ws >= 256
    assert _code(lambda: host.norm_compute(n, 1.0)) == D.E_STATE                       # not bound
    for bad in ([0x10002, 0, 0x20000], [0, 0, 0x20000], [0x10000, 0, 0x20001]):        # misaligned or NULL
        assert _code(lambda: host.norm_bind(n, bad, 0x100, ws, 0)) == D.E_ARG
    assert _code(lambda: host.norm_bind(n, GRADS, 0x100, ws - 1, 0)) == D.E_ARG        # workspace
    assert _code(lambda: host.norm_bind(n, GRADS, 0, ws, 0)) == D.E_ARG
    assert _code(lambda: host.norm_bind(n, GRADS, 0x140, ws, 0)) == D.E_ARG
    host.norm_bind(n, GRADS, 0x100, ws, 0)
    host.norm_compute(n, INF, -2.0)
    for mx, sc in ((0.0, 1.0), (-1.0, 1.0), (NAN, 1.0), (1.0, INF), (1.0, NAN)):
        assert _code(lambda: host.norm_compute(n, mx, sc)) == D.E_ARG
    assert _code(lambda: host.norm_compute(n, 1.0, 1.0, 2)) == D.E_ARG                 # flags
    host.norm_destroy(n)


def test_norm_of_nothing(host):
    n, ws = _norm(host, (), ())
    host.norm_bind(n, [], 0x100, ws, 0)
    host.norm_compute(n, 1.0)
    host.norm_destroy(n)


# ---- AdamW --------------------------------------------------------------------------

GOOD = dict(numel=[10, 0, 5000], R=2, param_dtype=D.F32, grad_dtype=D.F32, state=D.STATE_F32, flags=0, beta1=0.9,
            beta2=0.999, eps=1e-8, weight_decay=[0.0, 0.1, 0.2], lr_scale=None, seed=0)


@pytest.mark.parametrize("change", [
    dict(numel=[10, -1, 5]), dict(numel=[1 << 41, 0, 0]), dict(R=0), dict(R=65), dict(param_dtype=3), dict(grad_dtype=-1),
    dict(state=2), dict(flags=2), dict(flags=D.ADAMW_MASTER), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
    dict(beta2=NAN), dict(eps=-1e-8), dict(eps=INF), dict(eps=NAN), dict(weight_decay=[0, -0.1, 0]),
    dict(weight_decay=[0, INF, 0]), dict(lr_scale=[1, 1, NAN]), dict(lr_scale=[1, -1, 1])])
def test_adamw_create_refusals(host, change):
    assert _code(lambda: host.adamw_create(**{**GOOD, **change})) == D.E_ARG


def test_adamw_create_needs_one_value_for_each_variable(host):
    with pytest.raises(ValueError):
        host.adamw_create(**{**GOOD, "weight_decay": [0.1]})


def _at(k, n=3):
    """Addresses that do not overlap: 1 MiB for each array."""
    return [(k * 8 + i + 1) << 20 for i in range(n)]


def _bind_args(state=D.STATE_F32, master=False, R=2):
    f8 = state == D.STATE_F8
    return dict(params=_at(0) + (_at(1) if R == 2 else []), grads=_at(2), master=_at(3) if master else None,
                exp_avg=_at(4), second=_at(5), avg_scale=_at(6) if f8 else None, root_scale=_at(7) if f8 else None,
                step=0, workspace=1 << 30, ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("state", [D.STATE_F32, D.STATE_F8])
@pytest.mark.parametrize("pd,master", [(D.F32, False), (D.BF16, False), (D.F16, True)])
def test_adamw_bind_and_step(host, state, pd, master):
    a = host.adamw_create(**{**GOOD, "state": state, "param_dtype": pd, "flags": D.ADAMW_MASTER if master else 0})
    good = _bind_args(state, master)
    bind = lambda **kw: host.adamw_bind(a, **{**good, **kw})  # noqa: E731
    assert _code(lambda: host.adamw_step(a, 1e-3)) == D.E_STATE                        # not bound
    assert _code(lambda: host.adamw_set_step(a, 1)) == D.E_STATE
    assert _code(lambda: host.adamw_get_step(a)) == D.E_STATE
    for name in ("params", "grads", "exp_avg", "second") + (("master",) if master else ()) + (
            ("avg_scale", "root_scale") if state == D.STATE_F8 else ()):
        null = list(good[name])
        null[0] = 0
        assert _code(lambda: bind(**{name: null})) == D.E_ARG, name
        odd = list(good[name])
        odd[2] += 1
        byte = name.endswith("_scale") or (state == D.STATE_F8 and name in ("exp_avg", "second"))
        if not byte:                                                                   # bytes need no alignment
            assert _code(lambda: bind(**{name: odd})) == D.E_ARG, name
        assert _code(lambda: bind(**{name: None})) == D.E_ARG, name
    assert _code(lambda: bind(ws_bytes=host.adamw_workspace_bytes(a) - 1)) == D.E_ARG
    assert _code(lambda: bind(workspace=(1 << 30) + 64)) == D.E_ARG
    assert _code(lambda: bind(workspace=0)) == D.E_ARG
    for t in (-1, (1 << 53) + 1, (1 << 63) - 1):
        assert _code(lambda: bind(step=t)) == D.E_ARG
    empty = list(good["grads"])
    empty[1] = 0                                                                       # numel 0: may be NULL
    bind(grads=empty)
    host.adamw_step(a, 0.0)
    host.adamw_step(a, 1e-3, 0x1000, -0.5, 0x2000)
    for lr, sc in ((-1e-3, 1.0), (NAN, 1.0), (INF, 1.0), (1e-3, INF), (1e-3, NAN)):
        assert _code(lambda: host.adamw_step(a, lr, 0, sc)) == D.E_ARG
    assert _code(lambda: host.adamw_step(a, 1e-3, 0x1001)) == D.E_ARG
    assert _code(lambda: host.adamw_step(a, 1e-3, 0, 1.0, 0x2002)) == D.E_ARG
    for t in (-1, (1 << 53) + 1, (1 << 63) - 1):
        assert _code(lambda: host.adamw_set_step(a, t)) == D.E_ARG
    host.adamw_set_step(a, 1 << 53)
    host.adamw_destroy(a)


def test_memory_named_twice_is_refused(host):
    """Whatever a step writes has memory of its own; gradients, only read, may
    coincide with one another."""
    a = host.adamw_create(**{**GOOD, "numel": [1000, 1000, 1000], "state": D.STATE_F8})
    good = _bind_args(D.STATE_F8)
    bind = lambda **kw: host.adamw_bind(a, **{**good, **kw})  # noqa: E731
    tie = lambda xs, i, y: xs[:i] + [y] + xs[i + 1:]  # noqa: E731
    bind()
    bind(grads=[good["grads"][0]] * 3)
    p = good["params"]
    for kw in (dict(params=tie(p, 2, p[0])),                        # a tied parameter listed twice
               dict(params=tie(p, 3, p[0])),                        # a replica that is replica 0
               dict(params=tie(p, 1, p[0] + 3996)),                 # the last element of another
               dict(grads=tie(good["grads"], 1, p[4] + 100)),       # a gradient inside a parameter
               dict(exp_avg=tie(good["exp_avg"], 0, good["second"][0] + 999)),
               dict(avg_scale=tie(good["avg_scale"], 0, good["root_scale"][2] + 15)),
               dict(workspace=(p[0] // 256 - 1) * 256)):
        assert _code(lambda: bind(**kw)) == D.E_ARG, kw
    bind(params=tie(p, 1, p[0] + 4000), exp_avg=tie(good["exp_avg"], 0, good["second"][0] + 1000),
         avg_scale=tie(good["avg_scale"], 0, good["root_scale"][2] + 16))              # touching is fine
    host.adamw_destroy(a)


@pytest.mark.parametrize("state,pd,part,threads", [(D.STATE_F32, D.F32, 256, 64), (D.STATE_F8, D.F32, 1024, 256),
                                                   (D.STATE_F8, D.BF16, 2048, 256)])
def test_more_workgroups_than_one_launch_takes(host, state, pd, part, threads):
    """Fewer than 2^32 threads a launch, one workgroup for ``part`` elements or a
    variable's rest."""
    most = ((1 << 32) - 1) // threads
    for numel, ok in (([most * part], True), ([most * part + 1], False), ([1, (most - 1) * part], True),
                      ([1, (most - 1) * part + 1], False), ([1, 0, most * part], False)):
        a = host.adamw_create(**{**GOOD, "numel": numel, "weight_decay": None, "state": state, "param_dtype": pd})
        at = lambda k: [(k * 8 + i + 1) << 44 for i in range(len(numel))]  # noqa: E731
        sc = (at(5), at(6)) if state == D.STATE_F8 else (None, None)
        bind = lambda: host.adamw_bind(a, at(0) + at(1), at(2), None, at(3), at(4), *sc, 0, 1 << 30,  # noqa: E731
                                       1 << 29, 0)
        if ok:
            bind()
        else:
            assert _code(bind) == D.E_ARG
        host.adamw_destroy(a)


def test_adamw_of_nothing(host):
    a = host.adamw_create(**{**GOOD, "numel": [], "weight_decay": None})
    host.adamw_bind(a, [], [], None, [], [], None, None, 0, 1 << 30, 1 << 20, 0)
    host.adamw_step(a, 1e-3)
    host.adamw_destroy(a)


# ---- with a reducer -----------------------------------------------------------------

def test_calls_follow_the_reducers_state(host):
    red = D.Reducer([(10,), (0,), (5000,)], 2, 0, lib=host)
    n, ws = _norm(host, dtypes=(D.F32,) * 3)
    a = host.adamw_create(**GOOD)
    args = _bind_args()
    assert _code(lambda: host.norm_bind(n, GRADS, 0x100, ws, 0, red.h)) == D.E_STATE   # the reducer is unbound
    assert _code(lambda: host.adamw_bind(a, **args, reducer=red.h)) == D.E_STATE
    bind = lambda: red.bind_ptrs([0x1000 + 16 * i for i in range(6)], side_streams=[0])  # noqa: E731
    bind()
    host.norm_bind(n, GRADS, 0x100, ws, 0, red.h)
    host.adamw_bind(a, **args, reducer=red.h)
    both = (lambda: host.norm_compute(n, 1.0, reducer=red.h), lambda: host.adamw_step(a, 1e-3, reducer=red.h))
    for f in both:
        f()
    red.mark_ready(2)                                        # an iteration is open: gradients are not final
    for f in both:
        assert _code(f) == D.E_STATE
    with pytest.raises(D.DdpbError):
        red.finalize()                                       # incomplete: latched
    for f in both:
        assert _code(f) == D.E_INCOMPLETE
    red.reset()
    red.sync()
    for f in both:
        f()
    bind()                                                   # bound again: other gradients
    for f in both:
        assert _code(f) == D.E_STATE
    host.norm_bind(n, GRADS, 0x100, ws, 0, red.h)
    host.adamw_bind(a, **args, reducer=red.h)
    for f in both:
        f()
    red.sync()
    red.rebuild_buckets()                                    # unbound until the next bind
    for f in both:
        assert _code(f) == D.E_STATE
    host.norm_destroy(n)
    host.adamw_destroy(a)
    red.close()
