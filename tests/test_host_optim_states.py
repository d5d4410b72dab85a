"""When the norm and the AdamW step refuse, on the CPU: values that fp32 cannot
hold, and states of a reducer in which its gradients are not the averaged
ones. The host-only build enqueues nothing."""
import pytest

import ddp_bucketed_gradient_amd as D
from test_host_optim import GOOD, _bind_args, _code, host  # noqa: F401


def test_grad_scale_has_to_be_finite_in_fp32(host):  # noqa: F811
    """The step multiplies in fp32: 1e39 would be an infinite factor."""
    a = host.adamw_create(**GOOD)
    host.adamw_bind(a, **_bind_args())
    for sc in (1e39, -1e39, 1e300):
        assert _code(lambda: host.adamw_step(a, 1e-3, 0, sc)) == D.E_ARG
    host.adamw_step(a, 1e-3, 0, 3e38)
    host.adamw_step(a, 1e-3, 0, 1e-300)
    host.adamw_destroy(a)


# ---- with a reducer -----------------------------------------------------------------

STEPS = [[0x900000 + 0x10000 * i for i in range(6)]]


class Bound:
    """A reducer of 2 replicas x 3 variables with a norm and a step on it."""

    def __init__(self, host):  # noqa: F811
        self.lib, self.red = host, D.Reducer([(10,), (0,), (5000,)], 2, 0, lib=host)
        self.bind()
        self.n = host.norm_create([10, 0, 5000], [D.F32] * 3)
        self.a = host.adamw_create(**GOOD)
        self.handles()

    def bind(self):
        self.red.bind_ptrs([0x1000 + 16 * i for i in range(6)], side_streams=[0])

    def handles(self):
        self.lib.norm_bind(self.n, [0x10000, 0, 0x20000], 0x100, self.lib.norm_workspace_bytes(self.n), 0, self.red.h)
        self.lib.adamw_bind(self.a, **_bind_args(), reducer=self.red.h)

    def codes(self):
        out = []
        for f in (lambda: self.lib.norm_compute(self.n, 1.0, reducer=self.red.h),
                  lambda: self.lib.adamw_step(self.a, 1e-3, reducer=self.red.h)):
            try:
                f()
                out.append(D.OK)
            except D.DdpbError as e:
                out.append(e.code)
        assert out[0] == out[1]
        return out[0]

    def accumulate(self, first=True):
        self.lib.no_sync_accumulate(self.red.h, STEPS[0], D.F32, first)

    def set_step(self, first=True):
        self.lib.set_sync_step(self.red.h, STEPS[0], D.F32, first)

    def close(self):
        self.lib.norm_destroy(self.n)
        self.lib.adamw_destroy(self.a)
        self.red.close()


@pytest.fixture
def bound(host):  # noqa: F811
    b = Bound(host)
    yield b
    b.close()


def test_local_steps_are_not_averaged_gradients(bound):
    """After no_sync_accumulate the gradients hold replica sums until the next
    synchronisation, whatever the switch says."""
    assert bound.codes() == D.OK
    for switch in (False, True):
        if switch:
            bound.red.set_sync(False)
        bound.accumulate()
        assert bound.codes() == D.E_STATE
        bound.red.finalize() if switch else None              # nothing to do with the switch off
        assert bound.codes() == D.E_STATE
        bound.red.set_sync(True)
        assert bound.codes() == D.E_STATE
        bound.red.sync()
        assert bound.codes() == D.OK


def test_hooks_without_synchronisation(bound):
    """Switching off changes no gradient, a hook that fires then says that one
    was written; finalize reduces nothing."""
    bound.red.sync()
    bound.red.set_sync(False)
    assert bound.codes() == D.OK                              # the last synchronisation's gradients are still there
    bound.red.mark_ready(2)
    assert bound.codes() == D.E_STATE
    bound.red.finalize()
    assert bound.codes() == D.E_STATE
    bound.red.set_sync(True)
    assert bound.codes() == D.E_STATE
    bound.red.sync()
    assert bound.codes() == D.OK
    bound.red.set_sync(False)
    bound.red.mark_ready_many([0, 1])
    bound.red.set_sync(True)
    assert bound.codes() == D.E_STATE


def test_a_step_set_for_the_coming_synchronisation(bound):
    bound.red.sync()
    bound.set_step(first=False)
    assert bound.codes() == D.E_STATE                         # not in the gradients yet
    bound.red.sync()
    assert bound.codes() == D.OK
    bound.set_step()
    bound.red.reset()                                         # dropped, and nothing was written
    assert bound.codes() == D.OK


def test_an_iteration_that_failed_or_was_dropped(bound):
    """Some buckets may have been averaged, others not: reset clears the error,
    only a synchronisation makes the gradients averaged ones."""
    bound.red.mark_ready(2)
    with pytest.raises(D.DdpbError):
        bound.red.finalize()
    assert bound.codes() == D.E_INCOMPLETE
    bound.red.reset()
    assert bound.codes() == D.E_STATE
    bound.red.sync()
    assert bound.codes() == D.OK
    bound.red.mark_ready(2)
    bound.red.reset()                                         # abandoned
    assert bound.codes() == D.E_STATE
    bound.accumulate()
    bound.red.sync()
    assert bound.codes() == D.OK


def test_a_new_binding_starts_afresh(bound):
    bound.accumulate()
    assert bound.codes() == D.E_STATE
    bound.bind()                                              # other gradients, of which nothing is known
    bound.handles()
    assert bound.codes() == D.OK


def test_replays_of_a_captured_synchronisation(bound):
    """Local steps cannot be captured, the synchronisation that follows them can:
    the handle learns nothing of its replays, so that on a binding with a
    captured one written gradients may have been averaged since."""
    bound.lib.dll.ddpb_hostonly_set_capture(1)
    bound.red.sync()
    bound.lib.dll.ddpb_hostonly_set_capture(0)
    assert bound.codes() == D.OK
    bound.accumulate()
    bound.accumulate(first=False)
    assert bound.codes() == D.OK                              # behind a replay, for all the handle knows
    bound.red.mark_ready(2)
    assert bound.codes() == D.E_STATE                         # an iteration of its own it knows of
    bound.red.mark_ready_many([1, 0])
    bound.red.finalize()
    assert bound.codes() == D.OK
    bound.bind()
    bound.handles()
    bound.accumulate()
    assert bound.codes() == D.E_STATE                         # the graphs went with the binding


def test_one_replica_is_its_own_average(host):  # noqa: F811
    red = D.Reducer([(10,)], 1, 0, lib=host)
    red.bind_ptrs([0x1000], side_streams=[0])
    n = host.norm_create([10], [D.F32])
    host.norm_bind(n, [0x10000], 0x100, host.norm_workspace_bytes(n), 0, red.h)
    host.no_sync_accumulate(red.h, [0x2000], D.F32, True)
    host.norm_compute(n, 1.0, reducer=red.h)
    host.set_sync_step(red.h, [0x2000], D.F32, False)         # not in the gradient yet
    assert _code(lambda: host.norm_compute(n, 1.0, reducer=red.h)) == D.E_STATE
    red.sync()
    host.norm_compute(n, 1.0, reducer=red.h)
    host.norm_destroy(n)
    red.close()
