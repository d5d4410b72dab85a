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
