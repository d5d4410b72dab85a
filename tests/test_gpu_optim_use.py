"""What a program around the AdamW step relies on: tensors let go while a step is
in flight.
"""
import pytest
import torch

import ddp_bucketed_gradient_amd as D
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_memory_let_go_behind_a_step_is_not_reused_before_it(state):
    """Parameters, gradients and states of the current stream, a step on a busy
    side stream, everything let go: what is allocated next keeps its values."""
    n, side = 3 << 20, torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    codes = lambda k, dt: torch.zeros(k, dtype=torch.uint8, device="cuda").view(dt)  # noqa: E731
    p, g = [torch.ones(n, device="cuda")], [torch.ones(n, device="cuda")]
    states = {"exp_avg": [torch.zeros(n, device="cuda")], "exp_avg_sq": [torch.zeros(n, device="cuda")]} \
        if state == "f32" else \
        {"exp_avg": [codes(n, torch.float8_e4m3fn)], "exp_avg_root": [codes(n, torch.float8_e4m3fn)],
         "avg_scale": [codes(n // 64, torch.float8_e8m0fnu)], "root_scale": [codes(n // 64, torch.float8_e8m0fnu)]}
    opt = D.AdamW(p, g, lr=0.5, state=state, states=states, stream=side)
    norm = D.GradNorm(g, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            x = x @ x * 1e-3                              # keeps the side stream busy
    norm.compute()
    opt.step()
    opt.close()
    del opt, norm, p, g, states
    new = [torch.full((n,), 7.0, device="cuda") for _ in range(6)] + \
          [torch.full((k,), 7, dtype=torch.uint8, device="cuda") for k in (n, n, n // 64, n // 64)]
    torch.cuda.synchronize()
    assert all((t == 7).all().item() for t in new)
