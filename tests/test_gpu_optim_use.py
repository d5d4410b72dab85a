"""What a program around the AdamW step relies on: tensors let go while a step is
in flight, a handle made again from another's options, autograd's in-place check,
a rate in device memory, variables that were not used.
"""
import numpy as np
import pytest
import torch

import ddp_bucketed_gradient_amd as D
from gpu_util import require_gpu
from test_gpu_optim import Case, raw

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


@pytest.mark.parametrize("p,state,master", [("bf16", "f8", True), ("f32", "f8", False), ("f16", "f32", True)])
def test_options_make_a_handle_that_goes_on_bit_for_bit(p, state, master):
    """Another seed than 0, other betas, eps, decay and rate factors than the
    defaults: a handle made from ``options`` draws the same bits and takes the
    same steps."""
    n = len(Case(zero=True).numels)
    a, b = (Case(p, "f32", state, master, seed=91, step=9, random_seed=1234, betas=(0.8, 0.97), eps=1e-6, lr=3e-2,
                 weight_decay=[0.01 * v for v in range(n)], lr_scale=[1 + 0.1 * v for v in range(n)]) for _ in range(2))
    for rep in range(4):
        for c in (a, b):
            c.new_grads()
            c.opt.step()
        old = b.opt
        b.opt = D.AdamW(old.params[0], old.grads, step=old.steps_done, **old.options)
        assert b.opt.lr == 3e-2
        old.close()
    torch.cuda.synchronize()
    assert a.opt.steps_done == b.opt.steps_done == 13
    for k in a.stores:
        assert np.array_equal(a.stores[k].bytes.cpu().numpy(), b.stores[k].bytes.cpu().numpy()), k


def test_autograd_sees_the_step():
    """A backward that saved the old parameters is refused, as after an in-place
    operation of torch's own; every replica counts."""
    rows = [[torch.nn.Parameter(torch.ones(10, device="cuda"))] for _ in range(2)]
    opt = D.AdamW(rows, [torch.ones(10, device="cuda")])
    before = [r[0]._version for r in rows]
    losses = [(r[0] * r[0]).sum() for r in rows]
    opt.step()
    for r, b, loss in zip(rows, before, losses):
        assert r[0]._version > b
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    with torch.inference_mode():
        x = torch.ones(3, device="cuda")                  # has no counter
    D.AdamW([x], [torch.ones(3, device="cuda")], lr=0.125, weight_decay=0.0).step()
    assert (x < 1).all().item()


def test_a_rate_written_on_another_stream():
    """A rate that the busy current stream writes, a step on a side stream, the
    rate let go and its memory written again at once: the step takes the value
    that was written before it."""
    side = torch.cuda.Stream()
    a, b = (Case("f32", "f32", "f32", seed=93, stream=s) for s in (side, None))
    for c in (a, b):
        c.new_grads()
    x = torch.randn(4096, 4096, device="cuda")
    lr = torch.full((1,), 0.5, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        x = x @ x * 1e-3                                  # keeps the current stream busy
    lr.fill_(0.125)
    a.opt.step(lr=lr)
    del lr
    new = [torch.full((1,), 7.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    b.opt.step(lr=0.125)
    torch.cuda.synchronize()
    for k in a.stores:
        assert np.array_equal(a.stores[k].bytes.cpu().numpy(), b.stores[k].bytes.cpu().numpy()), k
    assert all(t.item() == 7.0 for t in new)


@pytest.mark.parametrize("view", [False, True])
def test_a_variable_that_no_replica_used_takes_the_step_as_it_stands(view):
    """Its gradient is what was there before the synchronisation (replica 0's),
    or zeros with bucket views."""
    shapes, R = [(100,), (70,), (300,)], 2
    red = D.Reducer(shapes, R, 4 * 200)
    grads = red.bind_bucket_views() if view else [[torch.empty(s, device="cuda") for s in shapes] for _ in range(R)]
    if not view:
        red.bind(grads)
    for r in range(R):
        for v, t in enumerate(grads[r]):
            t.fill_(1.0 + r + v)
    params = [torch.ones(s, device="cuda") for s in shapes]
    opt = red.adamw(params, lr=0.25, weight_decay=0.5, betas=(0.0, 0.0), eps=0.125)
    red.set_local_used([[True, False, True]] * R)
    red.sync([2, 0])
    opt.step()
    torch.cuda.synchronize()
    # with both betas 0: p (1 - lr wd) - lr g / (|g| + eps)
    for p, g in zip(params, (1.5, 0.0 if view else 2.0, 3.5)):
        want = 0.875 - 0.25 * g / (g + 0.125)
        # p's factor, product and difference (3 roundings of at most 1) and 13 of an update below lr
        assert (p.double() - want).abs().max().item() <= 2.0 ** -24 * (3 + 13 * 0.25)
    red.close()


def test_local_steps_then_a_replayed_synchronisation_then_a_step():
    """The synchronisation and the norm's and step's calls as a program mixes
    them: local steps eagerly, the synchronisation as a graph, the step eagerly;
    the same bits as with an eager synchronisation."""
    shapes, R = [(1000,), (70,), (5000,)], 2
    outs = []
    for graph in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(5)
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            grads = [[torch.zeros(s, device="cuda") for s in shapes] for _ in range(R)]
            steps = [[torch.zeros(s, device="cuda") for s in shapes] for _ in range(R)]
            params = [torch.ones(s, device="cuda") for s in shapes]
            red = D.Reducer(shapes, R, 4 * 3000)
            red.bind(grads, compute_stream=stream)
            opt, norm = red.adamw(params, lr=0.01), red.grad_norm()
            if graph:
                g = torch.cuda.CUDAGraph()
                stream.synchronize()
                with torch.cuda.graph(g, stream=stream):
                    red.sync()
            for _ in range(3):
                for first in (True, False):
                    for row in steps:
                        for t in row:
                            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
                    red.no_sync_accumulate(steps, first_step=first)
                g.replay() if graph else red.sync()
                norm.compute(max_norm=0.5)
                opt.step(clip=norm)
            stream.synchronize()
            outs.append([raw(t) for t in params + grads[0] + grads[1]])
        red.close()
    for a, b in zip(*outs):
        assert np.array_equal(a, b)
