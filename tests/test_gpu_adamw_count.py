"""AdamW whose number of updates is counted on the GPU: a step that the
clip factor skips there is no update, and a captured step counts its replays.

Against the host's count: the moments do not depend on it, so they are equal
to the bit.  The bias factors come from another power function, good to a few
units of fp64, so that each may round to the neighbouring fp32 value (2 u, u =
2^-24).  In the update term m / (sqrt(v) c + eps) * r that is 2 u for r, 2 u
for c, and 2 u for each of the two roundings between, of the sum and of the
quotient, which may fall the other way: 8 u of the term; the parameter's own
rounding is 2 u of it."""
import math
import os
import sys

import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=0.02, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SHAPES = [(33, 65), (7,), (9001,), (0,), (64, 64)]


def states(n, seed=91, grad=torch.bfloat16):
    """n equal sets of {params, grads, exp_avgs, exp_avg_sqs} on the GPU."""
    rng = np.random.default_rng(seed)

    def arrays(scale, dtype=torch.float32):
        return [torch.from_numpy(np.asarray(rng.normal(size=s) * scale)).to(dtype) for s in SHAPES]

    one = [arrays(1.0), arrays(0.5, grad), arrays(0.1), [t.square() for t in arrays(0.1)]]
    return [[[t.cuda() for t in a] for a in one] for _ in range(n)]


def counter(value=0):
    return torch.tensor([value], dtype=torch.int64, device="cuda")


def equal(a, b):
    return all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


@pytest.mark.parametrize("first", [1, 2, 1000, 10 ** 7])
def test_counts_like_the_host(first):
    gns = need_gpu()
    a, b = states(2)
    la, lb, count = gns.adamw_list(*a), gns.adamw_list(*b), counter(first - 1)
    for t in range(first, first + 4):
        say("counted", t)
        for x, y in zip(a, b):                          # the step before may have differed by its rounding
            for u, v in zip(x, y):
                u.copy_(v)
        before = [p.clone() for p in b[0]]
        gns.adamw_step(la, t, **HYPER)
        gns.adamw_step(lb, count=count, **HYPER)
        assert int(count) == t
        assert equal(a[1:], b[1:])
        for p, q, old in zip(a[0], b[0], before):
            term = (p.double() - old.double() * (1 - HYPER["lr"] * HYPER["weight_decay"])).abs()
            assert bool(((p.double() - q.double()).abs() <= 8 * U * term + 2 * U * p.double().abs()).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_skipped_steps_are_not_counted(bad):
    gns = need_gpu()
    a, b = states(2)
    la, lb, ca, cb = gns.adamw_list(*a), gns.adamw_list(*b), counter(), counter()
    ok, skip = torch.tensor(0.5, device="cuda"), torch.tensor(bad, device="cuda")
    say("skipped steps", bad)
    for i in range(4):
        gns.adamw_step(la, count=ca, grad_scale=ok, **HYPER)
        if i != 1:
            gns.adamw_step(lb, count=cb, grad_scale=skip, **HYPER)
            assert int(cb) == i
        gns.adamw_step(lb, count=cb, grad_scale=ok, **HYPER)
        assert int(ca) == int(cb) == i + 1 and equal(a, b)


def test_replays_are_further_updates():
    """A captured norm and update, replayed without a reset: each replay is
    the eager step that follows, with gradients of its own, one of them not
    finite; eager work and synchronisation between."""
    gns = need_gpu()
    a, b = states(2, grad=torch.float32)
    la, lb, ca, cb = gns.adamw_list(*a), gns.adamw_list(*b), counter(5), counter(5)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def step(lst, count):
        got = gns.grad_norm(lst, max_norm=3.0)
        gns.adamw_step(lst, count=count, grad_scale=got.clip, **HYPER)
        return got

    torch.cuda.synchronize()
    say("replays: capture")
    with torch.cuda.graph(graph, stream=stream):
        captured = step(la, ca)
    assert int(ca) == 5
    gen = torch.Generator(device="cuda").manual_seed(92)
    for rep in range(6):
        for g, h in zip(a[1], b[1]):
            g.normal_(0, 0.5, generator=gen)
            h.copy_(g)
        if rep == 2:
            a[1][2][4000] = b[1][2][4000] = math.nan
        say("replays:", rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = step(lb, cb)
        torch.cuda.synchronize()
        assert equal(a[:1], b[:1]) and equal(a[2:], b[2:]) and int(ca) == int(cb) == 6 + rep - (rep >= 2)
        assert torch.equal(captured.result.view(torch.int32), eager.result.view(torch.int32))


def test_other_stream_and_empty_list():
    gns = need_gpu()
    a, b = states(2)
    la, lb, ca, cb = gns.adamw_list(*a), gns.adamw_list(*b), counter(), counter()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("counted on another stream")
    for stream in (side, side.cuda_stream):
        gns.adamw_step(la, count=ca, stream=stream, **HYPER)
        gns.adamw_step(lb, count=cb, **HYPER)
    side.synchronize()
    assert int(ca) == int(cb) == 2 and equal(a, b)
    gns.adamw_step(gns.adamw_list([], [], [], []), count=ca, **HYPER)
    assert int(ca) == 3


def test_count_refusals():
    gns = need_gpu()
    state = states(1)[0]
    lst, kept = gns.adamw_list(*state), [[t.clone() for t in a] for a in state]
    for kw, name in (({"count": counter().int()}, "GNS_E_DTYPE"),
                     ({"count": torch.zeros(2, dtype=torch.int64, device="cuda")}, "GNS_E_DTYPE"),
                     ({"count": torch.zeros(1, dtype=torch.int64)}, "GNS_E_NULL"), ({}, "GNS_E_PARAM"),
                     ({"step": 1, "count": counter()}, "GNS_E_PARAM"), ({"step": 0}, "GNS_E_PARAM")):
        with pytest.raises(gns.GnsError) as e:
            gns.adamw_step(lst, **kw, **HYPER)
        assert e.value.name == name, kw
    assert equal(state, kept)


def test_smallest_eps():
    """Zero moments and no gradient leave 0 / eps = 0, with the smallest eps
    that is accepted."""
    gns = need_gpu()
    p, z = torch.full((70,), 2.0, device="cuda"), [torch.zeros(70, device="cuda") for _ in range(3)]
    gns.adamw_step(gns.adamw_list([p], z[:1], z[1:2], z[2:]), 1, lr=0.1, eps=2.0 ** -149, weight_decay=0.0)
    assert bool((p == 2.0).all())


def test_example_goes_on_after_a_skipped_step_as_if_it_had_not_been():
    need_gpu()
    import train_step

    def trained(with_nan):
        trainer = train_step.Trainer(train_step.Model(torch.Generator().manual_seed(1)).cuda())
        gen = torch.Generator(device="cuda").manual_seed(2)
        for i in range(4):
            trainer.G.normal_(0, 1e-3, generator=gen)
            trainer.flat_rest.normal_(0, 1e-3, generator=gen)
            trainer.step()
            if with_nan and i in (0, 2):
                trainer.G[3, 7, 11] = math.nan
                assert math.isnan(float(trainer.step().clip))
        return [trainer.W, trainer.M, trainer.v] + [t for a in trainer.adamw.tensors[1:] for t in a]

    say("example: four steps, then the same with two skipped ones between")
    for a, b in zip(trained(False), trained(True)):
        assert torch.equal(a, b)
