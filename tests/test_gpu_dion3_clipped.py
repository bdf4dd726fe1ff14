"""The Dion3 update of clipped gradients (gns_dion3_step_clipped).

With a factor that is a power of two c G is exact in G's own type, so the
clipped step must equal the plain step on c G to the bit; a factor of one
must equal it on G.  With other factors the momentum is the fused
multiply-add, checked to the bit, and the rest of the update is the plain
step's from that momentum and a zero gradient."""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_common import NS5, TOL_HALF, need_gpu, rel_err, say
from gram_newton_schulz_amd import synth

pytestmark = pytest.mark.gpu

HYPER = dict(lr=0.02, weight_decay=0.1, mu=0.9, beta2=0.9, eps=1e-8)


def run(gns, state, k, scale=None, **kw):
    W, G, M, v = (t.cuda() for t in state)
    gs = None if scale is None else torch.tensor(scale, dtype=torch.float32, device="cuda")
    S = gns.dion3_step(W, G, M, v, k, NS5, restarts=(2,), grad_scale=gs, **HYPER, **kw)
    torch.cuda.synchronize()
    return W.cpu(), M.cpu(), v.cpu(), S.cpu()


SHAPES = [(2, 96, 300, 24), (3, 150, 521, 40), (1, 64, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_power_of_two_factor(shape, dtype):
    gns = need_gpu()
    count, n, m, k = shape
    W, G, M, v = synth.dion3_state(count, n, m, seed=70, grad_dtype=dtype)
    for c in (1.0, 4.0):
        say("dion3 clipped", shape, dtype, c)
        want = run(gns, (W, (G.float() * c).to(dtype), M, v), k)
        got = run(gns, (W, G, M, v), k, scale=c)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("normuon", [True, False])
def test_any_factor(shape, normuon):
    gns = need_gpu()
    count, n, m, k = shape
    W, G, M, v = synth.dion3_state(count, n, m, seed=71)
    c = np.float32(0.3137)
    # the fused multiply-add: the product is exact in 64 bits (24 + 8 bits), and the sum's
    # rounding there is 2^-29 of the one to fp32
    Mc = (M.double() + float(c) * G.double()).float()
    say("dion3 clipped", shape, c)
    want = run(gns, (W, torch.zeros_like(G), Mc, v), k, normuon=normuon)
    got = run(gns, (W, G, M, v), k, scale=float(c), normuon=normuon)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ref = oracle.dion3_step(synth.as_f64(W[0]), float(c) * synth.as_f64(G[0]), synth.as_f64(M[0]),
                            synth.as_f64(v[0]), k, NS5, restarts=(2,), lr=0.02, weight_decay=0.1, momentum=0.9,
                            beta2=0.9, eps=1e-8, normuon=normuon)
    rows = got[3][0].numpy()
    assert np.array_equal(rows, oracle.dion3_select(synth.as_f64(Mc[0]), k))
    update = (float(np.float32(1 - 0.02 * 0.1)) * synth.as_f64(W[0]) - synth.as_f64(got[0][0]))[rows] / 0.02
    # the update is W's change, so it carries W's rounding: 2^-24 |W| / lr per element
    slack = 2.0 ** -23 * float(np.linalg.norm(synth.as_f64(W[0])[rows])) / 0.02 / float(np.linalg.norm(ref["O"]))
    assert rel_err(update, ref["O"]) <= 2 * TOL_HALF + slack


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nonfinite_factor_skips(bad):
    """W, M and v keep their bits, also where the gradient is not finite."""
    gns = need_gpu()
    for shape in SHAPES:
        count, n, m, k = shape
        W, G, M, v = synth.dion3_state(count, n, m, seed=72)
        G[0, 3, 5] = math.nan
        G[0, 7] = math.inf
        M[0, 2, 2] = -0.0
        say("dion3 skipped", shape, bad)
        got = run(gns, (W, G, M, v), k, scale=bad)
        for a, b in zip(got, (W, M, v)):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))
        assert np.array_equal(got[3][0].numpy(), oracle.dion3_select(synth.as_f64(M[0]), k))


def test_refusals():
    gns = need_gpu()
    W, G, M, v = (t.cuda() for t in synth.dion3_state(1, 16, 32, seed=73))
    for gs, name in ((torch.ones(2, device="cuda"), "GNS_E_DTYPE"), (torch.ones(1), "GNS_E_NULL"),
                     (torch.ones(1, dtype=torch.float64, device="cuda"), "GNS_E_DTYPE"),
                     (M.view(-1)[:1], "GNS_E_ALIAS")):
        with pytest.raises(gns.GnsError) as e:
            gns.dion3_step(W, G, M, v, 4, NS5, grad_scale=gs)
        assert e.value.name == name


def test_norm_to_update_in_one_graph():
    """The whole step of a model with both kinds of parameters, captured:
    the norm of all gradients, Dion3 of the matrices and AdamW of the rest,
    both clipped.  Every replay equals the eager step."""
    gns = need_gpu()
    W, G, M, v = synth.dion3_state(2, 96, 256, seed=74)
    rng = np.random.default_rng(74)
    vec = [torch.from_numpy(rng.normal(size=n)).float() for n in (256, 96, 1001)]
    state = [W, G, M, v] + [t for g in vec for t in (g.clone(), g * 0.5, g * 0.1, g * g)]
    dev = [t.cuda() for t in state]
    p, g, a, b = (dev[4 + i::4] for i in range(4))
    grads = gns.tensor_list([dev[1][0], dev[1][1]] + g)
    rest = gns.adamw_list(p, g, a, b)
    ws = torch.empty(gns.dion3_workspace_bytes(torch.bfloat16, 2, 96, 256, 24), dtype=torch.uint8, device="cuda")
    rows = torch.empty(2, 24, dtype=torch.int64, device="cuda")

    def reset():
        for d, s in zip(dev, state):
            d.copy_(s)

    def step(stream=None):
        got = gns.grad_norm(grads, max_norm=0.5, stream=stream)
        gns.dion3_step(dev[0], dev[1], dev[2], dev[3], 24, NS5, grad_scale=got.clip, row_idx=rows, workspace=ws,
                       stream=stream, **HYPER)
        gns.adamw_step(rest, 7, lr=1e-3, grad_scale=got.clip, stream=stream)
        return got.result

    say("one graph: eager")
    want_result = step().clone()
    want = [t.clone() for t in dev]
    assert 0.0 < float(want_result[1]) < 1.0
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("one graph: capture")
    with torch.cuda.graph(graph):
        result = step()
    for rep in range(3):
        reset()
        say("one graph: replay", rep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(result, want_result)
        assert all(torch.equal(x, y) for x, y in zip(dev, want))
        reset()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(dev, want))
