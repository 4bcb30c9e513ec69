"""The norm, the router and the rows' way to the experts and back, forward and
backward, from several host threads at once and in captured graphs whose inputs
change: the same results as one call after the other (calls hold no state)."""
import threading

import pytest
import torch

import block_scaled_precision_bf16_amd as mx
from layer_util import generator, normal

pytestmark = pytest.mark.gpu

# tokens, row length, experts, choices: rows in registers and in two passes, at any
# byte, streamed past the caches; slots in one workgroup, in one launch and in two
SIZES = [(100, 264, 16, 3), (37, 20481, 300, 8), (5000, 301, 64, 8), (2400, 7168, 8, 2)]


def inputs(T, K, E, top, seed):
    g = generator(seed)
    logits = torch.randn(T, E, generator=g) * 2
    logits[torch.rand(T, E, generator=g) < 0.05] = float("-inf")
    t = dict(x=normal(g, T, K), res=normal(g, T, K), w=normal(g, K), dy=normal(g, T, K),
             logits=logits, bias=torch.randn(E, generator=g) * 0.1,
             dscores=torch.randn(T, E, generator=g))
    return {k: v.cuda() for k, v in t.items()}


def steps(t, E, top, stream=None):
    n = mx.mx_rmsnorm(t["x"], t["w"], residual=t["res"], axis=3, want_y=True, checkpoint=True, stream=stream)
    flags = mx.ROUTE_SIGMOID | mx.ROUTE_RENORM
    r = mx.moe_route(t["logits"], top, bias=t["bias"], flags=flags, want_scores=True, stream=stream)
    s = mx.moe_sort(r["experts"], E, align=4, stream=stream)
    xs = mx.moe_gather(n["y"], s["slots"], top, stream=stream)
    out = mx.moe_combine(xs, r["weights"], s["pos"], stream=stream)
    b = mx.moe_combine_backward(t["dy"], xs, r["weights"], pos=s["pos"], slots=s["slots"], stream=stream)
    dl = mx.moe_route_backward(b["dweights"], t["logits"], r["experts"], flags=flags,
                               dscores=t["dscores"], stream=stream)
    nb = mx.mx_rmsnorm_backward(out, n["rstd"], t["w"], q_h=n["q_h"], s_h=n["s_h"], dres=t["dy"],
                                stream=stream)
    nh = mx.mx_rmsnorm_backward(out, n["rstd"], t["w"], h=n["h"], stream=stream)
    return [v for d in (n, r, s, b, nb, nh) for v in d.values()] + [xs, out, dl]


def same(a, b):
    return all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))


def test_threads():
    jobs = [(inputs(T, K, E, top, i), E, top) for i, (T, K, E, top) in enumerate(SIZES)]
    want = [steps(*job) for job in jobs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(jobs))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait(timeout=60)
            got = [steps(*jobs[i], stream=stream) for _ in range(6)]
            stream.synchronize()
            wrong.extend(i for g in got if not same(g, want[i]))
        except Exception as e:                     # reported by the test's own thread
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("T,K,E,top", SIZES)
def test_graphs(T, K, E, top):
    """Two graphs of the same steps, replayed in turn, with eager calls between."""
    ins = [inputs(T, K, E, top, 10 + i) for i in range(2)]
    steps(ins[0], E, top)
    torch.cuda.synchronize()
    graphs, got = [], []
    for t in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(steps(t, E, top))
    for seed in (20, 30, 40):
        for i, t in enumerate(ins):
            for k, v in inputs(T, K, E, top, seed + i).items():
                t[k].copy_(v)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, t in enumerate(ins):
            assert same(got[i], steps(t, E, top)), (seed, i)
