"""The layer of microscaled FP4 experts as programs use it: an expert named twice by a token,
two threads at once, forward and backward captured on a side stream."""
import threading

import pytest
import torch

import nvfp4_token_routed_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _layer(E, H, I, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return M.MxExperts((torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).to(dtype).to(DEV),
                       (torch.randn(E, H, I, generator=g) * I ** -0.5).to(dtype).to(DEV), "swiglu")


def test_an_expert_named_twice():
    """Two halves of one route: every step scales by a power of two, so the bits are the same
    as for the whole route."""
    T, E, H, I = 40, 6, 200, 96
    layer = _layer(E, H, I, 1, torch.float32)
    g = torch.Generator().manual_seed(2)
    x, dy = torch.randn(T, H, generator=g).to(DEV), torch.randn(T, H, generator=g).to(DEV)
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).to(DEV)
    y1, s1 = layer.forward(x, ids, torch.ones(T, 1, device=DEV))
    dx1, dw1 = layer.backward(s1, dy)
    y2, s2 = layer.forward(x, ids.repeat(1, 2), torch.full((T, 2), 0.5, device=DEV))
    dx2, dw2 = layer.backward(s2, dy)
    assert torch.equal(y1, y2) and torch.equal(dx1, dx2)
    assert torch.equal(dw2, dw1.expand(T, 2))


def test_two_threads_at_once():
    T, E, K, H, I = 130, 8, 3, 264, 160
    layer = _layer(E, H, I, 3)
    jobs = []
    for seed in range(2):
        g = torch.Generator().manual_seed(seed)
        jobs.append((torch.randn(T, H, generator=g).bfloat16().to(DEV),
                     torch.rand(T, E, generator=g).argsort(1)[:, :K].int().to(DEV),
                     torch.rand(T, K, generator=g).to(DEV),
                     torch.randn(T, H, generator=g).bfloat16().to(DEV)))

    def step(x, ids, w, dy):
        y, saved = layer.forward(x, ids, w)
        return [y, *layer.backward(saved, dy)]

    want = [step(*job) for job in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    got = step(*jobs[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    failed.append(i)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_captured_with_stream():
    """`stream` names the capturing stream; replays with other inputs, two graphs of one layer
    at once."""
    T, E, K, H, I = 90, 8, 2, 256, 128
    layer = _layer(E, H, I, 4)
    g = torch.Generator().manual_seed(5)
    rnd = lambda: torch.randn(T, H, generator=g).bfloat16().to(DEV)
    graphs = []
    for _ in range(2):
        x, dy = rnd(), rnd()
        ids = torch.rand(T, E, generator=g).argsort(1)[:, :K].int().to(DEV)
        w = torch.rand(T, K, generator=g).to(DEV)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y, saved = layer.forward(x, ids, w, stream=side)
            out = [y, *layer.backward(saved, dy, stream=side)]
        graphs.append((graph, side, (x, ids, w, dy), out))
    for _ in range(3):
        for _, _, (x, _, _, dy), _ in graphs:
            x.copy_(rnd()), dy.copy_(rnd())
        torch.cuda.synchronize()
        for _ in range(5):
            for graph, side, _, _ in graphs:
                with torch.cuda.stream(side):
                    graph.replay()
        torch.cuda.synchronize()
        for _, _, (x, ids, w, dy), out in graphs:
            y, saved = layer.forward(x, ids, w)
            for a, b in zip([y, *layer.backward(saved, dy)], out):
                assert torch.equal(a, b)
