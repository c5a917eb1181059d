"""The serving loop of test_gpu_paged_together.py on a wide table, so that its trees go to the kernels on clusters (two
CTAs for two tokens, four for more) between page updates and appends, on one workspace and one graph.

In some steps one request's drafted entries are 24-fold: its scores rise past what the four-CTA kernel holds and that
request is done again.  Their size, sm_scale sum |q_i e_i|, is about 24 x 0.072 x 576 x 0.64 = 640, so that fp32's sums
are off by 640 x 2^-21 = 3.1e-4 at most: with the 2^-12 of ordinary scores below the 2^-10 that the bounds of the weights
leave for them (twice the error), and below the 2^-11 + 2^-20 |lse| of the lse."""
import pytest

import test_gpu_paged_together as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("replayed", [False, True])
@pytest.mark.parametrize("tokens", [2, 7, 12])
def test_serving_steps_on_clusters(gpu_lib, monkeypatch, tokens, replayed):
    import torch
    monkeypatch.setattr(base, "T", tokens)
    monkeypatch.setattr(base, "MAX", 1 << 17)
    server = base.Server(gpu_lib, 20 + tokens + replayed)
    graph = None
    if replayed:
        server.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            server.step()
    now = [0] * base.B
    for step in range(7):
        want = []
        for n in now:
            r = server.rng.random()
            if n == 0:
                want.append(int(server.rng.integers(1, 4000)) if r < 0.7 else 0)
            else:
                want.append(0 if r < 0.1 else max(0, n - int(server.rng.integers(1, 9))) if r < 0.25
                            else n if r < 0.3 else min(5000, n + int(server.rng.integers(1, 500))))
        server.new_inputs(want)
        if step % 2 == 1:
            server.draft[step % base.B] *= 24.0
        if graph:
            graph.replay()
        else:
            server.step()
        torch.cuda.synchronize()
        server.check(now, want)
        assert not server.ws[:256].any()
        now = want
