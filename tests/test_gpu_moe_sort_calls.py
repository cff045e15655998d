"""The sorting of tokens by expert under capture with as many experts as there
may be (whose kernel asks for more LDS than a launch has by default), and on
several streams at once.  Exact by the definition, as the index is."""
import numpy as np
import pytest
import torch

import bit_weight_only_pack_amd as lb
from gpu_util import dev
from w8a8_util import routing, sort64

pytestmark = pytest.mark.gpu


class Sort:
    """Buffers of one sort, and the call."""

    def __init__(self, T, top_k, E):
        self.T, self.top_k, self.E, S = T, top_k, E, T * top_k
        self.ids = torch.zeros((T, top_k), dtype=torch.int32, device="cuda")
        self.out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (S, S, E + 1)]
        self.nb = lb.lowbit_moe_sort_workspace_bytes(T, top_k, E)
        self.work = torch.empty(max(self.nb, 1), dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        lb.check(lb.lowbit_moe_sort(self.ids, self.T, self.top_k, self.E, None, self.E, *self.out, self.work, self.nb,
                                    stream))

    def route(self, rng):
        ids = routing(rng, self.T, self.E, self.top_k)
        self.ids.copy_(torch.from_numpy(ids))
        for o in self.out:
            o.fill_(-7)
        self.work.fill_(0x5A)
        self.want = sort64(ids, self.E, None, self.E)

    def right(self):
        return all(np.array_equal(o.cpu().numpy(), w) for o, w in zip(self.out, self.want))


@pytest.mark.parametrize("T,top_k,E", [(60, 6, 1024), (1300, 6, 801), (3000, 8, 1024), (20000, 7, 1000)])
def test_sort_of_many_experts_graph_replays(T, top_k, E):
    """The first call of all is the captured one; then replays on new routings, with eager calls between."""
    rng = np.random.default_rng(T)
    s = Sort(T, top_k, E)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            s.call(stream.cuda_stream)
    for _ in range(3):
        s.route(rng)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert s.right()
        s.route(rng)
        s.call()
        torch.cuda.synchronize()
        assert s.right()


def test_sorts_on_several_streams_at_once():
    """Sorts with a workspace each in flight together, on streams that are and are not torch's current one."""
    rng = np.random.default_rng(9)
    sorts = [Sort(T, top_k, E) for T, top_k, E in ((4000, 8, 128), (9000, 2, 1024), (700, 8, 40), (30000, 3, 7))]
    assert sum(s.nb > 0 for s in sorts) == 3
    streams = [torch.cuda.Stream() for _ in sorts]
    for _ in range(2):
        for s in sorts:
            s.route(rng)
        torch.cuda.synchronize()
        for i, (s, st) in enumerate(zip(sorts, streams)):
            if i % 2:
                with torch.cuda.stream(st):
                    s.call()
            else:
                s.call(st)
        torch.cuda.synchronize()
        assert all(s.right() for s in sorts)


def test_rows_on_two_streams_at_once():
    """Permute, unpermute and its gradient of two batches in flight together give what they give alone."""
    rng = np.random.default_rng(10)
    batches = []
    for T, top_k, E, H in ((500, 4, 16, 1032), (9000, 2, 8, 2048)):
        sr = dev(sort64(routing(rng, T, E, top_k), E, None, E)[1])
        g = torch.Generator(device="cuda").manual_seed(T)
        x, dy = (torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
        w = torch.rand(T, top_k, device="cuda", generator=g)
        S = T * top_k

        def call(stream, T=T, top_k=top_k, H=H, S=S, sr=sr, x=x, dy=dy, w=w):
            e = lambda *n, t=torch.bfloat16: torch.empty(n, dtype=t, device="cuda")
            xp, y, dyp, dw = e(S, H), e(T, H), e(S, H), e(T, top_k, t=torch.float32)
            torch.cuda.synchronize()
            def run():
                lb.check(lb.lowbit_moe_permute(x, None, T, top_k, 2 * H, sr, xp, None, stream))
                lb.check(lb.lowbit_moe_unpermute(xp, lb.LOWBIT_BF16, w, T, top_k, H, sr, y, stream))
                lb.check(lb.lowbit_moe_unpermute_backward(dy, xp, lb.LOWBIT_BF16, w, T, top_k, H, sr, dyp, dw, stream))
            return run, (xp, y, dyp, dw)

        alone, want = call(None)
        alone()
        batches.append((want, *call(torch.cuda.Stream())))
    torch.cuda.synchronize()
    for _ in range(2):
        for _, run, _ in batches:
            run()
    torch.cuda.synchronize()
    for want, _, got in batches:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
