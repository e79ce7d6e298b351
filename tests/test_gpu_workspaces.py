"""The binding's workspaces on the GPU: calls of two threads on one stream, and captured calls whose graph is
replayed after larger eager calls, give the bits of calls made alone and write to nothing else."""
import threading

import pytest
import torch

from linear_attention_recurrent_chunked_b200 import gdn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


def recurrent(seed, T, H=4):
    """One sequence's inputs, long enough to be split into segments that hand states on through the workspace."""
    gen = torch.Generator().manual_seed(seed)
    q, k = (torch.nn.functional.normalize(torch.randn(T, H, 128, generator=gen), dim=-1).to(BF).cuda() for _ in range(2))
    v = torch.randn(T, H, 128, generator=gen).to(BF).cuda()
    return q, k, v, (-torch.rand(T, H, generator=gen)).cuda(), torch.rand(T, H, generator=gen).cuda()


def same(x, y):
    return all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.parametrize("call", [gdn.chunk_fwd, gdn.chunk_fwd_raw], ids=["chunk_fwd", "chunk_fwd_raw"])
def test_two_threads_on_one_stream(call):
    works = [recurrent(1, 2048), recurrent(2, 900)]
    want = [call(*w) for w in works]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def serve(w, y):
        start.wait()
        got = [call(*w) for _ in range(100)]
        torch.cuda.current_stream().synchronize()
        wrong.append(sum(not same(x, y) for x in got))

    threads = [threading.Thread(target=serve, args=a) for a in zip(works, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


def test_graph_replayed_after_larger_eager_calls():
    """The captured call's workspace stays the graph's: larger eager calls in between replace the cached one, and memory
    handed out since then is left alone."""
    stream = torch.cuda.Stream()
    small, large = recurrent(3, 1024), recurrent(4, 4096)
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
        want = gdn.chunk_fwd(*small)
        after = gdn.chunk_fwd(*large)
        o, S = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            gdn.chunk_fwd(*small, o=o, S_T=S)
        bigger = recurrent(5, 12000)
        gdn.chunk_fwd(*bigger)
        held = [torch.full((1 << 20,), 77, dtype=torch.uint8, device="cuda") for _ in range(200)]
        for _ in range(3):
            o.zero_()
            S.zero_()
            g.replay()
            again = gdn.chunk_fwd(*large)
            stream.synchronize()
            assert same((o, S), want) and same(again, after)
        assert all(bool((x == 77).all()) for x in held)
