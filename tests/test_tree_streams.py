"""The tree attention's and the page operators' own memory comes from the pool of the stream
that the call runs on; calls at once on several streams and threads share nothing."""
import threading

import numpy as np
import pytest
import torch

from test_wrapper_streams import FakeStream, FakeTensor, traced  # noqa: F401


def calls(F):
    bf = lambda *s: FakeTensor(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: FakeTensor(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: FakeTensor(*s, dtype=torch.float32)  # noqa: E731
    kc = FakeTensor(4, 2, 16, 64, dtype=torch.uint8)
    kv = (kc, kc, f32(4, 2, 16, 1), f32(4, 2, 16, 1))

    class Pages:  # what the wrappers ask of a KvPages
        device, num_blocks, n_kv_heads, block_size, per_token = kc.device, 4, 2, 16, True
        _args = (0x1000, 0x1000, 4)

    rows = (i32(3, 2), i32(3))
    return {
        "paged_tree_attention": lambda s: F.paged_tree_attention(
            bf(3, 4, 64), i32(4), i32(3), *kv, *rows, 2, 0.1, stream=s),
        "kv_keep_accepted": lambda s: F.kv_keep_accepted(i32(3, 2), i32(4), *rows, Pages, stream=s),
        "kv_compact": lambda s: F.kv_compact(*rows, i32(4), Pages, stream=s),
        "kv_fork": lambda s: F.kv_fork(i32(1), i32(1), *rows, i32(4), Pages, stream=s),
        "kv_resize": lambda s: F.kv_resize(i32(3), *rows, i32(4), 16, stream=s),
    }


NAMES = ["paged_tree_attention", "kv_keep_accepted", "kv_compact", "kv_fork", "kv_resize"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_is_allocated_on_the_stream_of_the_call(traced, name):  # noqa: F811
    from fp8_quantised_paged_gb300 import binding
    F, lib, made = traced
    binding._tree_need.cache_clear()
    out = calls(F)[name](FakeStream(7))
    binding._tree_need.cache_clear()
    assert lib.streams == [7] and made
    assert all(handle == 7 for handle, _ in made)
    if out is not None:  # the result is read on the current stream, too
        assert [s.cuda_stream for s in out.recorded] == [1]


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_everything_is_on_the_current_one(traced, name):  # noqa: F811
    from fp8_quantised_paged_gb300 import binding
    F, lib, made = traced
    binding._tree_need.cache_clear()
    out = calls(F)[name](None)
    binding._tree_need.cache_clear()
    assert lib.streams == [1] and made
    assert all(handle == 1 for handle, _ in made)
    assert out is None or not out.recorded


def _trees(F, fmt=0):
    from test_gpu_tree import Case, TOKEN_HEAD
    cases = [Case(31 + i, [900, 40], [9, 30 + i], 16, 2, 128, 16, fmt, TOKEN_HEAD) for i in range(2)]
    runs = []
    for c in cases:
        a, kw = c.args()
        runs.append(lambda s=None, a=a, kw=kw: F.paged_tree_attention(*a, **kw, stream=s))
    return runs


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 2])
def test_trees_on_two_streams_at_once(fmt):
    import fp8_quantised_paged_gb300 as F
    runs = _trees(F, fmt)
    want = [r().clone() for r in runs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a, b = runs[0](), runs[1](side)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert F.get_device_error() == 0


@pytest.mark.gpu
def test_two_graphs_of_trees_replayed_at_once():
    """Each graph holds the workspace of its own capture."""
    import fp8_quantised_paged_gb300 as F
    runs = _trees(F)
    want = [r().clone() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for r, s in zip(runs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(r())
        graphs.append(g)
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert F.get_device_error() == 0


@pytest.mark.gpu
def test_threads_that_call_at_once():
    """Each on a stream of its own: a tree, or growing and freeing rows of a pool of its own."""
    import fp8_quantised_paged_gb300 as F
    runs = _trees(F)
    want = [r().clone() for r in runs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda:0")  # noqa: E731
            t, n, r = i32(np.full((4, 8), -1)), i32([0] * 4), i32([0] * 32)
            for i in range(40):
                out = runs[(k + i) % 2]()
                F.kv_resize(i32([k, 16 + i, 50, 0]), t, n, r, 16)
                counts = int(r.sum()), n.tolist()
                if not torch.equal(out, want[(k + i) % 2]):
                    wrong.append((k, i))
                if counts != ((k + 15) // 16 + (31 + i) // 16 + 4, [k, 16 + i, 50, 0]):
                    wrong.append((k, i, counts))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and F.get_device_error() == 0
