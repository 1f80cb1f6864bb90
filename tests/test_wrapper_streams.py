"""A call's own memory comes from the pool of the stream that the call runs on.

PyTorch hands a freed block out again to the stream that it was allocated on, whose
later work follows the earlier uses of the block; another stream's work does not."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

DEV = torch.device("cuda", 0)


class FakeTensor:
    """What the wrappers ask of a CUDA tensor."""
    is_cuda = True
    device = DEV

    def __init__(self, *shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.recorded = []

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(self.dim()))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def record_stream(self, stream):
        self.recorded.append(stream)


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, DEV


class FakeLib:
    """Every entry point succeeds; sizes are 4096; handles of the launches are kept."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 4096
            h = args[-1]
            self.streams.append(h.value if isinstance(h, ctypes.c_void_p) else h)
            return 0
        return call


def calls(F):
    bf = lambda *s: FakeTensor(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: FakeTensor(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: FakeTensor(*s, dtype=torch.float32)  # noqa: E731
    kc = FakeTensor(4, 2, 16, 64, dtype=torch.uint8)
    kv = (kc, kc, f32(4, 2, 16, 1), f32(4, 2, 16, 1))
    at = (i32(3, 2), i32(3), 2, 0.1)
    return {
        "kv_append_rope": lambda s: F.kv_append_rope(
            bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), i32(3), f32(10, 64), i32(3), *kv, stream=s),
        "paged_decode_attention_mod": lambda s: F.paged_decode_attention_mod(
            bf(3, 4, 64), *kv, *at, stream=s),
        "paged_prefill_attention": lambda s: F.paged_prefill_attention(
            bf(3, 4, 64), i32(4), *kv, *at, stream=s),
        "paged_decode_attention": lambda s: F.paged_decode_attention(
            bf(3, 4, 64), *kv, *at, stream=s),
        "paged_multiquery_attention": lambda s: F.paged_multiquery_attention(
            bf(3, 2, 4, 64), *kv, *at, stream=s),
        "decode_step": lambda s: F.decode_step(
            bf(3, 2, 64), bf(3, 2, 64), i32(3), bf(3, 4, 64), *kv, *at, stream=s),
        "kv_channel_scales": lambda s: F.kv_channel_scales(bf(3, 2, 64), stream=s),
        "kv_scales_from_absmax": lambda s: F.kv_scales_from_absmax(f32(2, 64), stream=s),
    }


NAMES = ["kv_append_rope", "paged_decode_attention_mod", "paged_prefill_attention",
         "paged_decode_attention", "paged_multiquery_attention", "decode_step",
         "kv_channel_scales", "kv_scales_from_absmax"]


@pytest.fixture
def traced(monkeypatch):
    """The package over fakes; allocations are listed with their stream's handle."""
    from fp8_quantised_paged_gb300 import build
    build.build()
    import fp8_quantised_paged_gb300 as F
    from fp8_quantised_paged_gb300 import binding
    current = [FakeStream(1)]
    made = []

    @contextlib.contextmanager
    def on_stream(s):
        current.append(s)
        yield
        current.pop()

    def empty(*shape, dtype=None, device=None):
        shape = shape[0] if isinstance(shape[0], tuple) else shape
        t = FakeTensor(*shape, dtype=dtype)
        made.append((current[-1].cuda_stream, t))
        return t

    lib = FakeLib()
    monkeypatch.setattr(binding.N, "lib", lib)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream",
                        lambda i: current[-1].cuda_stream, raising=False)
    for cached in (binding._decode_need, binding._prefill_need):
        cached.cache_clear()
    yield F, lib, made
    for cached in (binding._decode_need, binding._prefill_need):
        cached.cache_clear()


@pytest.mark.parametrize("name", NAMES)
def test_memory_is_allocated_on_the_stream_of_the_call(traced, name):
    F, lib, made = traced
    side = FakeStream(7)
    out = calls(F)[name](side)
    assert lib.streams == [7] and made
    assert all(handle == 7 for handle, _ in made)
    # the result is the caller's to use on its own stream: it is not handed out again
    # before what that stream holds when it is freed
    assert [s.cuda_stream for s in out.recorded] == [1]


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_everything_is_on_the_current_one(traced, name):
    F, lib, made = traced
    out = calls(F)[name](None)
    assert lib.streams == [1] and made
    assert all(handle == 1 for handle, _ in made) and not out.recorded


@pytest.mark.gpu
def test_a_call_on_another_stream_beside_one_under_way():
    """Calls on the current stream that give their memory back while their kernels
    run, and at once the same calls on another stream: nothing is shared."""
    import serving_ref as R
    import fp8_quantised_paged_gb300 as F
    dev = "cuda:0"
    hq, hkv, d, bs, n = 64, 8, 128, 16, 4096
    rng = np.random.default_rng(0)
    bt, nb = R.make_tables(rng, [n], bs)
    cache = [t.to(dev) for t in R.make_cache(rng, nb, hkv, bs, d, R.E4M3, R.TOKEN_HEAD)]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    bt, lens, offsets = bt.to(dev), i32(n), i32(0, 1024)
    qs = [torch.randn(1024, hq, d, device=dev).bfloat16() for _ in range(2)]
    kv = torch.randn(1024, hkv, d, device=dev).bfloat16()
    pos, cs = torch.arange(1024, device=dev).int(), torch.randn(1024, d, device=dev)
    skip = torch.full((1024,), -1, dtype=torch.int32, device=dev)
    runs = [
        lambda q, s: F.paged_prefill_attention(q, offsets, *cache, bt, lens, hkv, 0.09, stream=s),
        lambda q, s: F.paged_decode_attention_mod(q[:1], *cache, bt, lens, hkv, 0.09, window=n,
                                                  stream=s),
        lambda q, s: F.paged_decode_attention(q[:1], *cache, bt, lens, hkv, 0.09, stream=s),
        lambda q, s: F.kv_append_rope(q, kv, kv, pos, cs, skip, *cache, stream=s)]
    side = torch.cuda.Stream()
    for run in runs:
        want = [run(q, None).clone() for q in qs]
        torch.cuda.synchronize()
        for _ in range(10):
            a = run(qs[0], None)  # its workspace is free again, its kernels are not done
            b = run(qs[1], side)
            torch.cuda.synchronize()
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert F.get_device_error() == 0


def _attention_calls(F, R):
    """A prefill and a decode over one cache as functions of q and stream."""
    dev = "cuda:0"
    hq, hkv, d, bs, n = 16, 2, 128, 16, 1000
    rng = np.random.default_rng(1)
    bt, nb = R.make_tables(rng, [n], bs)
    cache = [t.to(dev) for t in R.make_cache(rng, nb, hkv, bs, d, R.E4M3, R.TOKEN_HEAD)]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    bt, lens, offsets = bt.to(dev), i32(n), i32(0, 300)
    q = torch.randn(300, hq, d, device=dev).bfloat16()
    return [lambda s=None: F.paged_prefill_attention(q, offsets, *cache, bt, lens, hkv, 0.09,
                                                     window=n // 2, stream=s),
            lambda s=None: F.paged_decode_attention_mod(q[:1], *cache, bt, lens, hkv, 0.09,
                                                        logit_cap=20.0, stream=s)]


@pytest.mark.gpu
def test_calls_captured_on_a_forked_stream():
    import serving_ref as R
    import fp8_quantised_paged_gb300 as F
    runs = _attention_calls(F, R)
    want = [r().clone() for r in runs]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        outs = [r(side) for r in runs]
        torch.cuda.current_stream().wait_stream(side)
        copies = [o.clone() for o in outs]
    for _ in range(3):
        for o in outs + copies:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs + copies, want + want))
    assert F.get_device_error() == 0


@pytest.mark.gpu
def test_threads_that_call_at_once():
    """Each on a stream of its own, made current by it."""
    import threading

    import serving_ref as R
    import fp8_quantised_paged_gb300 as F
    runs = _attention_calls(F, R)
    want = [r().clone() for r in runs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for i in range(60):
                out = runs[(k + i) % 2]()
                s.synchronize()
                if not torch.equal(out, want[(k + i) % 2]):
                    wrong.append((k, i))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and F.get_device_error() == 0
