"""Compaction over more arrays than one launch takes, and a server's steps with static scales."""
import numpy as np
import pytest
import torch

import test_gpu_speculative as S
from pages_ref import Pool
from serving_ref import E4M3, E5M2, INT8, STATIC
from test_gpu_pages import F, arrays, device, i32, same  # noqa: F401
from tree_ref import tree_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n", [128, 129, 300])
def test_compact_many_arrays(F, n):  # noqa: F811
    rng = np.random.default_rng(n)
    host, dev = arrays(rng, 90, 1, 16, [1, 2, 5] * (n // 3) + [1] * (n % 3))
    p = Pool(9, 6, 90, 16, host).fill(rng, rng.integers(0, 96, 6))
    p.fork([0, 1], [6, 7])
    for x, d in zip(host, dev):
        d.copy_(torch.from_numpy(x))
    t, r_n, r = device(p)
    got = F.kv_compact(t, r_n, r, F.KvPages(dev))
    assert np.array_equal(got.cpu().numpy(), p.compact())
    assert p.flags == 0 and len(dev) == n
    same(F, p, (t, r_n, r), dev)


class StaticServer(S.Server):
    """Channel scales of every layer's K and V are fixed; the pages hold codes."""

    def __init__(self, F, rng, d, fmt):  # noqa: F811
        unit = {E4M3: 1 / 100, E5M2: 1 / 3000, INT8: 1 / 40}[fmt]
        made = lambda: torch.from_numpy(unit * np.exp(rng.normal(0, .5, (S.HKV, d)))).float().to(DEV)  # noqa: E731
        self.fixed = ()  # (the pages are made of the codes alone)
        super().__init__(F, rng, d, fmt, STATIC)
        self.fixed = made(), made()
        self.caches = [c + self.fixed for c in self.caches]

    def cache(self, nb):
        codes = lambda: torch.zeros(nb, S.HKV, S.BS, self.d, dtype=torch.uint8, device=DEV)  # noqa: E731
        return (codes(), codes()) + self.fixed

    def check(self):
        n = self.lens()
        assert n.tolist() == [len(h) for h in self.history]
        t = self.t.cpu().numpy()
        held = np.bincount([p for b in range(S.ROWS) for p in t[b, :-(-n[b] // S.BS)]], minlength=S.NB)
        assert np.array_equal(self.r.cpu().numpy(), held)
        for b in np.flatnonzero(n):
            caches, nb = self.fresh(b)
            at = self.t[b, :nb].long()
            for mine, own in zip(self.caches, caches):
                for x, y in zip(mine[:2], own[:2]):
                    x, y = (z.transpose(1, 2).flatten(0, 1)[:n[b]] for z in (x[at], y))
                    assert torch.equal(x, y), b
        assert self.F.get_device_error() == 0


@pytest.mark.parametrize("d,fmt", [(128, E4M3), (64, E5M2), (64, INT8)])
def test_sequences_with_static_scales(F, monkeypatch, d, fmt):  # noqa: F811
    torch.manual_seed(0)
    s = StaticServer(F, np.random.default_rng(0), d, fmt)

    def ref(*a, device):
        return tree_ref(*a, kchan=s.fixed[0].cpu(), device=device)

    monkeypatch.setattr(S, "tree_ref", ref)
    prompts = [0, 150, 33, 16, 1, 0]
    s.resize(prompts)
    for b, m in enumerate(prompts):
        if m:
            s.history[b] = s.make(m)
            s.append(s.caches, s.history[b], range(m), s.slots(b, range(m)))
    s.draft([0, 9, 33, 1, 17, 0])
    s.check()
    s.fork([1, 1], [0, 5])
    s.step([0, 1, 5, 3])
    s.draft([20, 12, 0, 5, 2, 64], window=50)
    s.check()
    s.free([1, 2])
    F.kv_compact(s.t, s.n, s.r, s.pages)
    s.check()
    s.fork([5], [2])
    s.draft([8, 0, 30, 7, 7, 7])
    s.check()
