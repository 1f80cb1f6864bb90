"""A server's steps with drafted trees, as they would be used together: pages for the drafts,
rotary append, tree attention, the accepted path kept, pages given back, sequences forked and
freed, the pool compacted, and single-token decodes between.  After every step the cached rows
are those of a cache that each sequence would have to itself, byte for byte."""
import numpy as np
import pytest
import torch

from serving_ref import E4M3, E5M2, INT8, MX, TOKEN_HEAD, chunk_values
from tree_ref import check_tree, lines, tree_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LAYERS, HQ, HKV, BS, ROWS, COLS, NB = 2, 12, 2, 16, 6, 20, 90


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).to(DEV)


class Server:
    def __init__(self, F, rng, d, fmt, mode):
        self.F, self.rng, self.d, self.fmt, self.mode = F, rng, d, fmt, mode
        self.kw = dict(fmt=fmt, scale_mode=mode, group_size=32)
        self.caches = [self.cache(NB) for _ in range(LAYERS)]
        self.pages = F.KvPages([x for c in self.caches for x in c])
        self.t, self.n, self.r = i32(np.full((ROWS, COLS), -1)), i32(np.zeros(ROWS)), i32(np.zeros(NB))
        self.cs = torch.from_numpy(rng.uniform(-1, 1, (COLS * BS, d)).astype(np.float32)).to(DEV)
        self.history = [[] for _ in range(ROWS)]  # of a row: numbers of its tokens
        self.tokens = []                          # k and v of every token made, before turning

    def cache(self, nb):
        codes = lambda: torch.zeros(nb, HKV, BS, self.d, dtype=torch.uint8, device=DEV)  # noqa: E731
        dt, w = (torch.uint8, self.d // 32) if self.mode == MX else (torch.float32, 1)
        scales = lambda: torch.zeros(nb, HKV, BS, w, dtype=dt, device=DEV)  # noqa: E731
        return codes(), codes(), scales(), scales()

    def make(self, n):
        """n new tokens' numbers."""
        for _ in range(n):
            x = self.rng.standard_normal((LAYERS, 2, HKV, self.d)).astype(np.float32)
            self.tokens.append(torch.from_numpy(x).bfloat16())
        return list(range(len(self.tokens) - n, len(self.tokens)))

    def append(self, caches, numbers, positions, slots, q=None):
        outs = []
        for layer, c in enumerate(caches):
            kv = torch.stack([self.tokens[i][layer] for i in numbers]).to(DEV)
            outs.append(self.F.kv_append_rope(
                None if q is None else q, kv[:, 0].contiguous(), kv[:, 1].contiguous(),
                i32(positions), self.cs, i32(slots), *c, **self.kw))
        return outs

    def resize(self, lens):
        self.F.kv_resize(i32(lens), self.t, self.n, self.r, BS)

    def lens(self):
        return self.n.cpu().numpy()

    def slots(self, row, places):
        t = self.t[row].cpu().numpy()
        return [int(t[p // BS]) * BS + p % BS for p in places]

    def fresh(self, row):
        """The row's sequence in caches of its own, pages in order."""
        h = self.history[row]
        nb = max(-(-len(h) // BS), 1)
        caches = [self.cache(nb) for _ in range(LAYERS)]
        if h:
            self.append(caches, h, range(len(h)), range(len(h)))
        return caches, nb

    def check(self):
        """Lengths, counts, bytes, and a decode of every row, which has the same bits."""
        F = self.F
        n = self.lens()
        assert n.tolist() == [len(h) for h in self.history]
        t = self.t.cpu().numpy()
        held = np.bincount([p for b in range(ROWS) for p in t[b, :-(-n[b] // BS)]], minlength=NB)
        assert np.array_equal(self.r.cpu().numpy(), held)
        for b in range(ROWS):
            if not n[b]:
                continue
            caches, nb = self.fresh(b)
            at = self.t[b, :nb].long()
            q = torch.randn(1, HQ, self.d, device=DEV).bfloat16()
            for mine, own in zip(self.caches, caches):
                for x, y in zip(mine, own):
                    x = x[at].transpose(1, 2).flatten(0, 1)[:n[b]]
                    y = y.transpose(1, 2).flatten(0, 1)[:n[b]]
                    assert torch.equal(x, y), b
                args = lambda c, t: (q, *c, t, self.n[b:b + 1], HKV, 0.1)  # noqa: E731
                x = F.paged_decode_attention(*args(mine, self.t[b:b + 1]), **self.kw)
                y = F.paged_decode_attention(*args(own, i32([np.arange(nb)])), **self.kw)
                assert torch.equal(x, y), b
        assert F.get_device_error() == 0

    def draft(self, nodes, window=0):
        """Verify trees of these sizes and keep a path of each."""
        F, rng, ctx = self.F, self.rng, self.lens()
        offsets = np.concatenate([[0], np.cumsum(nodes)])
        parents = [[int(rng.integers(max(-1, i - 5), i)) for i in range(m)] for m in nodes]
        self.resize(ctx + nodes)
        new, places, slots = [], [], []
        for b, m in enumerate(nodes):
            new.append(self.make(m))
            places += [ctx[b] + len(line) - 1 for line in lines(parents[b])]
            slots += self.slots(b, ctx[b] + np.arange(m))
        total = int(offsets[-1])
        q = torch.randn(total, HQ, self.d, device=DEV).bfloat16()
        turned = self.append(self.caches, sum(new, []), places, slots, q)
        for qt, c in zip(turned, self.caches):
            out = F.paged_tree_attention(qt, i32(offsets), i32(sum(parents, [])), *c, self.t, self.n,
                                         HKV, 0.1, window=window, **self.kw)
            values = chunk_values([x.cpu() for x in c], self.fmt, self.mode, 32)
            ref = tree_ref(qt.cpu(), offsets, sum(parents, []), self.lens(), self.t.cpu(), values,
                           HKV, 0.1, BS, self.fmt, self.mode, window, device=DEV)
            check_tree(out, ref, self.d, bf16=True)
        accepted = np.full((ROWS, 4), -1)
        for b, m in enumerate(nodes):
            if m:
                path = lines(parents[b])[rng.integers(0, m)][:rng.integers(0, 5)]
                accepted[b, :len(path)] = path
                self.history[b] += [new[b][i] for i in path]
        kept = F.kv_keep_accepted(i32(accepted), i32(offsets), self.t, self.n, self.pages)
        F.kv_resize(kept, self.t, self.n, self.r, BS)

    def step(self, rows):
        """A token more for some rows."""
        grow = np.zeros(ROWS, np.int64)
        grow[rows] = 1
        ctx = self.lens()
        self.resize(ctx + grow)
        new = self.make(len(rows))
        self.append(self.caches, new, ctx[rows], sum((self.slots(b, [ctx[b]]) for b in rows), []))
        for b, i in zip(rows, new):
            self.history[b].append(i)

    def fork(self, src, dst):
        self.F.kv_fork(i32(src), i32(dst), self.t, self.n, self.r, self.pages)
        for a, b in zip(src, dst):
            self.history[b] = list(self.history[a])

    def free(self, rows):
        lens = self.lens()
        lens[rows] = 0
        self.resize(lens)
        for b in rows:
            self.history[b] = []


@pytest.mark.parametrize("d,fmt,mode", [(128, E4M3, TOKEN_HEAD), (64, E5M2, TOKEN_HEAD),
                                        (128, INT8, TOKEN_HEAD), (64, E4M3, MX)])
def test_sequences_through_drafts_forks_and_compactions(d, fmt, mode):
    import fp8_quantised_paged_gb300 as F
    F.get_device_error()
    torch.manual_seed(0)
    s = Server(F, np.random.default_rng(0), d, fmt, mode)
    prompts = [0, 150, 33, 16, 1, 0]
    s.resize(prompts)
    for b, m in enumerate(prompts):
        if m:
            s.history[b] = s.make(m)
            s.append(s.caches, s.history[b], range(m), s.slots(b, range(m)))
    s.check()
    s.draft([0, 9, 33, 1, 17, 0])
    s.check()
    s.fork([1, 1], [0, 5])
    s.check()
    s.step([0, 1, 5, 3])  # the forks part
    s.check()
    s.draft([20, 12, 0, 5, 2, 64], window=50)
    s.check()
    s.free([1, 2])
    s.check()
    F.kv_compact(s.t, s.n, s.r, s.pages)
    live = int((s.r > 0).sum())
    assert (s.r[:live] > 0).all()
    s.check()
    s.fork([5], [2])
    s.draft([8, 0, 30, 7, 7, 7])
    s.step([2, 5])
    s.check()
    s.free(range(ROWS))
    assert int(s.r.abs().sum()) == 0
    s.check()
