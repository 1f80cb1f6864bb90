"""Cases and plain forms of the operators that a server needs where sequences
branch on the quantised paged KV cache: attention for a tree of drafted tokens,
keeping the accepted path's rows, and forking, resizing and compacting the
sequences' pages.

``run`` makes one pass: the framework's call where ``own`` is true, the plain
form in 32-bit elementary torch operations otherwise.  ``exact`` states each
operator once more in 64 bits.  The page operators change their state in place,
so a pass first puts the tables, lengths and counts back (one small copy, on both
sides); what they copy inside the cache is the same again in every pass.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
E4M3, E5M2, INT8 = 0, 1, 2
TOKEN_HEAD, CHANNEL_STATIC, MX_BLOCK = 0, 1, 3
FMAX = {E4M3: 448.0, E5M2: 57344.0, INT8: 127.0}
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}


# ------------------------------------------------------------------ cases
def _tree(name, batch, length, ragged, nodes, hq, hkv, d, bs, fmt, mode, window=0, prefix=0,
          cap=0.0, alibi=False, lens_seed=0):
    return {"name": name, "op": "tree", "batch": batch, "length": length, "ragged": ragged,
            "nodes": nodes, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "fmt": fmt, "mode": mode,
            "window": window, "prefix": prefix, "cap": cap, "alibi": alibi,
            "lens_seed": lens_seed}


def _pages(name, op, rows, length, ragged, spare, layers, hkv, d, bs, lens_seed, **kw):
    return {"name": name, "op": op, "rows": rows, "length": length, "ragged": ragged,
            "spare": spare, "layers": layers, "hkv": hkv, "d": d, "bs": bs,
            "lens_seed": lens_seed, **kw}


def listed():
    return [
        # a chat turn's few drafted tokens: the smallest attention call, capped scores
        _tree("tree one 700", 1, 700, False, 5, 64, 8, 128, 16, E4M3, TOKEN_HEAD, cap=50.0),
        # the Llama-shaped layer step with a tree of 16 drafted tokens for every request
        _tree("tree 12x16K", 12, 16384, False, 16, 64, 8, 128, 16, E4M3, TOKEN_HEAD),
        # a ragged batch of requests at different stages, trees of up to 24, static scales
        _tree("tree ragged 64", 64, 32768, True, 24, 32, 8, 128, 32, E5M2, CHANNEL_STATIC,
              lens_seed=11),
        # wide trees over long contexts, MX block scales, distance bias
        _tree("tree wide 8x32K", 8, 32768, False, 64, 32, 8, 128, 64, E4M3, MX_BLOCK, alibi=True),
        # one layer of one request: latency
        _pages("keep one", "keep", 1, 700, False, 8, 1, 8, 128, 16, 1, nodes=8, depth=4),
        # every layer of a model's part, a batch of wide trees
        _pages("keep 64 x 16 layers", "keep", 64, 1024, True, 64, 16, 8, 128, 16, 2, nodes=64,
               depth=8),
        # four samples of one prompt
        _pages("fork 1 to 4", "fork", 1, 700, False, 64, 1, 8, 128, 16, 3, children=4),
        # beams of a batch: eight children of each of 16 sequences, 16 layers
        _pages("fork 16 to 128", "fork", 16, 4096, True, 256, 16, 8, 128, 16, 4, children=8),
        # a decode step: every sequence grows by a token, some into a new page
        _pages("resize step 256", "resize", 256, 4096, True, 2000, 0, 8, 128, 16, 5, mixed=False),
        # a scheduler's step on a large pool: some finish, some arrive, some take drafts back
        _pages("resize mixed 1024", "resize", 1024, 16384, True, 60000, 0, 8, 128, 16, 6,
               mixed=True),
        # a small pool, one layer
        _pages("compact 2K", "compact", 64, 1024, True, 1000, 1, 8, 128, 16, 7),
        # half a pool of 16K pages is free and scattered, four layers
        _pages("compact 16K", "compact", 256, 4096, True, 8000, 4, 8, 128, 16, 8),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "keep", "fork", "resize", "compact"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32, 64])
    seed = rng.randrange(1 << 20)
    if op == "tree":
        g = rng.choice([1, 2, 3, 4, 8])
        fmt, mode = rng.choice([(E4M3, TOKEN_HEAD), (E5M2, CHANNEL_STATIC), (INT8, TOKEN_HEAD),
                                (E5M2, TOKEN_HEAD), (E4M3, MX_BLOCK)])
        batch = _spread(rng, 1, 48)
        return _tree("", batch, _spread(rng, 1, min(65536, 200000 // batch)), rng.random() < 0.6,
                     _spread(rng, 1, 64), hkv * g, hkv, d, bs, fmt, mode,
                     window=rng.choice([0, 0, _spread(rng, 1, 5000)]),
                     prefix=rng.choice([0, 0, _spread(rng, 1, 300)]),
                     cap=rng.choice([0.0, 0.0, rng.uniform(10.0, 60.0)]),
                     alibi=rng.random() < 0.3, lens_seed=seed)
    ragged = rng.random() < 0.7
    layers = rng.choice([1, 2, 3, 8])
    if op == "keep":
        return _pages("", op, _spread(rng, 1, 64), _spread(rng, 1, 1024), ragged,
                      rng.randint(1, 50), layers, hkv, d, bs, seed, nodes=_spread(rng, 1, 64),
                      depth=rng.randint(1, 8))
    if op == "fork":
        return _pages("", op, _spread(rng, 1, 16), _spread(rng, 1, 4096), ragged,
                      rng.randint(200, 400), layers, hkv, d, bs, seed, children=rng.randint(1, 8))
    rows = _spread(rng, 1, 256)
    if op == "resize":
        return _pages("", op, rows, _spread(rng, 1, 8192), ragged, _spread(rng, 300, 20000), 0,
                      hkv, d, bs, seed, mixed=rng.random() < 0.5)
    return _pages("", op, rows, _spread(rng, 1, 2048), ragged, _spread(rng, 1, 4000), layers, hkv,
                  d, bs, seed)


def _lengths(case):
    """Cached length (the tree's tokens included) and tree size of every request."""
    rng = random.Random(case["lens_seed"])
    some = lambda n: _spread(rng, 1, n) if case["ragged"] else n  # noqa: E731
    nodes = [some(case["nodes"]) for _ in range(case["batch"])]
    return np.array([some(case["length"]) + n for n in nodes]), np.array(nodes)


# ------------------------------------------------------------------ inputs: trees
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _quantised(x, fmt, mode):
    """Codes and scales of float32 rows [blocks, heads, block, d], made for the inputs."""
    f = FMAX[fmt]
    if mode == MX_BLOCK:
        nb, h, bs, d = x.shape
        y = x.view(nb, h, bs, d // 32, 32)
        e = torch.floor(torch.log2(y.abs().amax(-1).clamp_min(1e-30))) - (8 if fmt == E4M3 else 15)
        z = (y * torch.exp2(-e)[..., None]).clamp(-f, f)
        return z.to(F8[fmt]).view(torch.uint8).view(nb, h, bs, d), (e + 127).to(torch.uint8)
    if mode == CHANNEL_STATIC:
        s = (x.abs().amax((0, 2)) / f).clamp_min(1e-12)
        z = x / s[None, :, None, :]
    else:
        s = (x.abs().amax(-1, keepdim=True) / f).clamp_min(1e-12)
        z = x / s
    z = z.clamp(-f, f)
    if fmt == INT8:
        return (z.round() + 128).to(torch.uint8), s
    return z.to(F8[fmt]).view(torch.uint8), s


def _grown(rng, n):
    """Parents of a drafted tree of n tokens in the order of their depth: about three
    candidates behind each token."""
    parents = [-1]
    while len(parents) < n:
        step = rng.random() < 0.35
        parents.append(min(max(parents[-1], 0) + step, len(parents) - 1))
    return parents


def _prepare_tree(case, seed):
    g = _generator(seed)
    hq, hkv, d, bs = (case[k] for k in ("hq", "hkv", "d", "bs"))
    lens, nodes = _lengths(case)
    pages = (lens + bs - 1) // bs
    nb = int(pages.sum())
    # physical blocks in a random order, unused table entries -1
    order = torch.randperm(nb, device=DEV, generator=g).int()
    col = torch.arange(int(pages.max()), device=DEV)[None]
    held = torch.from_numpy(pages).to(DEV)[:, None]
    first = torch.from_numpy(np.cumsum(pages) - pages).to(DEV)[:, None]
    tables = torch.where(col < held, order[torch.clamp(first + col, max=nb - 1)], -1)
    # a few channels are larger than the rest, as keys' are
    gain = 1.0 + 3.0 * (torch.rand(hkv, 1, d, device=DEV, generator=g) < 0.03)
    kc, ks = _quantised(torch.randn(nb, hkv, bs, d, device=DEV, generator=g) * gain,
                        case["fmt"], case["mode"])
    vc, vs = _quantised(torch.randn(nb, hkv, bs, d, device=DEV, generator=g), case["fmt"],
                        case["mode"])
    rng = random.Random(seed)
    parents = [p for n in nodes.tolist() for p in _grown(rng, n)]
    slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq).float()
    prefix = torch.randint(case["prefix"] + 1, (len(lens),), device=DEV, generator=g).int()
    return {"q": torch.randn(len(parents), hq, d, device=DEV, generator=g).bfloat16(),
            "parents": torch.tensor(parents, dtype=torch.int32, device=DEV),
            "offsets": torch.from_numpy(np.concatenate([[0], np.cumsum(nodes)])).int().to(DEV),
            "kc": kc, "vc": vc, "ks": ks, "vs": vs, "tables": tables.int().contiguous(),
            "lens": torch.from_numpy(lens).int().to(DEV), "most": int(nodes.max()),
            "slopes": slopes if case["alibi"] else None,
            "prefix": prefix if case["prefix"] else None}


# ------------------------------------------------------------------ inputs: pages
def _row_lengths(case):
    """Lengths of the sequences, and what they become where the case resizes them."""
    rng = random.Random(case["lens_seed"])
    lens = [_spread(rng, 1, case["length"]) if case["ragged"] else case["length"]
            for _ in range(case["rows"])]
    if case["op"] != "resize":
        return np.array(lens), None
    if not case["mixed"]:
        return np.array(lens), np.array(lens) + 1
    was, then = [], []
    for n in lens:
        kind = rng.random()
        was.append(0 if kind < 0.05 else n)  # arrives
        drop = rng.randint(1, 8)
        then.append(n if kind < 0.05 else 0 if kind < 0.1 else max(n - drop, (n // 2) // case["bs"]
                    * case["bs"], 1) if kind < 0.4 else n + 1)
    return np.array(was), np.array(then)


def _pool_size(case):
    """Pages of the rows, pages in the pool and columns of the tables."""
    bs = case["bs"]
    lens, then = _row_lengths(case)
    most = lens if then is None else np.maximum(lens, then)
    if case["op"] == "keep":
        lens = most = lens + case["nodes"]
    pages = (lens + bs - 1) // bs
    held = (most + bs - 1) // bs
    return pages, int(held.sum()) + case["spare"], int(held.max()) + 1


def _cache(case, nb, g):
    """Finite codes and scales of every layer's K and V: [2, layers, blocks, heads, block, d]."""
    shape = (2, case["layers"], nb, case["hkv"], case["bs"])
    codes = torch.randint(256, shape + (case["d"],), dtype=torch.uint8, device=DEV, generator=g)
    return codes.bitwise_and_(0xF7), torch.rand(shape + (1,), device=DEV, generator=g)


def _prepare_pages(case, seed):
    g, rng = _generator(seed), random.Random(seed)
    bs, rows = case["bs"], case["rows"]
    pages, nb, cols = _pool_size(case)
    lens, then = _row_lengths(case)
    made = {}
    if case["op"] == "keep":
        lens = lens + case["nodes"]
        parents = [_grown(rng, case["nodes"]) for _ in range(rows)]
        paths = np.full((rows, case["depth"]), -1, np.int32)
        for b, tree in enumerate(parents):
            # a path from the first token down that reads no row that it also writes, so that a
            # pass can be made again on the same state
            at, path, want = 0, [0], rng.randint(1, case["depth"])
            while len(path) < want:
                below = [i for i, p in enumerate(tree) if p == at and i > 0
                         and (i == len(path) or i >= case["depth"])]
                if not below:
                    break
                at = rng.choice(below)
                path.append(at)
            paths[b, :len(path)] = path
        made["accepted"] = torch.from_numpy(paths).to(DEV)
        made["offsets"] = (torch.arange(rows + 1, device=DEV) * case["nodes"]).int()
    children = case.get("children", 0)
    order = np.random.RandomState(seed).permutation(nb).astype(np.int32)
    tables = np.full((rows * (1 + children), cols), -1, np.int32)
    at = 0
    for b in range(rows):
        tables[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        if case["op"] in ("resize", "compact") and b % 2:
            # a pair of rows shares its common prompt's pages
            n = int(min(lens[b - 1], lens[b])) // 2 // bs
            tables[b, :n] = tables[b - 1, :n]
    refs = np.bincount(tables[tables >= 0], minlength=nb).astype(np.int32)
    lens = np.concatenate([lens, np.zeros(rows * children, np.int64)]).astype(np.int32)
    small = torch.from_numpy(np.concatenate([tables.ravel(), lens, refs])).to(DEV)
    now = small.clone()
    made.update(small=small, now=now, tables=now[:tables.size].view(tables.shape),
                lens=now[tables.size:tables.size + lens.size], refs=now[-nb:])
    if children:
        order = list(range(rows, rows * (1 + children)))
        rng.shuffle(order)
        made["dst"] = torch.tensor(order, dtype=torch.int32, device=DEV)
        made["src"] = torch.tensor([i % rows for i in range(len(order))], dtype=torch.int32,
                                   device=DEV)
    if then is not None:
        made["then"] = torch.from_numpy(then.astype(np.int32)).to(DEV)
        # another seed is another turn of the same scheduler's rows
        turn = torch.from_numpy(np.random.RandomState(seed).permutation(rows)).to(DEV)
        for t in (made["tables"], made["lens"], made["then"]):
            t.copy_(t[turn].clone())
        made["small"].copy_(now)
    if case["layers"]:
        made["codes"], made["scales"] = _cache(case, nb, g)
    return made


def prepare(case, seed):
    state = _prepare_tree(case, seed) if case["op"] == "tree" else _prepare_pages(case, seed)
    state["case"] = case
    return state


# ------------------------------------------------------------------ plain forms: trees
def _values(codes, scale, tables, case):
    """Dequantised rows of every request's pages: float32 [batch, heads, tokens, d]."""
    fmt, mode = case["fmt"], case["mode"]
    t = tables.long().clamp_min(0)
    c = codes[t]
    x = c.float() - 128.0 if fmt == INT8 else c.view(F8[fmt]).float()
    b, p, h, bs, d = x.shape
    if mode == MX_BLOCK:
        s = torch.exp2(scale[t].float() - 127.0)
        x = (x.view(b, p, h, bs, d // 32, 32) * s[..., None]).view(b, p, h, bs, d)
    elif mode == CHANNEL_STATIC:
        x = x * scale[:, None, :]
    else:
        x = x * scale[t]
    return x.transpose(1, 2).reshape(b, h, p * bs, d)


def _plain_tree(st, case):
    d, hq, hkv, cap = case["d"], case["hq"], case["hkv"], case["cap"]
    g = hq // hkv
    lens, offs, n = st["lens"].long(), st["offsets"].long(), st["most"]
    b, size = lens.numel(), offs[1:] - offs[:-1]
    i = torch.arange(n, device=DEV)
    here = (offs[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)
    held = i < size[:, None]
    # who descends from whom: the sum of all powers of the parent relation, an inverse
    par = torch.where(held, st["parents"][here].long(), -1)
    eye = torch.eye(n, device=DEV)
    up = eye - (par[:, :, None] == i).float()
    line = torch.linalg.solve_triangular(up, eye.expand(b, n, n), upper=False, unitriangular=True)
    line = line > 0.5
    depth = line.sum(-1) - 1
    q = st["q"][here].float().view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    k = _values(st["kc"], st["ks"], st["tables"], case)
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).view(b, hkv, g, n, -1)
    del k
    if cap:
        z = z.div_(cap).tanh_().mul_(cap)
    ctx = (lens - size)[:, None]
    j = torch.arange(z.shape[-1], device=DEV)[None].expand(b, -1)
    node = (j - ctx).clamp(0, n - 1)
    drafted = j >= ctx
    place = torch.where(drafted, ctx + depth.gather(1, node), j)  # a token's position
    far = (ctx + depth)[:, :, None] - place[:, None]
    if st["slopes"] is not None:
        z = z.sub_(st["slopes"].view(1, hkv, g, 1, 1) * far[:, None, None].float())
    see = torch.where(drafted[:, None], line.gather(2, node[:, None].expand(b, n, -1)), True)
    if case["window"]:
        near = far < case["window"]
        if st["prefix"] is not None:
            near |= (j < st["prefix"].long()[:, None].minimum(ctx))[:, None]
        see &= near
    see &= (j < lens[:, None])[:, None]
    z = z.masked_fill_(~see[:, None, None], -math.inf)
    p = z.sub_(z.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp_min(1e-30)).view(b, hkv, g * n, -1)
    o = torch.matmul(p, _values(st["vc"], st["vs"], st["tables"], case))
    o = o.view(b, hkv, g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    return o[held].bfloat16()


# ------------------------------------------------------------------ plain forms: pages
def _plain_keep(st, case):
    bs, acc, offs = case["bs"], st["accepted"].long(), st["offsets"].long()
    ctx = st["lens"].long() - (offs[1:] - offs[:-1])
    ok = acc >= 0
    count = ok.sum(1)
    # an unused entry repeats the first move
    src = ctx[:, None] + torch.where(ok, acc, acc[:, :1].clamp_min(0))
    dst = ctx[:, None] + torch.where(ok, torch.arange(acc.shape[1], device=DEV), 0)
    t = st["tables"].long()
    sb, db = t.gather(1, src // bs), t.gather(1, dst // bs)
    for x in (st["codes"], st["scales"]):
        x[:, :, db, :, dst % bs] = x[:, :, sb, :, src % bs]
    st["new"] = (ctx + count).int()
    return {"lens": st["new"], "codes": st["codes"].view(F8[E4M3]), "scales": st["scales"]}


def _page_outputs(st, case, **more):
    out = {"tables": st["tables"], "lens": st["lens"], "refs": st["refs"], **more}
    if case["layers"]:
        out.update(codes=st["codes"].view(F8[E4M3]), scales=st["scales"])
    return out


def _free(refs):
    """The free pages' numbers, the lowest first (then the others)."""
    return torch.sort(refs.ne(0).to(torch.uint8), stable=True).indices


def _plain_fork(st, case):
    bs, src, dst = case["bs"], st["src"].long(), st["dst"].long()
    n = st["lens"].long()[src]
    last, tail = n // bs, n % bs != 0
    row = st["tables"].long()[src]
    fresh = _free(st["refs"])[(tail.long().cumsum(0) - 1).clamp_min(0)]
    col = torch.arange(row.shape[1], device=DEV)
    old = row.gather(1, last[:, None])[:, 0]
    new = torch.where((col == last[:, None]) & tail[:, None], fresh[:, None], row)
    used = col < ((n + bs - 1) // bs)[:, None]
    new = torch.where(used, new, -1)
    st["tables"][dst] = new.int()
    st["lens"][dst] = n.int()
    st["refs"].scatter_add_(0, new.clamp_min(0).flatten(), used.int().flatten())
    # a sequence that ends with a page copies its first page onto itself
    fr, to = torch.where(tail, old, row[:, 0]), torch.where(tail, fresh, row[:, 0])
    st["codes"][:, :, to] = st["codes"][:, :, fr]
    st["scales"][:, :, to] = st["scales"][:, :, fr]
    return _page_outputs(st, case)


def _plain_resize(st, case):
    bs, t, refs = case["bs"], st["tables"], st["refs"]
    col = torch.arange(t.shape[1], device=DEV)
    old = ((st["lens"].long() + bs - 1) // bs)[:, None]
    new = ((st["then"].long() + bs - 1) // bs)[:, None]
    gone, come = (col >= new) & (col < old), (col >= old) & (col < new)
    refs.scatter_add_(0, t.long().clamp_min(0).flatten(), -gone.int().flatten())
    rank = come.flatten().long().cumsum(0) - 1
    got = _free(refs)[rank.clamp(0, refs.numel() - 1)].view(t.shape)
    t.copy_(torch.where(come, got, torch.where(gone, -1, t.long())))
    refs.scatter_add_(0, t.long().clamp_min(0).flatten(), come.int().flatten())
    st["lens"].copy_(st["then"])
    return _page_outputs(st, case)


def _plain_compact(st, case):
    t, refs = st["tables"], st["refs"]
    page = torch.arange(refs.numel(), device=DEV)
    live = refs > 0
    n = live.sum()
    high, low = live & (page >= n), ~live & (page < n)
    m = int(high.sum())
    fr, to = _free(~high)[:m], _free(~low)[:m]
    moved = torch.where(live, page, -1)
    moved[fr] = to
    st["codes"][:, :, to] = st["codes"][:, :, fr]
    st["scales"][:, :, to] = st["scales"][:, :, fr]
    t.copy_(torch.where(t >= 0, moved[t.long().clamp_min(0)], -1))
    refs[to] = refs[fr]
    refs[fr] = 0
    return _page_outputs(st, case, moved=moved.int())


PLAIN = {"tree": _plain_tree, "keep": _plain_keep, "fork": _plain_fork, "resize": _plain_resize,
         "compact": _plain_compact}


def _own(st, case):
    import fp8_quantised_paged_gb300 as F
    op = case["op"]
    if op == "tree":
        return F.paged_tree_attention(
            st["q"], st["offsets"], st["parents"], st["kc"], st["vc"], st["ks"], st["vs"],
            st["tables"], st["lens"], case["hkv"], case["d"] ** -0.5, window=case["window"],
            prefix_lens=st["prefix"], logit_cap=case["cap"], alibi_slopes=st["slopes"],
            fmt=case["fmt"], scale_mode=case["mode"], group_size=32)
    if op == "resize":
        F.kv_resize(st["then"], st["tables"], st["lens"], st["refs"], case["bs"])
        return _page_outputs(st, case)
    if "pages" not in st:  # a server makes it once, with the cache
        st["pages"] = F.KvPages([*st["codes"].flatten(0, 1).unbind(),
                                 *st["scales"].flatten(0, 1).unbind()])
    if op == "keep":
        new = F.kv_keep_accepted(st["accepted"], st["offsets"], st["tables"], st["lens"],
                                 st["pages"])
        return {"lens": new, "codes": st["codes"].view(F8[E4M3]), "scales": st["scales"]}
    if op == "fork":
        F.kv_fork(st["src"], st["dst"], st["tables"], st["lens"], st["refs"], st["pages"])
        return _page_outputs(st, case)
    moved = F.kv_compact(st["tables"], st["lens"], st["refs"], st["pages"])
    return _page_outputs(st, case, moved=moved)


def run(state):
    case = state["case"]
    if case["op"] in ("fork", "resize", "compact"):
        state["now"].copy_(state["small"])
    return _own(state, case) if own else PLAIN[case["op"]](state, case)


# ------------------------------------------------------------------ what a pass needs
def _tree_work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens, nodes = _lengths(case)
    seen = read = 0
    for n, m in zip(lens.tolist(), nodes.tolist()):
        ctx = n - m
        near = min(ctx, case["window"]) if case["window"] else ctx
        near += min(case["prefix"] // 2, ctx - near)
        read += near + m
        # a node's line is about as long as the logarithm of the tree's size
        seen += m * (near + 1 + int(math.log2(m)))
    mode = case["mode"]
    scales = (hkv * d * 4 if mode == CHANNEL_STATIC
              else read * hkv * (d // 32 if mode == MX_BLOCK else 4))
    moved = read * hkv * d * 2 + 2 * scales + read // case["bs"] * 4
    return {"bytes": moved + int(nodes.sum()) * (hq * d * 4 + 4), "flops": 4 * d * hq * seen}


def work(case):
    if case["op"] == "tree":
        return _tree_work(case)
    bs, rows, layers = case["bs"], case["rows"], case["layers"]
    lens, then = _row_lengths(case)
    pages, nb, cols = _pool_size(case)
    row = case["hkv"] * (case["d"] + 4) * 2 * layers  # a token in every layer
    if case["op"] == "keep":
        depth = min(case["depth"], 1 + math.log2(case["nodes"]))
        return {"bytes": int(rows * (depth - 1) * row * 2 + rows * (case["depth"] + 4) * 4),
                "flops": 0}
    if case["op"] == "fork":
        kids = case["children"]
        tails = int((lens % bs != 0).sum()) * kids
        return {"bytes": tails * bs * row * 2 + int(pages.sum()) * kids * 16 + nb * 4, "flops": 0}
    if case["op"] == "resize":
        changed = np.abs((then + bs - 1) // bs - pages).sum()
        return {"bytes": int(changed) * 16 + nb * 4 + rows * 16, "flops": 0}
    live = int(pages.sum())
    moved = live * (nb - live) // nb
    return {"bytes": moved * bs * row * 2 + nb * 12 + live * 8, "flops": 0}


# ------------------------------------------------------------------ in 64 bits
def _exact_values(codes, scale, blocks, case):
    """Float64 rows [heads, tokens, d] of one request's pages, from its codes."""
    c = codes[blocks].permute(1, 0, 2, 3)
    c = c.double() - 128 if case["fmt"] == INT8 else c.contiguous().view(F8[case["fmt"]]).double()
    if case["mode"] == MX_BLOCK:
        s = torch.exp2(scale[blocks].double() - 127).repeat_interleave(32, -1)
        c = c * s.permute(1, 0, 2, 3)
    elif case["mode"] == CHANNEL_STATIC:
        c = c * scale.double()[:, None, None]
    else:
        c = c * scale[blocks].double().permute(1, 0, 2, 3)
    return c.flatten(1, 2)


def _exact_tree(case, st):
    lens, nodes = _lengths(case)
    if 4 * case["d"] * case["hq"] * float((lens * nodes).sum()) > 6e12:
        return None  # minutes in 64 bits
    g = case["hq"] // case["hkv"]
    parents = st["parents"].tolist()
    outs, row = [], 0
    for b, (n, m) in enumerate(zip(lens.tolist(), nodes.tolist())):
        ctx = n - m
        see = torch.zeros(m, n, dtype=torch.bool)
        place = torch.arange(n, dtype=torch.float64)
        for i in range(m):
            at, line = i, []
            while at >= 0:
                line.append(at)
                at = parents[row + at]
            place[ctx + i] = ctx + len(line) - 1
            see[i, :ctx] = True
            for at in line:
                see[i, ctx + at] = True
        dist = place[ctx:, None] - place[None]
        if case["window"]:
            keep = dist < case["window"]
            if st["prefix"] is not None:
                keep[:, :min(int(st["prefix"][b]), ctx)] = True
            see &= keep
        see, dist = see.to(DEV), dist.to(DEV)
        blocks = st["tables"][b, :(n + case["bs"] - 1) // case["bs"]].long()
        k = _exact_values(st["kc"], st["ks"], blocks, case)[:, :n]
        v = _exact_values(st["vc"], st["vs"], blocks, case)[:, :n]
        o = torch.empty(m, case["hq"], case["d"], dtype=torch.float64, device=DEV)
        for h in range(case["hq"]):
            z = st["q"][row:row + m, h].double() @ k[h // g].T / math.sqrt(case["d"])
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if st["slopes"] is not None:
                z = z - st["slopes"][h].double() * dist
            o[:, h] = torch.softmax(torch.where(see, z, -math.inf), -1) @ v[h // g]
        outs.append(o)
        row += m
    return torch.cat(outs)


def _exact_pages(case, st):
    """The operators page by page, on the host's numbers."""
    if case["layers"] * st["refs"].numel() * case["hkv"] * case["bs"] * case["d"] > 3e9:
        return None
    bs = case["bs"]
    tables, lens, refs = (st[k].cpu().tolist() for k in ("tables", "lens", "refs"))
    moves, more = [], {}  # ((page, offset or None) from, to)
    if case["op"] == "keep":
        new = []
        for row, n, path in zip(tables, lens, st["accepted"].tolist()):
            kept = [a for a in path if a >= 0]
            ctx = n - case["nodes"]
            for t, a in enumerate(kept):
                i, o = ctx + a, ctx + t
                moves.append(((row[i // bs], i % bs), (row[o // bs], o % bs)))
            new.append(ctx + len(kept))
        lens = new
    elif case["op"] == "fork":
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            n = lens[s]
            tables[d], lens[d] = list(tables[s]), n
            if n % bs:
                page = refs.index(0)
                moves.append(((tables[s][n // bs], None), (page, None)))
                tables[d][n // bs] = page
            for p in tables[d][:-(-n // bs)]:
                refs[p] += 1
    elif case["op"] == "resize":
        then = st["then"].tolist()
        for row, n, m in zip(tables, lens, then):
            for c in range(-(-m // bs), -(-n // bs)):
                refs[row[c]] -= 1
                row[c] = -1
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for row, n, m in zip(tables, lens, then):
            for c in range(-(-n // bs), -(-m // bs)):
                row[c] = next(free)
                refs[row[c]] = 1
        lens = then
    else:
        live = [p for p, r in enumerate(refs) if r > 0]
        low = [p for p in range(len(live)) if refs[p] == 0]
        to = {p: p for p in live}
        to.update(zip([p for p in live if p >= len(live)], low))
        for p, t in to.items():
            if p != t:
                moves.append(((p, None), (t, None)))
                refs[t], refs[p] = refs[p], 0
        tables = [[to[p] if p >= 0 else -1 for p in row] for row in tables]
        more["moved"] = torch.tensor([to.get(p, -1) for p in range(len(refs))])
    out = {"lens": torch.tensor(lens), **more}
    if case["op"] != "keep":
        out.update(tables=torch.tensor(tables), refs=torch.tensor(refs))
    if case["layers"]:
        codes, scales = st["codes"], st["scales"]
        for (p, i), (t, o) in moves:
            for x in (codes, scales):
                if i is None:
                    x[:, :, t] = x[:, :, p]
                elif (p, i) != (t, o):
                    x[:, :, t, :, o] = x[:, :, p, :, i]
        out.update(codes=codes.view(F8[E4M3]).double(), scales=scales.double())
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_tree(case, st) if case["op"] == "tree" else _exact_pages(case, st)
