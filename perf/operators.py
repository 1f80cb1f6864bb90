"""Cases and plain forms of the serving path's operators: the append with
rotary positions, decode attention with score modifiers, and prefill
attention over ragged chunks, all on the quantised paged KV cache.

``run`` makes one pass: the framework's call where ``own`` is true, the plain
form in 32-bit elementary torch operations otherwise.  ``exact`` states each
operator once more in 64 bits.
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
def _append(name, tokens, hq, hkv, d, bs, fmt, mode, rot, interleaved, max_pos, far):
    return {"name": name, "op": "append", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d,
            "bs": bs, "fmt": fmt, "mode": mode, "rot": rot, "interleaved": interleaved,
            "max_pos": max_pos, "far": far}


def _attention(name, op, batch, length, ragged, chunk, hq, hkv, d, bs, fmt, mode, window=0,
               prefix=0, cap=0.0, alibi=False, lens_seed=0):
    return {"name": name, "op": op, "batch": batch, "length": length, "ragged": ragged,
            "chunk": chunk, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "fmt": fmt, "mode": mode,
            "window": window, "prefix": prefix, "cap": cap, "alibi": alibi,
            "lens_seed": lens_seed}


def listed():
    return [
        # the new tokens of a 12-request decode step, one per request, far into their contexts
        _append("append step 12", 12, 64, 8, 128, 16, E4M3, TOKEN_HEAD, 128, False, 131072, True),
        # a prefill batch of one layer: whole prompts, positions from 0
        _append("append bulk 16384", 16384, 64, 8, 128, 16, E4M3, TOKEN_HEAD, 128, False, 16384,
                False),
        # a ragged batch of odd size, half of each head rotated in interleaved pairs, static scales
        _append("append odd 1531", 1531, 32, 8, 128, 32, E5M2, CHANNEL_STATIC, 64, True, 32768,
                True),
        # one short chat turn, capped scores: the smallest attention call
        _attention("decode one 700", "decode", 1, 700, False, 1, 64, 8, 128, 16, E4M3,
                   TOKEN_HEAD, cap=50.0),
        # the Llama-shaped layer step with a sliding window over part of the context
        _attention("decode window 12x16K", "decode", 12, 16384, False, 1, 64, 8, 128, 16, E4M3,
                   TOKEN_HEAD, window=4096, prefix=4),
        # long contexts with a distance bias on every token
        _attention("decode alibi 4x128K", "decode", 4, 131072, False, 1, 64, 8, 128, 16, E4M3,
                   TOKEN_HEAD, alibi=True),
        # a ragged batch of requests at different stages, static scales, capped scores
        _attention("decode ragged cap 64", "decode", 64, 32768, True, 1, 64, 8, 128, 32, E5M2,
                   CHANNEL_STATIC, cap=30.0, lens_seed=11),
        # a short prompt on an empty cache: latency
        _attention("prefill 1x200", "prefill", 1, 200, False, 200, 64, 8, 128, 16, E4M3,
                   TOKEN_HEAD),
        # one chunk of a long prompt after 14K cached tokens
        _attention("prefill 2048 of 16K", "prefill", 1, 16384, False, 2048, 64, 8, 128, 16, E4M3,
                   TOKEN_HEAD),
        # the same layer with capped scores over a window
        _attention("prefill cap window", "prefill", 1, 16384, False, 2048, 64, 8, 128, 16, E4M3,
                   TOKEN_HEAD, window=4096, cap=50.0),
        # many prompts of odd lengths in one batch, bidirectional prefix, small heads, INT8 codes
        _attention("prefill ragged prefix", "prefill", 21, 3000, True, 700, 16, 4, 64, 32, INT8,
                   TOKEN_HEAD, prefix=130, lens_seed=5),
        # a few draft tokens per request over long contexts, distance bias, MX block scales
        _attention("prefill short 8x32K", "prefill", 8, 32768, False, 16, 32, 8, 128, 64, E4M3,
                   MX_BLOCK, alibi=True),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32, 64])
    if op == "append":
        tokens = _spread(rng, 1, 12000)
        rot = rng.choice([d, d, d // 2, 32])
        fmt = rng.choice([E4M3, E5M2])
        return _append("", tokens, hkv * g, hkv, d, bs, fmt, rng.choice([TOKEN_HEAD,
                       CHANNEL_STATIC]), rot, rng.random() < 0.5, _spread(rng, 2000, 131072),
                       rng.random() < 0.5)
    fmt, mode = rng.choice([(E4M3, TOKEN_HEAD), (E5M2, CHANNEL_STATIC), (INT8, TOKEN_HEAD),
                            (E5M2, TOKEN_HEAD), (E4M3, MX_BLOCK)])
    kw = {"window": rng.choice([0, 0, _spread(rng, 1, 5000)]),
          "prefix": rng.choice([0, 0, _spread(rng, 1, 300)]),
          "cap": rng.choice([0.0, 0.0, rng.uniform(10.0, 60.0)]),
          "alibi": rng.random() < 0.3, "lens_seed": rng.randrange(1 << 20)}
    ragged = rng.random() < 0.6
    if op == "decode":
        batch = _spread(rng, 1, 64)
        length = _spread(rng, 1, min(131072, 400000 // batch))
        return _attention("", op, batch, length, ragged, 1, hkv * g, hkv, d, bs, fmt, mode, **kw)
    batch = _spread(rng, 1, 24)
    length = _spread(rng, 2, 16384 // batch)
    chunk = _spread(rng, 1, min(length, 2048))
    return _attention("", op, batch, length, ragged, chunk, hkv * g, hkv, d, bs, fmt, mode, **kw)


def _lengths(case):
    """Cached length (the chunk included) and chunk length of every request."""
    rng = random.Random(case["lens_seed"])
    lens = [_spread(rng, 1, case["length"]) if case["ragged"] else case["length"]
            for _ in range(case["batch"])]
    if case["op"] == "decode":
        return np.array(lens), np.ones(len(lens), dtype=np.int64)
    chunks = [min(n, _spread(rng, 1, case["chunk"]) if case["ragged"] else case["chunk"])
              for n in lens]
    return np.array(lens), np.array(chunks)


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _quantised(x, fmt, mode):
    """Codes and scales of float32 rows [blocks, heads, block, d], made for the inputs."""
    f = FMAX[fmt]
    if mode == MX_BLOCK:
        nb, h, bs, d = x.shape
        y = x.view(nb, h, bs, d // 32, 32)
        emax = 8 if fmt == E4M3 else 15
        e = torch.floor(torch.log2(y.abs().amax(-1).clamp_min(1e-30))) - emax
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


def _prepare_append(case, seed):
    g = _generator(seed)
    n, hq, hkv, d, bs = (case[k] for k in ("tokens", "hq", "hkv", "d", "bs"))
    wide = torch.randn(n, (hq + 2 * hkv) * d, device=DEV, generator=g).bfloat16()
    # q, k and v are slices of one fused projection's output
    q = wide[:, :hq * d].view(n, hq, d)
    k = wide[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    v = wide[:, (hq + hkv) * d:].view(n, hkv, d)
    nb = (2 * n + bs - 1) // bs + 1
    slots = torch.randperm(nb * bs, device=DEV, generator=g)[:n].int()
    if case["far"]:
        pos = torch.randint(case["max_pos"], (n,), device=DEV, generator=g).int()
    else:
        pos = (torch.arange(n, device=DEV) % case["max_pos"]).int()
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    angle = torch.arange(case["max_pos"], device=DEV, dtype=torch.float64)[:, None] * inv
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    kc = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device=DEV)
    if case["mode"] == CHANNEL_STATIC:
        ks = torch.rand(hkv, d, device=DEV, generator=g) * 4.0 / FMAX[case["fmt"]] + 1e-4
        vs = torch.rand(hkv, d, device=DEV, generator=g) * 4.0 / FMAX[case["fmt"]] + 1e-4
    else:
        ks = torch.zeros(nb, hkv, bs, 1, device=DEV)
        vs = torch.zeros_like(ks)
    return {"q": q, "k": k, "v": v, "pos": pos, "table": table, "slots": slots, "kc": kc,
            "vc": torch.zeros_like(kc), "ks": ks, "vs": vs, "q_out": torch.zeros(
                n, hq, d, dtype=torch.bfloat16, device=DEV)}


def _prepare_attention(case, seed):
    g = _generator(seed)
    hq, hkv, d, bs = (case[k] for k in ("hq", "hkv", "d", "bs"))
    lens, chunks = _lengths(case)
    pages = (lens + bs - 1) // bs
    nb = int(pages.sum())
    # physical blocks in a random order, unused table entries -1
    order = torch.randperm(nb, device=DEV, generator=g).int()
    col = torch.arange(int(pages.max()), device=DEV)[None]
    np_ = torch.from_numpy(pages).to(DEV)[:, None]
    first = torch.from_numpy(np.cumsum(pages) - pages).to(DEV)[:, None]
    tables = torch.where(col < np_, order[torch.clamp(first + col, max=nb - 1)], -1)
    # a few channels are larger than the rest, as keys' are
    gain = 1.0 + 3.0 * (torch.rand(hkv, 1, d, device=DEV, generator=g) < 0.03)
    kc, ks = _quantised(torch.randn(nb, hkv, bs, d, device=DEV, generator=g) * gain,
                        case["fmt"], case["mode"])
    vc, vs = _quantised(torch.randn(nb, hkv, bs, d, device=DEV, generator=g), case["fmt"],
                        case["mode"])
    q = torch.randn(int(chunks.sum()), hq, d, device=DEV, generator=g).bfloat16()
    offsets = np.concatenate([[0], np.cumsum(chunks)])
    slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq).float()
    prefix = torch.randint(case["prefix"] + 1, (len(lens),), device=DEV, generator=g).int()
    return {"q": q, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "tables": tables.int().contiguous(),
            "lens": torch.from_numpy(lens).int().to(DEV),
            "offsets": torch.from_numpy(offsets).int().to(DEV),
            "chunk": int(chunks.max()),
            "slopes": slopes if case["alibi"] else None,
            "prefix": prefix if case["prefix"] else None}


def prepare(case, seed):
    state = _prepare_append(case, seed) if case["op"] == "append" else _prepare_attention(
        case, seed)
    state["case"] = case
    return state


# ------------------------------------------------------------------ plain forms
def _rotated(x, cos, sin, case):
    """The first `rot` dims of float rows x [n, heads, d] turned by their tokens' angles."""
    rot, half = case["rot"], case["rot"] // 2
    c, s = cos[:, None], sin[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _stored(x, slots, cache, scale, case):
    """Quantise float rows [n, heads, d] and put them into their slots."""
    fmt, bs = case["fmt"], case["bs"]
    blk, off = slots.long() // bs, slots.long() % bs
    # a divisor on the device: every quotient is the rounded quotient
    fmax = torch.full((), FMAX[fmt], device=x.device, dtype=x.dtype).expand(x.shape[:2])[..., None]
    if case["mode"] == CHANNEL_STATIC:
        s = scale
    else:
        s = (x.abs().amax(-1, keepdim=True) / fmax).clamp_min(1e-12)
        scale[blk, :, off] = s
    codes = (x / s).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])
    cache[blk, :, off] = codes.view(torch.uint8)


def _plain_append(st, case):
    half = case["rot"] // 2
    row = st["table"][st["pos"].long()]
    cos, sin = row[:, :half], row[:, half:]
    st["q_out"].copy_(_rotated(st["q"].float(), cos, sin, case))
    _stored(_rotated(st["k"].float(), cos, sin, case), st["slots"], st["kc"], st["ks"], case)
    _stored(st["v"].float(), st["slots"], st["vc"], st["vs"], case)
    return _append_outputs(st, case)


def _append_outputs(st, case):
    out = {"q": st["q_out"], "k": st["kc"].view(F8[case["fmt"]]),
           "v": st["vc"].view(F8[case["fmt"]])}
    if case["mode"] == TOKEN_HEAD:
        out.update(k_scale=st["ks"], v_scale=st["vs"])
    return out


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


def _plain_attention(st, case):
    d, hq, hkv, cap = case["d"], case["hq"], case["hkv"], case["cap"]
    g = hq // hkv
    lens, offs, n = st["lens"].long(), st["offsets"].long(), st["chunk"]
    b = lens.numel()
    i = torch.arange(n, device=DEV)
    here = offs[:-1, None] + i  # row of query i of each request, past its chunk: any row
    held = i < (offs[1:] - offs[:-1])[:, None]
    q = st["q"][here.clamp_max(st["q"].shape[0] - 1)].float()  # [b, n, hq, d]
    q = q.view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    k = _values(st["kc"], st["ks"], st["tables"], case)
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).view(b, hkv, g, n, -1)
    del k
    if cap:
        z = z.div_(cap).tanh_().mul_(cap)
    pos = (lens - (offs[1:] - offs[:-1]))[:, None] + i  # a query's position in its request
    j = torch.arange(z.shape[-1], device=DEV)
    far = pos[:, :, None] - j  # [b, n, tokens]
    if st["slopes"] is not None:
        z = z.sub_(st["slopes"].view(1, hkv, g, 1, 1) * far[:, None, None].abs().float())
    see = far >= 0
    if case["window"]:
        see &= far < case["window"]
    if st["prefix"] is not None:
        see |= j < st["prefix"].long()[:, None, None]
    see &= j < lens[:, None, None]
    z = z.masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-1e30)
    p = z.sub_(top).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp_min(1e-30)).view(b, hkv, g * n, -1)
    o = torch.matmul(p, _values(st["vc"], st["vs"], st["tables"], case))
    o = o.view(b, hkv, g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    return o[held].bfloat16()


def run(state):
    st, case = state, state["case"]
    if not own:
        return _plain_append(st, case) if case["op"] == "append" else _plain_attention(st, case)
    import fp8_quantised_paged_gb300 as F
    kv = (st["kc"], st["vc"], st["ks"], st["vs"])
    form = {"fmt": case["fmt"], "scale_mode": case["mode"], "group_size": 32}
    if case["op"] == "append":
        F.kv_append_rope(st["q"], st["k"], st["v"], st["pos"], st["table"], st["slots"], *kv,
                         interleaved=case["interleaved"], q_out=st["q_out"], **form)
        return _append_outputs(st, case)
    mods = {"window": case["window"], "prefix_lens": st["prefix"], "logit_cap": case["cap"],
            "alibi_slopes": st["slopes"]}
    scale = case["d"] ** -0.5
    if case["op"] == "decode":
        return F.paged_decode_attention_mod(st["q"], *kv, st["tables"], st["lens"], case["hkv"],
                                            scale, **mods, **form)
    return F.paged_prefill_attention(st["q"], st["offsets"], *kv, st["tables"], st["lens"],
                                     case["hkv"], scale, **mods, **form)


# ------------------------------------------------------------------ what a pass needs
def _scale_bytes(case, rows):
    """Scale bytes of `rows` rows of one tensor, static scales counted once per head."""
    if case["mode"] == CHANNEL_STATIC:
        return case["hkv"] * case["d"] * 4
    return rows * (case["d"] // 32 if case["mode"] == MX_BLOCK else 4)


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        n = case["tokens"]
        rows = min(n, case["max_pos"])
        moved = n * (hq * d * 4 + 2 * hkv * d * 3 + 8) + rows * case["rot"] * 4
        moved += 2 * _scale_bytes(case, n * hkv)
        return {"bytes": moved, "flops": n * ((hq + hkv) * case["rot"] * 3 + 2 * hkv * d * 2)}
    lens, chunks = _lengths(case)
    seen = read = 0
    for n, m in zip(lens.tolist(), chunks.tolist()):
        pos = np.arange(n - m, n)
        first = np.maximum(pos - case["window"] + 1, 0) if case["window"] else 0 * pos
        # the mean always-visible prefix of a request, what the window leaves of it
        pre = min(case["prefix"] // 2, n)
        ahead = np.maximum(pre - pos - 1, 0)
        seen += int((pos - first + 1 + np.minimum(pre, first) + ahead).sum())
        read += int(n - first[0] + min(pre, first[0]))
    moved = read * hkv * d * 2 + 2 * _scale_bytes(case, read * hkv)
    moved += int(chunks.sum()) * hq * d * 4 + read // case["bs"] * 4
    return {"bytes": moved, "flops": 4 * d * hq * seen}


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


def _exact_attention(case, st):
    lens, chunks = _lengths(case)
    if 4 * case["d"] * case["hq"] * float((lens * chunks).sum()) > 6e12:
        return None  # minutes in 64 bits
    g = case["hq"] // case["hkv"]
    outs, row = [], 0
    for b, (n, m) in enumerate(zip(lens.tolist(), chunks.tolist())):
        blocks = st["tables"][b, :(n + case["bs"] - 1) // case["bs"]].long()
        k = _exact_values(st["kc"], st["ks"], blocks, case)[:, :n]
        v = _exact_values(st["vc"], st["vs"], blocks, case)[:, :n]
        dist = torch.arange(n - m, n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None]
        see = dist >= 0
        if case["window"]:
            see = see & (dist < case["window"])
        if st["prefix"] is not None:
            see = see | (torch.arange(n, device=DEV)[None] < int(st["prefix"][b]))
        o = torch.empty(m, case["hq"], case["d"], dtype=torch.float64, device=DEV)
        for h in range(case["hq"]):
            z = st["q"][row:row + m, h].double() @ k[h // g].T / math.sqrt(case["d"])
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if st["slopes"] is not None:
                z = z - st["slopes"][h].double() * dist.abs()
            z = torch.where(see, z, -math.inf)
            o[:, h] = torch.softmax(z, -1) @ v[h // g]
        outs.append(o)
        row += m
    return torch.cat(outs)


def _exact_rows(x, static, case):
    """Scales of 64-bit rows and the values their codes stand for (without the scale)."""
    top = FMAX[case["fmt"]]
    s = static.double() if case["mode"] == CHANNEL_STATIC else (
        x.abs().amax(-1, keepdim=True) / top).clamp_min(1e-12)
    z = (x / s).clamp(-top, top)
    mant, low = (3, -6) if case["fmt"] == E4M3 else (2, -14)
    e = torch.floor(torch.log2(z.abs().clamp_min(1e-300))).clamp_min(low) - mant
    return s, (torch.round(z * torch.exp2(-e)) * torch.exp2(e)).clamp(-top, top)


def _exact_append(case, st):
    half, rot = case["rot"] // 2, case["rot"]
    first = torch.arange(half, device=DEV) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    cs = st["table"][st["pos"].long()].double()
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]

    def rotate(x):
        y = x.double().clone()
        w = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = w.real, w.imag
        return y

    assert rot <= case["d"]
    slots = st["slots"].long()
    out = {"q": rotate(st["q"])}
    for name, x, static in (("k", rotate(st["k"]), st["ks"]), ("v", st["v"].double(), st["vs"])):
        s, z = _exact_rows(x, static, case)
        shape = st["kc"].shape
        rows = torch.zeros(shape[0] * shape[2], shape[1], shape[3], dtype=torch.float64,
                           device=DEV)
        rows[slots] = z
        out[name] = rows.view(shape[0], shape[2], shape[1], shape[3]).transpose(1, 2)
        if case["mode"] == TOKEN_HEAD:
            rows = torch.zeros(shape[0] * shape[2], shape[1], 1, dtype=torch.float64, device=DEV)
            rows[slots] = s
            out[name + "_scale"] = rows.view(shape[0], shape[2], shape[1], 1).transpose(1, 2)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(case, st) if case["op"] == "append" else _exact_attention(case, st)
