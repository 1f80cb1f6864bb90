"""Plain 64-bit references of the rotary append and of attention with score
modifiers, and the caches their tests run on.

Tolerances (stated before any run).  With A_i[d] = sum_j p_ij |v^_j[d]| the
attention of |v^|, an output element may be off by

  A * (2 dz + r) + half a bf16 step of the result (bf16 outputs),

dz the error of a score: its dot product accumulates D products in fp32 (at
most (D / 16 + 4) sums of relative error 2^-22, a tensor-core step of 16 being
one sum), of magnitude at most Z = sm_scale * sum_d |q_d k^_d|, and every later
operation (scale, cap, bias, exponent) rounds a value of at most
B = Z + |bias| by 2^-22.  Both p and the sum that divides it carry e^dz, hence
the factor 2.  r collects what is relative to p: 2^-19 for exponent, scale and
sums in fp32.

The prefill (`half`) adds f16 roundings of half a step, 2^-11: of P (r), of V^
(r, where scales are per token or segment), and of K^ or of q with static channel
scales in it (2^-11 Z in dz; MX scales are exact).  Below f16's normal range
(2^-14) a rounding is off by up to 2^-25 instead:
 - K^ holds code * ks / 2^e with 2^e at most twice the largest ks of its group:
   sm_scale * sum_d |q_d| * 2^-24 ks_max more in dz (F);
 - V^ likewise: 2^-24 vs_max more in the output;
 - P = 2^(z - ref + 12 + e), ref <= max z + e_max, so the sum it is divided by is
   at least 2^(12 - e_max) >= 2^11 / vs_max, and every visible token adds at most
   2^-25 |code_jd| vs_max / 2^11: 2^-36 vs_max sum_j |code_jd| in all (times the
   channel's scale where scales are static).
W is the sum of the last two; vs_max and ks_max are taken over the request.

A cap of at most 64 may take tanh as 1 - 2 / (e^2x + 1), whose quotient is good to
2^-21: 2^-20 cap more in dz.
"""
from __future__ import annotations

import numpy as np
import torch

E4M3, E5M2, INT8 = 0, 1, 2
TOKEN_HEAD, STATIC, GROUP, MX, SEGMENT = 0, 1, 2, 3, 4
FMAX = {E4M3: 448.0, E5M2: 57344.0, INT8: 127.0}
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}


# ------------------------------------------------------------------ codec
def decode_codes(codes, fmt):
    """uint8 codes -> float64 values."""
    if fmt == INT8:
        return codes.double() - 128.0
    return codes.view(F8[fmt]).double()


def dequant(codes, scale, fmt, mode, gs):
    """[nb, hkv, bs, d] codes with their scales -> float64 values."""
    x = decode_codes(codes, fmt)
    nb, h, bs, d = x.shape
    if mode == STATIC:
        return x * scale.double().view(1, h, 1, d)
    if mode == SEGMENT:
        return x * scale.double()[:, :h].view(nb, h, 1, 1)
    if mode in (GROUP, MX):
        s = scale.view(nb, h, bs, d // gs)
        s = torch.exp2(s.double() - 127.0) if mode == MX else s.double()
        return x * s.repeat_interleave(gs, -1)
    return x * scale.double().view(nb, h, bs, 1)


def encode_rows(x, fmt, mode, gs=64, static=None):
    """float32 rows [n, h, d] -> (codes uint8, scales) by the stated fp32 formulas."""
    x = x.float()
    n, h, d = x.shape
    top = torch.full((1,), FMAX[fmt], dtype=torch.float32)
    if mode == STATIC:
        s, full = None, static.view(1, h, d).expand(n, h, d)
        q = x / full
    elif mode == MX:
        m = x.abs().view(n, h, d // gs, gs).amax(-1)
        ef = (m.view(torch.int32) >> 23) & 0xFF
        e = torch.where(ef == 0, -127, (ef - 127 - (8 if fmt == E4M3 else 15)).clamp(-127, 127))
        s = (e + 127).to(torch.uint8)
        q = (x.double() * torch.exp2(-e.double()).repeat_interleave(gs, -1)).float()
    else:
        g = gs if mode == GROUP else d
        m = x.abs().view(n, h, d // g, g).amax(-1)
        s = torch.maximum(m / top, torch.full((1,), 1e-12))
        q = x / s.repeat_interleave(g, -1)
    if fmt == INT8:
        codes = (q.clamp(-127, 127).round() + 128).to(torch.uint8)
    else:
        codes = q.clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)
    return codes, s


def rotate(x, cos, sin, offset=0, interleaved=False):
    """float32 rows [n, h, d] turned by cos/sin [n, rot / 2]; every operation rounds to fp32."""
    x = x.float().clone()
    half = cos.shape[1]
    c, s = cos.float()[:, None], sin.float()[:, None]
    r = x[..., offset:offset + 2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    p, q = a * c - b * s, b * c + a * s
    x[..., offset:offset + 2 * half] = (torch.stack([p, q], -1).flatten(-2) if interleaved
                                        else torch.cat([p, q], -1))
    return x


# ------------------------------------------------------------------ caches
def make_cache(rng, nb, hkv, bs, d, fmt, mode, gs=32):
    """Random codes of every finite kind and scales over three decades."""
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a))  # noqa: E731
    out = []
    for _ in range(2):
        x = rng.standard_normal((nb, hkv, bs, d)) * np.exp(rng.normal(0, 0.5, (nb, hkv, bs, 1)))
        if fmt == INT8:
            codes = t(np.clip(np.rint(x * 40), -127, 127) + 128).to(torch.uint8)
            unit = 1 / 40
        else:
            top = 100.0 if fmt == E4M3 else 3000.0
            codes = t(np.clip(x * top, -FMAX[fmt], FMAX[fmt])).float().to(F8[fmt])
            codes = codes.view(torch.uint8)
            unit = 1 / top
        if mode == STATIC:
            s = t((unit * np.exp(rng.normal(0, 0.7, (hkv, d)))).astype(np.float32))
        elif mode == SEGMENT:
            s = t((unit * np.exp(rng.normal(0, 0.3, (nb, (hkv + 3) // 4 * 4)))).astype(np.float32))
        elif mode == MX:
            base = int(round(np.log2(unit))) + 127
            s = t(rng.integers(base - 2, base + 3, (nb, hkv, bs, d // gs)).astype(np.uint8))
        else:
            s = t((unit * np.exp(rng.normal(0, 0.5, (nb, hkv, bs, 1)))).astype(np.float32))
        out.append((codes, s))
    (kc, ks), (vc, vs) = out
    return kc, vc, ks, vs


def make_tables(rng, lens, bs, spare=3):
    """Block tables over a shuffled pool (unused entries -1) and the pool's size."""
    pages = [(int(n) + bs - 1) // bs for n in lens]
    order = rng.permutation(sum(pages) + spare)
    bt = np.full((len(lens), max(1, max(pages) + 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(bt), len(order)


# ------------------------------------------------------------------ attention
def attention_row(q, k, v, pos, prefix, sm, window=0, cap=0.0, slope=0.0):
    """One query q [d] at `pos` over k, v [L, d] (float64): the output, A and dz's
    two magnitudes (Z, B) over the visible tokens."""
    L = k.shape[0]
    j = torch.arange(L)
    see = j <= pos
    if window:
        see &= pos - j < window
    see |= j < prefix
    if not bool(see.any()):
        z0 = torch.zeros(k.shape[1], dtype=torch.float64)
        return z0, z0, 0.0, 0.0
    k, v, j = k[see], v[see], j[see]
    z = sm * (k @ q)
    zabs = float((abs(sm) * (k.abs() @ q.abs())).max())
    if cap:
        z = cap * torch.tanh(z / cap)
    bias = slope * (pos - j).abs().double()
    z = z - bias
    # a token far down the exponent has no weight, whatever its bias rounds to
    near = z > z.max() - 60
    b = zabs + float(bias[near].abs().max())
    p = torch.softmax(z, 0)
    return p @ v, p @ v.abs(), zabs, b


def attention_ref(q, rows, chunk_of, lens, bt, values, hkv, sm, bs, window=0, prefix=None,
                  cap=0.0, slopes=None):
    """Reference rows: q [n, hq, d]; row i belongs to request rows[i] at position
    chunk_of[i].  Returns out, A, Z, B as numpy [n, hq, d] / [n, hq, 1], and no W and F."""
    kd, vd = values
    n, hq, d = q.shape
    g = hq // hkv
    q = q.double()
    out = np.zeros((n, hq, d))
    A, Z, Bm = np.zeros((n, hq, d)), np.zeros((n, hq, 1)), np.zeros((n, hq, 1))
    cache = {}
    for i in range(n):
        b = int(rows[i])
        L = int(lens[b])
        if b not in cache:
            blk = bt[b, :(L + bs - 1) // bs].long()
            cache = {b: tuple(x[blk].permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :L]
                              for x in (kd, vd))}
        k, v = cache[b]
        pre = 0 if prefix is None else min(max(int(prefix[b]), 0), L)
        for h in range(hq):
            o, a, z, bm = attention_row(q[i, h], k[h // g], v[h // g], int(chunk_of[i]), pre, sm,
                                        window, cap, 0.0 if slopes is None else float(slopes[h]))
            out[i, h], A[i, h], Z[i, h], Bm[i, h] = o.numpy(), a.numpy(), z, bm
    return out, A, Z, Bm, 0.0, 0.0


def half_step_bf16(x):
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
    return np.exp2(e - 8)


def check(got, ref, d, bf16=False, half=None, cap=0.0, what=""):
    """Hold `got` to the bound at the head of this file; half: the scale mode of a
    prefill (None: a decode)."""
    want, A, Z, B, W, Fl = ref
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    dz = (d / 16 + 4) * 2.0 ** -22 * Z + 4 * 2.0 ** -22 * B
    r = 2.0 ** -19
    if cap <= 64:
        dz = dz + 2.0 ** -20 * cap
    if half is not None:
        dz = dz + (2.0 ** -11 * Z if half != MX else 0.0) + Fl
        r += 2.0 ** -11 * (2 if half in (TOKEN_HEAD, SEGMENT) else 1)
    bound = A * (2 * dz + r) + 1e-30 + (W if half is not None else 0.0)
    if bf16:
        bound = bound + half_step_bf16(np.abs(want) + bound)
    over = np.abs(got - want) / bound
    worst = float(over.max()) if over.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound at {np.unravel_index(over.argmax(), over.shape)}"
    return worst


def chunk_ref(q, offsets, lens, bt, values, hkv, sm, bs, window=0, prefix=None, cap=0.0,
              slopes=None, device="cpu"):
    """attention_ref for ragged chunks: request b's queries are rows offsets[b] ..
    offsets[b + 1] - 1, the last one at position lens[b] - 1.  values: K, V, and
    V's code values (channel scales in), and both token scales (for W and F)."""
    kd, vd, vcode, vscale, kscale = (x.to(device) for x in values)
    n, hq, d = q.shape
    g = hq // hkv
    q = q.double().to(device)
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=device)
    A, Z, Bm = torch.zeros_like(out), torch.zeros_like(out[..., :1]), torch.zeros_like(out[..., :1])
    W, Fl = torch.zeros_like(out), torch.zeros_like(Z)
    for b in range(len(lens)):
        lo, hi, L = int(offsets[b]), int(offsets[b + 1]), int(lens[b])
        if hi <= lo or L == 0:
            continue
        blk = bt[b, :(L + bs - 1) // bs].long().to(device)
        k, v, vcd, vsc, ksc = (x[blk].permute(1, 0, 2, 3).flatten(1, 2)[:, :L]
                               for x in (kd, vd, vcode, vscale, kscale))
        pos = torch.arange(L - (hi - lo), L, device=device)[:, None]
        j = torch.arange(L, device=device)[None]
        see = j <= pos
        if window:
            see = see & (pos - j < window)
        if prefix is not None:
            see = see | (j < min(max(int(prefix[b]), 0), L))
        live = see.any(1, keepdim=True)
        for h in range(hq):
            z = sm * (q[lo:hi, h] @ k[h // g].T)
            zabs = abs(sm) * (q[lo:hi, h].abs() @ k[h // g].abs().T)
            if cap:
                z = cap * torch.tanh(z / cap)
            bias = (0.0 if slopes is None else float(slopes[h])) * (pos - j).abs().double()
            z = torch.where(see, z - bias, -torch.inf)
            near = see & (z > z.amax(1, keepdim=True) - 60)
            p = torch.where(live, torch.softmax(z, 1), 0.0)
            out[lo:hi, h] = p @ v[h // g]
            A[lo:hi, h] = p @ v[h // g].abs()
            Z[lo:hi, h, 0] = torch.where(see, zabs, 0.0).amax(1)
            Bm[lo:hi, h, 0] = Z[lo:hi, h, 0] + torch.where(near, bias.abs(), 0.0).amax(1)
            top = float(vsc[h // g].max())
            W[lo:hi, h] = top * (2.0 ** -36 * (see.double() @ vcd[h // g].abs()) + 2.0 ** -24)
            Fl[lo:hi, h, 0] = abs(sm) * q[lo:hi, h].abs().sum(1) * 2.0 ** -24 * float(
                ksc[h // g].max())
    return tuple(x.cpu().numpy() for x in (out, A, Z, Bm, W, Fl))


def chunk_values(cache, fmt, mode, gs):
    """The `values` of chunk_ref for a cache."""
    kc, vc, ks, vs = cache
    x = decode_codes(vc, fmt)
    nb, h, bs, d = x.shape
    if mode == STATIC:
        x = x * vs.double().view(1, h, 1, d)

    def per_token(s):
        if mode == STATIC:
            return torch.ones(nb, h, bs, 1, dtype=torch.float64, device=x.device)
        if mode == SEGMENT:
            return s[:, :h].double().view(nb, h, 1, 1).expand(nb, h, bs, 1)
        if mode == MX:
            return torch.exp2(s.view(nb, h, bs, d // gs).double().amax(-1, keepdim=True) - 127.0)
        return s.double().view(nb, h, bs, 1)

    return (dequant(kc, ks, fmt, mode, gs), dequant(vc, vs, fmt, mode, gs), x, per_token(vs),
            per_token(ks))
