"""A plain 64-bit reference of tree attention over the paged cache.

Tolerances (stated before any run).  With A = sum_j p_j |v^_j| and Z, B as at the head of
serving_ref.py, an output element may be off by

  A * (2 dz + r) + W + half a bf16 step of the result (bf16 outputs).

dz, the error of a score: accumulation, scale, cap, bias and exponent as there,
  (D / 16 + 4) 2^-22 Z + 4 2^-22 B + 2^-20 cap (caps up to 64);
q is taken as two E4M3 terms hi + lo of q c, c the power of two that puts the row's largest
element into [2^7, 2^8).  hi is off by at most 2^(e - 4) of an element of exponent e, and an
element of bf16 is a multiple of 2^(e - 7), so that lo, at most 8 such steps, is exact while
these are multiples of 2^-9, E4M3's smallest: elements below 2^-2 / c are off by at most
2^-10 / c, 2^-17 of the largest:
  sm_scale 2^-17 max_d |q_d| sum_d |k^_d|.
With static channel scales q times the scales (rounded to fp32) has no such steps: lo rounds
what hi leaves, at most 2^(e - 4), by 2^-5 of that (half a step of E4M3 in the binade
below): 2^-9 of each element more, 2^-9 Z.  Codes that no E4M3 or E5M2 product takes (INT8,
MX blocks) meet q as f16, 2^-11 Z (it is exact for all but elements 2^-17 below the
largest, as there), and their K^ is exact in f16 but for small factors (see W).
r: 2^-19 as there, and 2^-11 for the softmax weights, which enter the second product as f16
times V's scale.
W: a weight times V's scale, relative to the largest scale of its group of 32 tokens, is
below f16's normal range off by 2^-25: 2^-36 vs_max sum_j |code_j| as there.  V^ of MX blocks
is a code times its block's factor relative to the token's largest, and K^ likewise.  An
E4M3 code (at most 448 < 2^9) leaves f16 (2^16) seven exponents, by which the factor is raised:
half of f16's smallest step, 2^-25, is then 2^-32 of the largest factor, and 2^-31 is allowed.
An E5M2 code (at most 57344) leaves none: half a step is 2^-25 of it.
"""
import numpy as np
import torch

from serving_ref import MX, STATIC, half_step_bf16


def lines(parents):
    """The nodes on every node's line, itself last; a parent out of order counts as -1."""
    out = []
    for i, p in enumerate(parents):
        p = int(p)
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def tree_ref(q, offsets, parents, lens, bt, values, hkv, sm, bs, fmt, mode, window=0, prefix=None,
             cap=0.0, slopes=None, kchan=None, device="cpu"):
    """Reference rows and what the tolerance is made of.  values: chunk_values' (K, V, V's
    code values, both token scales); kchan: the channels' scales of K, where they are static."""
    kd, vd, vcode, vscale, kscale = (x.to(device) for x in values)
    n, hq, d = q.shape
    g = hq // hkv
    q = q.double().to(device)
    f16_k = fmt == 2 or mode == MX
    mx_step = 2.0 ** -25 if fmt == 1 else 2.0 ** -31
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=device)
    A, Z, Bm = torch.zeros_like(out), torch.zeros_like(out[..., :1]), torch.zeros_like(out[..., :1])
    W, Fl = torch.zeros_like(out), torch.zeros_like(Z)
    for b in range(len(lens)):
        lo, hi, L = int(offsets[b]), int(offsets[b + 1]), int(lens[b])
        m = hi - lo
        if m <= 0 or L < m:
            continue
        ctx = L - m
        line = lines(parents[lo:hi])
        see = torch.zeros(m, L, dtype=torch.bool)
        place = torch.arange(L)
        for i, nodes in enumerate(line):
            place[ctx + i] = ctx + len(nodes) - 1
            see[i, [ctx + x for x in nodes]] = True
        dist = place[ctx:, None] - place[None]
        see[:, :ctx] = True
        if window:
            near = dist < window
            if prefix is not None:
                near[:, :min(max(int(prefix[b]), 0), ctx)] = True
            see &= near
        see, dist = see.to(device), dist.to(device).double()
        blk = bt[b, :(L + bs - 1) // bs].long().to(device)
        k, v, vcd, vsc, ksc = (x[blk].permute(1, 0, 2, 3).flatten(1, 2)[:, :L]
                               for x in (kd, vd, vcode, vscale, kscale))
        for h in range(hq):
            kk = torch.where(torch.isfinite(k[h // g]), k[h // g], 0.0)
            vv = torch.where(torch.isfinite(v[h // g]), v[h // g], 0.0)
            z = sm * (q[lo:hi, h] @ kk.T)
            zabs = abs(sm) * (q[lo:hi, h].abs() @ kk.abs().T)
            if cap:
                z = cap * torch.tanh(z / cap)
            bias = (0.0 if slopes is None else float(slopes[h])) * dist.abs()
            z = torch.where(see, z - bias, -torch.inf)
            near = see & (z > z.amax(1, keepdim=True) - 60)
            p = torch.softmax(z, 1)
            out[lo:hi, h] = p @ vv
            A[lo:hi, h] = p @ vv.abs()
            Z[lo:hi, h, 0] = torch.where(see, zabs, 0.0).amax(1)
            Bm[lo:hi, h, 0] = Z[lo:hi, h, 0] + torch.where(near, bias, 0.0).amax(1)
            some = see.any(0)
            top = float(vsc[h // g][some].max())
            codes = torch.where(torch.isfinite(vcd[h // g]), vcd[h // g], 0.0).abs()
            W[lo:hi, h] = top * 2.0 ** -36 * (see.double() @ codes)
            if mode == MX:
                W[lo:hi, h] += top * mx_step
            if mode == STATIC:
                ks = kchan.double().to(device)[h // g]
                codes = torch.where(ks > 0, kk / ks, 0.0).abs().sum(1)
                Fl[lo:hi, h, 0] = 2.0 ** -9 * Z[lo:hi, h, 0] + abs(sm) * 2.0 ** -17 * (
                    q[lo:hi, h].abs() * ks).amax(1) * float(codes[some].max())
            elif f16_k:
                Fl[lo:hi, h, 0] = 2.0 ** -11 * Z[lo:hi, h, 0]
                if mode == MX:
                    Fl[lo:hi, h, 0] += abs(sm) * q[lo:hi, h].abs().sum(1) * mx_step * float(
                        ksc[h // g][some].max())
            else:
                Fl[lo:hi, h, 0] = abs(sm) * 2.0 ** -17 * q[lo:hi, h].abs().amax(1) * float(
                    kk[some].abs().sum(1).max())
    return tuple(x.cpu().numpy() for x in (out, A, Z, Bm, W, Fl))


def check_tree(got, ref, d, bf16=False, cap=0.0, what=""):
    """Hold `got` to the bound at the head of this file."""
    want, A, Z, B, W, Fl = ref
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    dz = (d / 16 + 4) * 2.0 ** -22 * Z + 4 * 2.0 ** -22 * B + Fl
    if cap <= 64:
        dz = dz + 2.0 ** -20 * cap
    bound = A * (2 * dz + 2.0 ** -19 + 2.0 ** -11) + 1e-30 + W
    if bf16:
        bound = bound + half_step_bf16(np.abs(want) + bound)
    over = np.abs(got - want) / bound
    worst = float(over.max()) if over.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound at {np.unravel_index(over.argmax(), over.shape)}"
    return worst
