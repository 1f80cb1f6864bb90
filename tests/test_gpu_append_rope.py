"""The append with rotary positions: codes, scales and turned queries equal the
stated fp32 formulas bit for bit, on contiguous and strided rows, in every
scale mode, and tokens that are to be left alone are."""
import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def F():
    import fp8_quantised_paged_gb300 as F
    torch.cuda.set_device(0)
    F.get_device_error()
    return F


def table(max_pos, rot, base=10000.0):
    half = rot // 2
    inv = base ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def inputs(n, hq, hkv, d, rot, max_pos=500, seed=0, strided=False, with_v=True):
    g = torch.Generator().manual_seed(seed)
    pad = 8 if strided else 0
    wide = torch.randn(n, (hq + 2 * hkv) * d + pad, generator=g)
    wide[:, ::17] *= 20.0
    wide = wide.bfloat16()
    q = wide[:, :hq * d].unflatten(1, (hq, d))
    k = wide[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = wide[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d)) if with_v else None
    if not strided:
        q, k = q.contiguous(), k.contiguous()
        v = None if v is None else v.contiguous()
    pos = torch.randint(max_pos, (n,), generator=g).int()
    return q, k, v, pos, table(max_pos, rot)


def scale_tensor(nb, hkv, bs, d, mode, gs):
    if mode == R.MX:
        return torch.full((nb, hkv, bs, d // gs), 77, dtype=torch.uint8, device=DEV)
    groups = d // gs if mode == R.GROUP else 1
    return torch.full((nb, hkv, bs, groups), 7.5, device=DEV)


def run_case(F, n, hq, hkv, d, bs, fmt, mode, rot, offset=0, interleaved=False, gs=64,
             strided=False, with_v=True, seed=0):
    q, k, v, pos, cs = inputs(n, hq, hkv, d, rot, seed=seed, strided=strided, with_v=with_v)
    rng = np.random.default_rng(seed)
    nb = (n + bs - 1) // bs + 2
    slots = torch.from_numpy(rng.permutation(nb * bs)[:n].astype(np.int32))
    if n > 3:
        slots[n // 2] = -1
    kc = torch.full((nb, hkv, bs, d), 3, dtype=torch.uint8, device=DEV)
    vc = kc.clone() if with_v else None
    static = None
    if mode == R.STATIC:
        static = torch.from_numpy(np.exp(rng.normal(-4, 1, (hkv, d))).astype(np.float32))
        ks, vs = static.to(DEV), static.to(DEV)
    else:
        ks = scale_tensor(nb, hkv, bs, d, mode, gs)
        vs = ks.clone()
    dev = lambda t: None if t is None else (  # noqa: E731
        torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV).copy_(t))
    if strided:  # slices of one device buffer
        base = torch.zeros(n, q.stride(0), dtype=torch.bfloat16, device=DEV)
        wide = torch.cat([q.flatten(1), k.flatten(1)] + ([v.flatten(1)] if with_v else []), 1)
        base[:, :wide.shape[1]] = wide.to(DEV)
        qd = base[:, :hq * d].unflatten(1, (hq, d))
        kd = base[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        vd = base[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d)) if with_v else None
    else:
        qd, kd, vd = dev(q), dev(k), dev(v)
    out = F.kv_append_rope(qd, kd, vd, pos.to(DEV), cs.to(DEV), slots.to(DEV), kc, vc, ks,
                           vs if with_v else None, rot_offset=offset, interleaved=interleaved,
                           fmt=fmt, scale_mode=mode, group_size=gs)
    torch.cuda.synchronize()
    assert F.get_device_error() == 0
    half = rot // 2
    cos, sin = cs[pos.long()][:, :half], cs[pos.long()][:, half:]
    want_q = R.rotate(q, cos, sin, offset, interleaved).bfloat16()
    assert torch.equal(out.cpu().view(torch.int16), want_q.view(torch.int16))
    keep = slots >= 0
    blk, off = slots[keep].long() // bs, slots[keep].long() % bs
    for x, cache, scale, rope in ((k, kc, ks, True), (v, vc, vs, False)):
        if x is None:
            continue
        x32 = R.rotate(x, cos, sin, offset, interleaved) if rope else x.float()
        codes, s = R.encode_rows(x32, fmt, mode, gs, static)
        want = torch.full_like(kc, 3).cpu()
        want[blk, :, off] = codes[keep]
        assert torch.equal(cache.cpu(), want)
        if s is not None:
            want_s = scale_tensor(nb, hkv, bs, d, mode, gs).cpu()
            want_s[blk, :, off] = s[keep]
            assert torch.equal(scale.cpu(), want_s)


MODES = [(R.E4M3, R.TOKEN_HEAD, 64), (R.E5M2, R.TOKEN_HEAD, 64), (R.INT8, R.TOKEN_HEAD, 64),
         (R.E4M3, R.STATIC, 64), (R.E5M2, R.GROUP, 64), (R.INT8, R.GROUP, 32),
         (R.E4M3, R.MX, 32), (R.E5M2, R.MX, 16)]


@pytest.mark.parametrize("fmt,mode,gs", MODES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_formats_and_scale_modes(F, fmt, mode, gs, interleaved):
    run_case(F, 37, 8, 2, 128, 16, fmt, mode, 128, interleaved=interleaved, gs=gs)


@pytest.mark.parametrize("n,hq,hkv,d,bs,rot,offset", [
    (1, 1, 1, 64, 16, 64, 0), (1, 64, 8, 128, 16, 128, 0), (5, 3, 1, 128, 7, 64, 0),
    (33, 5, 5, 64, 32, 32, 16), (2, 7, 1, 96, 16, 48, 8), (9, 4, 2, 256, 16, 256, 0),
    (17, 12, 3, 48, 16, 16, 32), (4, 2, 1, 16, 16, 16, 0), (1300, 12, 3, 128, 16, 96, 0),
    (1025, 16, 4, 64, 64, 64, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_shapes_partial_ranges_and_bulk(F, n, hq, hkv, d, bs, rot, offset, interleaved):
    run_case(F, n, hq, hkv, d, bs, R.E4M3, R.TOKEN_HEAD, rot, offset, interleaved, seed=n)


@pytest.mark.parametrize("interleaved", [False, True])
def test_latent_rows_turn_their_last_64_dims(F, interleaved):
    run_case(F, 21, 16, 1, 576, 64, R.E4M3, R.GROUP, 64, 512, interleaved, with_v=False)


@pytest.mark.parametrize("n", [3, 700])
def test_strided_rows_of_a_fused_projection(F, n):
    run_case(F, n, 24, 4, 128, 16, R.E4M3, R.TOKEN_HEAD, 128, strided=True)


def test_in_place_and_without_queries(F):
    q, k, v, pos, cs = inputs(50, 6, 2, 128, 128)
    qd = q.to(DEV)
    kc = torch.zeros(4, 2, 16, 128, dtype=torch.uint8, device=DEV)
    vc, ks = torch.zeros_like(kc), torch.zeros(4, 2, 16, 1, device=DEV)
    vs = torch.zeros_like(ks)
    slots = torch.arange(50, dtype=torch.int32, device=DEV)
    args = (k.to(DEV), v.to(DEV), pos.to(DEV), cs.to(DEV), slots)
    out = F.kv_append_rope(qd, *args, kc, vc, ks, vs, q_out=qd)
    assert out.data_ptr() == qd.data_ptr()
    want = R.rotate(q, cs[pos.long()][:, :64], cs[pos.long()][:, 64:]).bfloat16()
    assert torch.equal(qd.cpu(), want)
    kc2, vc2, ks2, vs2 = (torch.zeros_like(t) for t in (kc, vc, ks, vs))
    assert F.kv_append_rope(None, *args, kc2, vc2, ks2, vs2) is None
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    assert torch.equal(ks, ks2) and torch.equal(vs, vs2)


def test_padding_and_bad_tokens_are_left_alone(F):
    n = 8
    q, k, v, pos, cs = inputs(n, 4, 2, 64, 64)
    pos[1], pos[2], pos[3] = -1, 500, 2 ** 31 - 1   # outside the table
    slots = torch.arange(n, dtype=torch.int32)
    slots[1] = -1                                   # padding: no flag by itself
    slots[5] = 16 * 3 + 1                           # past the pool
    slots[6] = -7                                   # cache alone, q turned
    kc = torch.full((3, 2, 16, 64), 9, dtype=torch.uint8, device=DEV)
    vc, ks = kc.clone(), torch.full((3, 2, 16, 1), 2.0, device=DEV)
    vs = ks.clone()
    mark = torch.full((n, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    F.kv_append_rope(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), cs.to(DEV), slots.to(DEV), kc,
                     vc, ks, vs, q_out=mark)
    from fp8_quantised_paged_gb300 import _native as N
    assert F.get_device_error() == N.DEVERR_POSITION | N.DEVERR_SLOT_RANGE
    ok = [0, 4, 5, 6, 7]
    sel = pos[ok].long()
    want = torch.full((n, 4, 64), 5.0).bfloat16()
    want[ok] = R.rotate(q[ok], cs[sel][:, :32], cs[sel][:, 32:]).bfloat16()
    assert torch.equal(mark.cpu(), want)
    written = (kc.cpu() != 9).flatten(3).any(-1).any(1)  # [block, offset]
    assert written.nonzero().tolist() == [[0, 0], [0, 4], [0, 7]]
    assert (vs.cpu() != 2.0).sum().item() == 3 * 2
    # padding alone raises nothing
    F.kv_append_rope(q[1:2].to(DEV), k[1:2].to(DEV), v[1:2].to(DEV), pos[1:2].to(DEV),
                     cs.to(DEV), slots[1:2].to(DEV), kc, vc, ks, vs)
    assert F.get_device_error() == 0


def test_no_tokens(F):
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    kc = torch.zeros(1, 2, 16, 64, dtype=torch.uint8, device=DEV)
    ks = torch.zeros(1, 2, 16, 1, device=DEV)
    out = F.kv_append_rope(e, e, e, i, torch.zeros(4, 64, device=DEV), i, kc, kc, ks, ks)
    assert out.shape == (0, 2, 64)


def test_other_stream_and_graph(F):
    q, k, v, pos, cs = inputs(70, 8, 2, 128, 128)
    kc = torch.zeros(5, 2, 16, 128, dtype=torch.uint8, device=DEV)
    bufs = [kc, torch.zeros_like(kc), torch.zeros(5, 2, 16, 1, device=DEV),
            torch.zeros(5, 2, 16, 1, device=DEV)]
    want = [t.clone() for t in bufs]
    args = [t.to(DEV) for t in (q, k, v, pos, cs, torch.arange(70, dtype=torch.int32))]
    wq = F.kv_append_rope(*args, *want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = F.kv_append_rope(*args, *bufs, stream=side)
    side.synchronize()
    assert torch.equal(got, wq) and all(torch.equal(a, b) for a, b in zip(bufs, want))
    for t in bufs:
        t.zero_()
    out = torch.zeros_like(wq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.kv_append_rope(*args, *bufs, q_out=out)
    assert not out.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, wq) and all(torch.equal(a, b) for a, b in zip(bufs, want))
