"""Ragged batches on the GPU: csa2_kv_append_ragged against the oracle's appends
(bytes), csa2_kv_read / csa2_window_read against the planes' bytes decoded in
64 bits (exact), csa2_chunk_attn against a plain 64-bit form, and the calls
together as a serving loop makes them."""
import math

import numpy as np
import pytest
import torch

import ragged_util as ru
from fp4_compressed_sparse_gb300 import csa2
from fp4_compressed_sparse_gb300 import workloads as wl
from gpu_util import assert_cache_equal, attn_close, cmp_rows, u16

pytestmark = pytest.mark.gpu
THETA = 10000.0
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp4_compressed_sparse_gb300 import build_lib
    build_lib.build()
    csa2.load()


def _cu(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _cache(batch, cap, ratio=1, swa=csa2.SWA_MXFP8, page=None, fmt=csa2.ENTRY_FP4, seed=0):
    if not page:
        return csa2.Cache(batch, cap, ratio=ratio, swa_dtype=swa, entry_format=fmt)
    cap = -(-cap // page) * page
    per = cap // page
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(batch * per + 4, generator=g)[:batch * per].to(torch.int32).view(batch, per)
    return csa2.Cache(batch, cap, ratio=ratio, swa_dtype=swa, page_entries=page, n_pages=batch * per + 4,
                      block_table=table, entry_format=fmt)


class _PagedView:
    """A paged cache's planes per sequence, for assert_cache_equal()."""

    def __init__(self, c):
        self.swa_codes, self.swa_scales, self.swa_dtype = c.swa_codes, c.swa_scales, c.swa_dtype
        for n in ("lat_codes", "lat_scales", "rope_codes", "rope_scales"):
            setattr(self, n, c.plane(n) if getattr(c, n) is not None else None)
        self.idx_entries = c.idx_entries


def _rows(seed, counts, t0, width, stream):
    parts = [wl.token_rows(seed, stream, b, t, n, width) for b, (n, t) in enumerate(zip(counts, t0)) if n]
    return torch.cat(parts) if parts else torch.zeros(0, width)


STEPS = [[5, 0, 140, 1], [1, 1, 1, 1], [130, 3, 0, 300], [0, 127, 129, 128], [1, 0, 1, 1]]


@pytest.mark.parametrize("swa", [csa2.SWA_MXFP8, csa2.SWA_BF16])
@pytest.mark.parametrize("fmt,page,bf16", [(csa2.ENTRY_FP4, None, False), (csa2.ENTRY_FP4, 128, True),
                                           (csa2.ENTRY_FP8, 256, False)])
@pytest.mark.parametrize("window", [False, True])
def test_append_ragged_r1(orc, swa, fmt, page, bf16, window):
    """Chunks of unequal lengths over several calls: the bytes of per-sequence appends; a strided
    source; rows of no sequence ignored; the window rows of each chunk."""
    B, cap, seed = 4, 640, 5
    c = _cache(B, cap, swa=swa, page=page, fmt=fmt)
    oc = [orc.Cache(cap, swa_dtype=swa, entry_format=fmt) for _ in range(B)]
    rope, err, t0 = csa2.rope_table(THETA, cap), _err(), [0] * B
    for counts in STEPS:
        total = sum(counts)
        kv, ik = _rows(seed, counts, t0, 576, wl.S_KV), _rows(seed, counts, t0, 128, wl.S_IK)
        if bf16:
            kv, ik = kv.to(torch.bfloat16), ik.to(torch.bfloat16)
        wide = torch.full((total + 3, 576 + 128 + 8), float("nan"), dtype=kv.dtype)  # 3 rows of no sequence
        wide[:total, :576], wide[:total, 576:704] = kv, ik
        wide = wide.to(DEV)
        win = csa2.chunk_window(c, total + 3) if window else None
        if window:
            win.codes.fill_(77)
        old = [(o.swa_codes.copy(), None if o.swa_scales is None else o.swa_scales.copy()) for o in oc]
        csa2.kv_append_ragged(c, _cu(counts), rope, kv=wide[:, :576], idx_key=wide[:, 576:704],
                              max_new=max(counts), win=win, err=err)
        at = 0
        for b, n in enumerate(counts):
            if n:
                orc.append_r1(oc[b], kv[at:at + n].float().numpy(), ik[at:at + n].float().numpy(), THETA)
            if window:
                # older tokens from the ring as it was, the chunk's last 128 as the ring holds them now
                got, sc = win.codes.cpu().numpy(), win.scales.cpu().numpy()
                for i in list(range(128)) + list(range(max(128, n), 128 + n)):
                    t = t0[b] - 128 + i
                    row = at + 128 * b + i
                    want = (old[b] if i < 128 else (oc[b].swa_codes, oc[b].swa_scales))
                    if t < 0:
                        assert not got[row].any()
                        continue
                    assert np.array_equal(got[row], want[0][t % 128].view(np.uint8).reshape(-1)), (b, i)
                    if swa == csa2.SWA_MXFP8:
                        assert np.array_equal(sc[row, :18], want[1][t % 128])
            at += n
        if window:
            assert (win.codes[total + 128 * B:] == 77).all()
        t0 = [t + n for t, n in zip(t0, counts)]
        assert c.n_tokens.tolist() == t0
    assert int(err) == 0
    view = c if not page else _PagedView(c)
    for b in range(B):
        class One:
            pass
        one = One()
        one.swa_dtype = swa
        for n in ("lat_codes", "lat_scales", "rope_codes", "rope_scales"):
            p = getattr(view, n)
            setattr(one, n, None if p is None else p[b:b + 1])
        one.swa_codes, one.swa_scales = c.swa_codes[b:b + 1], c.swa_scales[b:b + 1]
        ic, isc = view.idx_entries()
        one.idx_entries = lambda ic=ic, isc=isc, b=b: (ic[b:b + 1], isc[b:b + 1])
        assert_cache_equal(one, [oc[b]], t0[b])


@pytest.mark.parametrize("swa,page,fmt", [(csa2.SWA_MXFP8, None, csa2.ENTRY_FP4), (csa2.SWA_BF16, 128, csa2.ENTRY_FP8)])
@pytest.mark.parametrize("window", [False, True])
def test_append_ragged_r2(swa, page, fmt, window):
    """Two tokens per entry: the same planes, ring, compression buffer and counts as csa2_kv_append of
    every sequence by itself (which the parity tests hold to the oracle)."""
    B, cap, seed = 4, 320, 9
    c = _cache(B, cap, ratio=2, swa=swa, page=page, fmt=fmt)
    alone = [_cache(1, cap, ratio=2, swa=swa, page=page, fmt=fmt, seed=1) for _ in range(B)]
    rope, err, t0 = csa2.rope_table(THETA, 2 * cap), _err(), [0] * B
    g = torch.Generator().manual_seed(3)
    ba, bb = (torch.randn(2, 704, generator=g) * 0.5).to(DEV), (torch.randn(2, 704, generator=g) * 0.5).to(DEV)
    for counts in STEPS:
        total = sum(counts)
        rows = [torch.cat([cmp_rows(seed, b, t, n)[i] for b, (n, t) in enumerate(zip(counts, t0)) if n]).to(DEV)
                for i in range(4)]
        win = csa2.chunk_window(c, total) if window else None
        csa2.kv_append_ragged(c, _cu(counts), rope, cmp=rows + [ba, bb], max_new=max(counts), win=win, err=err)
        at = 0
        for b, n in enumerate(counts):
            if n:
                csa2.kv_append(alone[b], rope_cs=rope, cmp=[r[at:at + n][None].contiguous() for r in rows] + [ba, bb], err=err)
            if window and n:
                m = min(n, 128)
                slots = torch.arange(t0[b] + n - m, t0[b] + n, device=DEV) % 128
                r0 = at + 128 * b + 128 + n - m
                assert torch.equal(win.codes[r0:r0 + m], alone[b].swa_codes[0, slots])
            at += n
        t0 = [t + n for t, n in zip(t0, counts)]
    assert int(err) == 0 and c.n_tokens.tolist() == t0
    for b in range(B):
        ent = torch.arange(t0[b] // 2, device=DEV)
        assert torch.equal(ru.main_values(c, ru.phys(c, b, ent)), ru.main_values(alone[b], ru.phys(alone[b], 0, ent)))
        assert torch.equal(ru.key_values(c, b, ent), ru.key_values(alone[b], 0, ent))
        assert torch.equal(c.swa_codes[b], alone[b].swa_codes[0])
        if swa == csa2.SWA_MXFP8:
            assert torch.equal(c.swa_scales[b, :, :18], alone[b].swa_scales[0, :, :18])
        assert torch.equal(c.cmp_buf[b], alone[b].cmp_buf[0])


def test_append_ragged_device_errors():
    """A sequence past the capacity, one past the RoPE table, one over max_new, a page id outside the
    pool: each reports its bit and is left alone; the others are appended."""
    def fresh(cap=256, page=None):
        c = _cache(3, cap, page=page)
        c.n_tokens.copy_(torch.tensor([10, 250, 100]))
        return c
    kv, ik = torch.randn(30, 576, device=DEV), torch.randn(30, 128, device=DEV)
    rope, cu = csa2.rope_table(THETA, 300), _cu([10, 10, 10])
    c, err = fresh(), _err()
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, max_new=10, err=err)
    assert int(err) == csa2.DEVERR_CAPACITY and c.n_tokens.tolist() == [20, 250, 110]
    assert not c.lat_codes[1].any() and c.lat_codes[0, 10:20].any() and c.lat_codes[2, 100:110].any()
    c, err = fresh(512), _err()
    csa2.kv_append_ragged(c, cu, rope[:256], kv=kv, idx_key=ik, max_new=10, err=err)
    assert int(err) == csa2.DEVERR_ROPE and c.n_tokens.tolist() == [20, 250, 110]
    for bad, moved in ((_cu([10, 5, 15]), [20, 255, 100]),        # over max_new
                       (torch.tensor([0, 10, 8, 18], dtype=torch.int32, device=DEV), None),   # decreasing
                       (torch.tensor([0, 10, 20, 900], dtype=torch.int32, device=DEV), None)):  # past the rows
        c, err = fresh(512), _err()
        csa2.kv_append_ragged(c, bad, rope, kv=kv, idx_key=ik, max_new=10, win=csa2.chunk_window(c, 30), err=err)
        assert int(err) & csa2.DEVERR_INDEX
        if moved:
            assert c.n_tokens.tolist() == moved
    c, err = fresh(512, 128), _err()
    c.block_table[1, 1] = 10 ** 6
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, max_new=10, err=err)
    assert int(err) == csa2.DEVERR_INDEX


def _filled(batch, lens, cap, ratio=1, swa=csa2.SWA_MXFP8, page=None, fmt=csa2.ENTRY_FP4, seed=1, scale=1.0):
    c = _cache(batch, cap, ratio=ratio, swa=swa, page=page, fmt=fmt, seed=seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    rope, err = csa2.rope_table(THETA, cap * ratio + 8), _err()
    total = sum(lens)
    rnd = lambda w: torch.randn(total, w, generator=g, device=DEV) * scale
    if ratio == 1:
        csa2.kv_append_ragged(c, _cu(lens), rope, kv=rnd(576), idx_key=rnd(128), err=err)
    else:
        bias = [torch.zeros(2, 704, device=DEV)] * 2
        csa2.kv_append_ragged(c, _cu(lens), rope, cmp=[rnd(704) for _ in range(4)] + bias, err=err)
    assert int(err) == 0
    return c, rope


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,page,ratio", [(csa2.ENTRY_FP4, None, 1), (csa2.ENTRY_FP4, 128, 2), (csa2.ENTRY_FP8, 256, 1)])
def test_kv_read(dtype, fmt, page, ratio):
    """Exact values, ranges and lists, strided outputs, idle sequences, rows of no sequence untouched."""
    lens = [700, 0, 129, 1000]
    c, _ = _filled(4, [n * ratio for n in lens], 1024, ratio=ratio, page=page, fmt=fmt)
    g = torch.Generator().manual_seed(2)
    counts = [300, 0, 129, 411]
    start = torch.tensor([400, 0, 0, 589], device=DEV)
    total, cu = sum(counts), _cu(counts)
    pos = torch.cat([torch.randint(-2, max(1, n), (k,), generator=g) for n, k in zip(lens, counts)]).to(torch.int32).to(DEV)
    for use in ("range", "list"):
        wide = torch.full((total + 5, 576 + 16), 99.0, dtype=dtype, device=DEV)
        keys = torch.full((total + 5, 128), 99.0, dtype=dtype, device=DEV)
        err = _err()
        p = torch.cat([pos, pos[:5]]) if use == "list" else None
        csa2.kv_read(c, cu, out_main=wide[:, :576], out_key=keys, pos=p, start=start if p is None else None, err=err)
        assert int(err) == 0
        at = 0
        for b, k in enumerate(counts):
            ent = pos[at:at + k].long() if use == "list" else start[b] + torch.arange(k, device=DEV)
            some = (ent >= 0)[:, None]
            e0 = ent.clamp(min=0)
            assert torch.equal(wide[at:at + k, :576].double(), torch.where(some, ru.main_values(c, ru.phys(c, b, e0)), 0.0))
            assert torch.equal(keys[at:at + k].double(), torch.where(some, ru.key_values(c, b, e0), 0.0))
            at += k
        assert (wide[:, 576:] == 99).all() and (wide[total:] == 99).all() and (keys[total:] == 99).all()
    only = torch.zeros(total, 128, dtype=dtype, device=DEV)
    csa2.kv_read(c, cu, out_key=only, start=start)
    csa2.kv_read(c, cu, out_main=wide[:total, :576], start=start)
    k2 = torch.empty_like(only)
    csa2.kv_read(c, cu, out_main=torch.empty(total, 576, dtype=dtype, device=DEV), out_key=k2, start=start)
    assert torch.equal(only, k2)


def test_kv_read_index_errors():
    c, _ = _filled(2, [100, 60], 256, page=128)
    out = torch.ones(4, 576, device=DEV)
    for pos, start in ((torch.tensor([0, 100, 59, 60], dtype=torch.int32, device=DEV), None),
                       (None, torch.tensor([99, 59], device=DEV)), (None, torch.tensor([98, -1], device=DEV))):
        err = _err()
        csa2.kv_read(c, _cu([2, 2]), out_main=out, pos=pos, start=start, err=err)
        assert int(err) == csa2.DEVERR_INDEX
    assert not out[2].any() and out[3].any()  # entry -1 of a range, then entry 0
    c.block_table[1, 0] = -7
    err = _err()
    csa2.kv_read(c, _cu([2, 2]), out_main=out, start=torch.tensor([0, 0], device=DEV), err=err)
    assert int(err) == csa2.DEVERR_INDEX and out[:2].any() and not out[2:].any()


@pytest.mark.parametrize("swa", [csa2.SWA_MXFP8, csa2.SWA_BF16])
def test_window_read(swa):
    lens = [0, 5, 128, 333]
    c, _ = _filled(4, lens, 512, swa=swa)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((4, 128, 576), 3.0, dtype=dt, device=DEV)
        csa2.window_read(c, out)
        for b, n in enumerate(lens):
            t = torch.arange(n - 128, n, device=DEV)
            want = ru.window_values(c.swa_codes[b][t % 128], c.swa_scales[b][t % 128], swa)
            assert torch.equal(out[b].double(), torch.where((t >= 0)[:, None], want, 0.0))


def _attn(c, q, cu, win=None, sink=None, dtype=torch.float32, max_new=None, scale=None, pad=0):
    total, H = q.shape[0], q.shape[1]
    out = torch.full((total, H, 512), 5.0, dtype=dtype, device=DEV)
    lse = torch.full((total, H), 5.0, device=DEV)
    err = _err()
    csa2.chunk_attn(c, q, cu, out, lse, csa2.chunk_attn_workspace(total, H, c.batch), scale or 1 / math.sqrt(576),
                    max_new=max_new, win=win, sink=sink, err=err)
    return out, lse, int(err)


def _q(total, H, seed=4, s=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(total, H, 576, generator=g, device=DEV) * s).to(torch.bfloat16)


ATTN = [  # prior tokens, new tokens, heads, ratio, swa, page, fmt
    ([0], [1], 16, 1, csa2.SWA_MXFP8, None, csa2.ENTRY_FP4),            # nothing but the token itself
    ([1, 0, 63], [1, 1, 1], 64, 1, csa2.SWA_BF16, 128, csa2.ENTRY_FP4),
    ([127, 128, 129, 255], [1, 1, 1, 1], 32, 1, csa2.SWA_MXFP8, 128, csa2.ENTRY_FP8),
    ([0, 300], [200, 77], 64, 1, csa2.SWA_MXFP8, 256, csa2.ENTRY_FP4),   # a prompt, a chunk over a prefix
    ([500, 0, 1000, 90], [3, 0, 65, 1], 48, 1, csa2.SWA_BF16, 128, csa2.ENTRY_FP8),
    ([2500, 4000], [1, 1], 128, 1, csa2.SWA_MXFP8, 1024, csa2.ENTRY_FP4),
    ([2222], [130], 128, 1, csa2.SWA_MXFP8, None, csa2.ENTRY_FP4),
    ([0, 1, 501, 640], [5, 1, 8, 1], 16, 2, csa2.SWA_MXFP8, 128, csa2.ENTRY_FP4),
    ([30000], [2], 64, 1, csa2.SWA_MXFP8, 256, csa2.ENTRY_FP4),
    ([1, 2, 3, 5, 700, 40, 41, 0, 9, 10, 11, 600], [1] * 12, 112, 1, csa2.SWA_MXFP8, None, csa2.ENTRY_FP4),
]


@pytest.mark.parametrize("prior,new,H,ratio,swa,page,fmt", ATTN)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_chunk_attn(prior, new, H, ratio, swa, page, fmt, dtype):
    B = len(prior)
    cap = max(p + n for p, n in zip(prior, new)) // ratio + 1
    c, rope = _filled(B, prior, cap, ratio=ratio, swa=swa, page=page, fmt=fmt, seed=7) if sum(prior) else \
        (_cache(B, cap, ratio=ratio, swa=swa, page=page, fmt=fmt), csa2.rope_table(THETA, cap * ratio + 8))
    g = torch.Generator(device=DEV).manual_seed(8)
    total, cu, err = sum(new), _cu(new), _err()
    win = csa2.chunk_window(c, total)
    rnd = lambda w: torch.randn(total, w, generator=g, device=DEV)
    kw = dict(kv=rnd(576), idx_key=rnd(128)) if ratio == 1 else \
        dict(cmp=[rnd(704) for _ in range(4)] + [torch.zeros(2, 704, device=DEV)] * 2)
    csa2.kv_append_ragged(c, cu, rope, max_new=max(new), win=win, err=err, **kw)
    assert int(err) == 0
    q, sink = _q(total, H), torch.randn(H, generator=g, device=DEV) * 2
    for s in (None, sink):
        out, lse, e = _attn(c, q, cu, win, s, dtype, max_new=max(new))
        assert e == 0
        ru.attn_within(out, lse, ru.chunk_attn(c, q, cu, 1 / math.sqrt(576), win, s))
    again, lse2, _ = _attn(c, q, cu, win, sink, dtype, max_new=max(new))
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    if max(new) == 1:  # single tokens: the ring gives the same window
        ring, lse3, e = _attn(c, q, cu, None, sink, dtype, max_new=1)
        assert e == 0 and torch.equal(ring, out) and torch.equal(lse3, lse)


@pytest.mark.parametrize("H,ratio,fmt", [(64, 1, csa2.ENTRY_FP4), (16, 2, csa2.ENTRY_FP8)])
def test_chunk_attn_matches_sparse_with_every_entry(H, ratio, fmt):
    """The decode step's attention with every visible entry selected is the same definition."""
    lens = [1500 * ratio, 70 * ratio, 1]
    c, _ = _filled(3, lens, 2048, ratio=ratio, fmt=fmt)
    q = _q(3, H)
    out, lse, e = _attn(c, q, _cu([1, 1, 1]), max_new=1)
    k = 1500
    q_pos = c.n_tokens - 1
    idx = torch.arange(k, device=DEV)[None].expand(3, k)
    idx = torch.where(idx < (q_pos // ratio)[:, None], idx, -1).to(torch.int32).contiguous()
    ro, rl, err = torch.empty(3, H, 512, device=DEV), torch.empty(3, H, device=DEV), _err()
    csa2.sparse_attn_decode(c, q, q_pos, idx, ro, rl, csa2.attn_workspace(3, H, k), 1 / math.sqrt(576), err=err)
    assert e == 0 and int(err) == 0
    attn_close(out.cpu().numpy(), lse.cpu().numpy(), ro.cpu().numpy(), rl.cpu().numpy(), 4e-3)  # 2e-3 on each side


def test_chunk_attn_against_the_oracle(orc):
    T, H, seed = 333, 64, 21
    oc = orc.Cache(400, swa_dtype=orc.SWA_MXFP8)
    kv, ik = wl.token_rows(seed, wl.S_KV, 0, 0, T, 576), wl.token_rows(seed, wl.S_IK, 0, 0, T, 128)
    orc.append_r1(oc, kv.numpy(), ik.numpy(), THETA)
    c, rope = csa2.Cache(1, 400), csa2.rope_table(THETA, 400)
    csa2.kv_append_ragged(c, _cu([T]), rope, kv=kv.to(DEV), idx_key=ik.to(DEV))
    q = _q(1, H)
    out, lse, e = _attn(c, q, _cu([1]), max_new=1)
    ro, rl = orc.sparse_attn(oc, u16(q[0]), np.arange(T - 1, dtype=np.int32), T - 1, 1 / math.sqrt(576))
    assert e == 0
    attn_close(out[0].cpu().numpy(), lse[0].cpu().numpy(), ro, rl)


def test_chunk_attn_rows_of_no_sequence_and_errors():
    c, rope = _filled(2, [300, 40], 512, page=128)
    cu, total = _cu([4, 3]), 12
    win = csa2.chunk_window(c, total)
    kv, ik = torch.randn(total, 576, device=DEV), torch.randn(total, 128, device=DEV)
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, max_new=4, win=win)
    q = _q(total, 32)
    out, lse, e = _attn(c, q, cu, win, max_new=4)
    assert e == 0 and (out[7:] == 5).all() and (lse[7:] == 5).all()
    ru.attn_within(out, lse, ru.chunk_attn(c, q, cu, 1 / math.sqrt(576), win), slice(0, 7))
    # without the window rows the chunk's earlier queries miss tokens behind the ring
    assert _attn(c, q, cu, None, max_new=4)[2] == csa2.DEVERR_INDEX
    # a sequence over max_new, cu past the rows, a page outside the pool
    assert _attn(c, q, cu, win, max_new=3)[2] == csa2.DEVERR_INDEX
    assert _attn(c, q, torch.tensor([0, 4, 40], dtype=torch.int32, device=DEV), win, max_new=40)[2] == csa2.DEVERR_INDEX
    c.block_table[0, 1] = c.n_pages
    out2, lse2, e = _attn(c, q, cu, win, max_new=4)
    assert e == csa2.DEVERR_INDEX and torch.equal(out2[4:7], out[4:7])


def test_chunk_attn_large_and_tiny_values():
    """Values beyond fp16 in the window, all-zero entries, logits far apart, a key that outweighs all."""
    c, rope = _filled(2, [200, 500], 640, seed=3)
    n = [70, 1]
    cu, win = _cu(n), csa2.chunk_window(c, 71)
    g = torch.Generator(device=DEV).manual_seed(5)
    kv = torch.randn(71, 576, generator=g, device=DEV)
    kv[10] *= 2.0 ** 20
    kv[20] *= 2.0 ** -20
    kv[30] = 0
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=torch.zeros(71, 128, device=DEV), max_new=70, win=win)
    q = _q(71, 16, s=1.0)
    q[5] *= 30
    q[40, 3] = 0
    q[11:] *= 2.0 ** -18
    out, lse, e = _attn(c, q, cu, win, max_new=70)
    assert e == 0
    ru.attn_within(out, lse, ru.chunk_attn(c, q, cu, 1 / math.sqrt(576), win))


def test_streams_and_graphs():
    """A captured append + read + attention, replayed with other lengths, on another stream than the
    tensors' own; the results of the eager calls."""
    B, total, H = 3, 24, 64
    def run(c, st, stream=None):
        csa2.kv_append_ragged(c, st["cu"], st["rope"], kv=st["kv"], idx_key=st["ik"], max_new=16, win=st["win"], err=st["err"], stream=stream)
        csa2.kv_read(c, st["cu"], out_main=st["main"], start=st["start"], err=st["err"], stream=stream)
        csa2.chunk_attn(c, st["q"], st["cu"], st["out"], st["lse"], st["ws"], 0.05, max_new=16, win=st["win"], err=st["err"], stream=stream)
    def state(c):
        st = dict(cu=_cu([1, 16, 5]), kv=torch.randn(total, 576, device=DEV), ik=torch.randn(total, 128, device=DEV),
                  q=_q(total, H), win=csa2.chunk_window(c, total), err=_err(), rope=csa2.rope_table(THETA, 600),
                  main=torch.zeros(total, 576, device=DEV), out=torch.zeros(total, H, 512, device=DEV),
                  lse=torch.zeros(total, H, device=DEV), ws=csa2.chunk_attn_workspace(total, H, B))
        st["start"] = c.n_tokens.clone()
        return st
    lens = [400, 130, 3]
    c1, _ = _filled(B, lens, 512)
    c2, _ = _filled(B, lens, 512)
    torch.manual_seed(0)
    a = state(c1)
    torch.manual_seed(0)
    b = state(c2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    keep = [t.clone() for t in (c2.n_tokens, c2.swa_codes, c2.swa_scales)]
    with torch.cuda.stream(side):
        run(c2, b)  # warm: attributes set outside the capture
        side.synchronize()
    for t, k in zip((c2.n_tokens, c2.swa_codes, c2.swa_scales), keep):
        t.copy_(k)
    with torch.cuda.graph(graph, stream=side):
        run(c2, b)
    for counts in ([1, 16, 5], [0, 3, 11], [2, 0, 0]):
        for c, st in ((c1, a), (c2, b)):
            st["cu"].copy_(_cu(counts))
            st["start"].copy_(c.n_tokens)
        run(c1, a)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(counts)
        assert int(a["err"]) == 0 and int(b["err"]) == 0
        assert torch.equal(c1.n_tokens, c2.n_tokens)
        for k in ("main", "out", "lse"):
            assert torch.equal(a[k][:n], b[k][:n]), k


def test_serving_loop():
    """Prompts in ragged chunks, then drafted tokens, then single tokens: append, attend and read back
    together; every call against the plain form, the read-back against the stored bytes."""
    B, H, cap, page = 3, 64, 768, 128
    c, rope, err = _cache(B, cap, page=page), csa2.rope_table(THETA, cap), _err()
    g = torch.Generator(device=DEV).manual_seed(11)
    for step, counts in enumerate([[300, 1, 90], [0, 257, 40], [4, 4, 4], [1, 1, 1], [1, 0, 1]]):
        total, cu = sum(counts), _cu(counts)
        before = c.n_tokens.clone()
        one = max(counts) == 1
        win = None if one else csa2.chunk_window(c, total)
        csa2.kv_append_ragged(c, cu, rope, kv=torch.randn(total, 576, generator=g, device=DEV).to(torch.bfloat16),
                              idx_key=torch.randn(total, 128, generator=g, device=DEV).to(torch.bfloat16),
                              max_new=max(counts), win=win, err=err)
        q = _q(total, H, seed=step)
        out, lse, e = _attn(c, q, cu, win, None, torch.bfloat16, max_new=max(counts))
        main = torch.empty(total, 576, dtype=torch.bfloat16, device=DEV)
        csa2.kv_read(c, cu, out_main=main, start=before, err=err)
        assert e == 0 and int(err) == 0
        ru.attn_within(out, lse, ru.chunk_attn(c, q, cu, 1 / math.sqrt(576), win))
        at = 0
        for b, n in enumerate(counts):
            ent = before[b] + torch.arange(n, device=DEV)
            assert torch.equal(main[at:at + n].double(), ru.main_values(c, ru.phys(c, b, ent)))
            at += n


def test_from_planes_shares_memory():
    c, _ = _filled(2, [100, 50], 256, page=128)
    names = ("lat_codes", "lat_scales", "rope_codes", "rope_scales", "idx_codes", "idx_scales", "swa_codes", "swa_scales", "n_tokens")
    d = csa2.Cache.from_planes(2, 256, {n: getattr(c, n) for n in names}, page_entries=128, n_pages=c.n_pages,
                               block_table=c.block_table)
    a, b = (torch.empty(150, 576, device=DEV) for _ in range(2))
    for x, o in ((c, a), (d, b)):
        csa2.kv_read(x, _cu([100, 50]), out_main=o, start=torch.zeros(2, dtype=torch.int64, device=DEV))
    assert torch.equal(a, b) and a.any()


def test_python_refusals():
    c, rope = _filled(2, [10, 5], 128)
    cu = _cu([1, 1])
    kv, ik = torch.randn(2, 576, device=DEV), torch.randn(2, 128, device=DEV)
    bad = [dict(kv=kv.half(), idx_key=ik), dict(kv=kv, idx_key=ik.to(torch.bfloat16)), dict(kv=kv[:, :512], idx_key=ik),
           dict(kv=kv.cpu(), idx_key=ik), dict(kv=kv, idx_key=ik[:1]), dict(kv=kv, idx_key=ik, cmp=[kv]),
           dict(kv=kv, idx_key=ik, win=csa2.chunk_window(c, 3))]
    for kw in bad:
        with pytest.raises(ValueError):
            csa2.kv_append_ragged(c, cu, rope, **kw)
    with pytest.raises(csa2.Csa2Error):  # a row stride that is no multiple of 8
        csa2.kv_append_ragged(c, cu, rope, kv=torch.randn(2, 580, device=DEV)[:, :576], idx_key=ik)
    with pytest.raises(ValueError):
        csa2.kv_append_ragged(c, cu.long(), rope, kv=kv, idx_key=ik)
    out = torch.empty(2, 576, device=DEV)
    for kw in (dict(), dict(out_main=out), dict(out_main=out, start=torch.zeros(2, device=DEV)),
               dict(out_main=out, out_key=torch.empty(2, 128, device=DEV, dtype=torch.bfloat16), start=torch.zeros(2, dtype=torch.int64, device=DEV)),
               dict(out_main=out, pos=torch.zeros(2, dtype=torch.int32, device=DEV), start=torch.zeros(2, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            csa2.kv_read(c, cu, **kw)
    q, o, l = _q(2, 64), torch.empty(2, 64, 512, device=DEV), torch.empty(2, 64, device=DEV)
    ws = csa2.chunk_attn_workspace(2, 64, 2)
    for args in ((q.float(), cu, o, l, ws), (q, cu[:2], o, l, ws), (q, cu, o[:1], l, ws), (q, cu, o, l.double(), ws),
                 (q.transpose(0, 1), cu, o, l, ws)):
        with pytest.raises(ValueError):
            csa2.chunk_attn(c, *args, 0.1)
    with pytest.raises(csa2.Csa2Error):
        csa2.chunk_attn(c, q, cu, o, l, ws[:16], 0.1)
    with pytest.raises(csa2.Csa2Error):
        csa2.chunk_attn(c, q, cu, o, l, ws, float("nan"))
    assert c.n_tokens.tolist() == [10, 5]


@pytest.mark.parametrize("swa", [csa2.SWA_MXFP8, csa2.SWA_BF16])
@pytest.mark.parametrize("fmt", [csa2.ENTRY_FP4, csa2.ENTRY_FP8])
@pytest.mark.parametrize("bf16", [False, True])
def test_append_special_values(swa, fmt, bf16):
    """NaN, infinities, zeros of both signs, subnormals, wide ranges and values halfway between codes:
    the bytes of csa2_kv_append."""
    n = 96
    g = torch.Generator(device=DEV).manual_seed(3)
    kv, ik = (torch.randn(n, w, generator=g, device=DEV) for w in (576, 128))
    for t in (kv, ik):
        t[1] = 0.0
        t[2] = -0.0
        t[3, 5], t[4, 7], t[5, 9] = math.nan, math.inf, -math.inf
        t[6] = math.nan
        t[7] = -math.inf
        t[8] *= 2.0 ** -140
        t[9] *= 2.0 ** 120
        t[10] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device=DEV).repeat(t.shape[1] // 8)
        t[11] = -t[10] * 3
        t[12] = 0.0
        t[12, -1] = 2.0 ** -20
        t[13:40] *= torch.exp2(torch.randint(-30, 30, t[13:40].shape, generator=g, device=DEV).float())
        t[40:60] = t[40:60].to(torch.float8_e4m3fn).float() * 1.0625
    if bf16:
        kv, ik = kv.to(torch.bfloat16), ik.to(torch.bfloat16)
    rope = csa2.rope_table(THETA, 256)
    a, b = (_cache(1, 256, swa=swa, fmt=fmt) for _ in range(2))
    ea, eb = _err(), _err()
    csa2.kv_append_ragged(a, _cu([n]), rope, kv=kv, idx_key=ik, err=ea)
    csa2.kv_append(b, kv[None], ik[None], rope, err=eb)
    assert int(ea) == int(eb) == 0
    for name in ("lat_codes", "lat_scales", "rope_codes", "rope_scales", "idx_codes", "idx_scales", "swa_codes", "swa_scales"):
        x, y = getattr(a, name), getattr(b, name)
        if x is not None and not (name == "swa_scales" and swa == csa2.SWA_BF16):
            assert torch.equal(x, y), name


@pytest.mark.parametrize("fmt", [csa2.ENTRY_FP4, csa2.ENTRY_FP8])
def test_kv_read_rows_on_16_bytes(fmt):
    """fp32 rows that start 16 B, not 32 B, aligned."""
    c, _ = _filled(1, [70], 128, fmt=fmt)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    want, wk = torch.empty(70, 576, device=DEV), torch.empty(70, 128, device=DEV)
    csa2.kv_read(c, _cu([70]), out_main=want, out_key=wk, start=zero)
    main = torch.full((70 * 576 + 8,), 9.0, device=DEV)
    key = torch.full((70 * 128 + 8,), 9.0, device=DEV)
    csa2.kv_read(c, _cu([70]), out_main=main[4:-4].view(70, 576), out_key=key[4:-4].view(70, 128), start=zero)
    assert torch.equal(main[4:-4].view(70, 576), want) and torch.equal(key[4:-4].view(70, 128), wk)
    for t in (main, key):
        assert (t[:4] == 9).all() and (t[-4:] == 9).all()


def test_far_pages():
    """Pages at the end of a pool whose planes pass 2^32 bytes."""
    n_pages, page = 18000, 1024  # 18.4 M entries: 4.7 GB of latent codes
    table = torch.tensor([[n_pages - 1, 0], [n_pages - 3, n_pages - 2]], dtype=torch.int32)
    c = csa2.Cache(2, 2 * page, page_entries=page, n_pages=n_pages, block_table=table)
    lens = [1100, 1500]
    g = torch.Generator(device=DEV).manual_seed(9)
    rope, err = csa2.rope_table(THETA, 2 * page), _err()
    kv, ik = (torch.randn(sum(lens), w, generator=g, device=DEV) for w in (576, 128))
    csa2.kv_append_ragged(c, _cu(lens), rope, kv=kv, idx_key=ik, err=err)
    near = csa2.Cache(2, 2 * page)
    csa2.kv_append_ragged(near, _cu(lens), rope, kv=kv, idx_key=ik, err=err)
    q, zero = _q(2, 64), torch.zeros(2, dtype=torch.int64, device=DEV)
    outs = []
    for x in (c, near):
        main, key = torch.empty(sum(lens), 576, device=DEV), torch.empty(sum(lens), 128, device=DEV)
        csa2.kv_read(x, _cu(lens), out_main=main, out_key=key, start=zero, err=err)
        outs.append((main, key) + _attn(x, q, _cu([1, 1]), max_new=1))
    assert int(err) == 0 and outs[0][4] == outs[1][4] == 0
    for x, y in zip(outs[0][:4], outs[1][:4]):
        assert torch.equal(x, y)


def test_many_sequences():
    """More sequences and row tiles than the plan keeps in shared memory; some sequences idle."""
    B, H = 1500, 128
    g = torch.Generator().manual_seed(10)
    prior = torch.randint(0, 20, (B,), generator=g).tolist()
    new = torch.randint(0, 3, (B,), generator=g).tolist()
    c, rope = _filled(B, prior, 24)
    total, cu, err = sum(new), _cu(new), _err()
    assert total * H > 2048 * 64
    win = csa2.chunk_window(c, total)
    csa2.kv_append_ragged(c, cu, rope, kv=torch.randn(total, 576, device=DEV), idx_key=torch.randn(total, 128, device=DEV),
                          max_new=2, win=win, err=err)
    q = _q(total, H)
    out, lse, e = _attn(c, q, cu, win, max_new=2)
    assert e == 0 and int(err) == 0
    ru.attn_within(out, lse, ru.chunk_attn(c, q, cu, 1 / math.sqrt(576), win))


def test_two_calls_at_once():
    """Two attentions with a workspace each, on two streams, over one cache, beside an append to another."""
    c, rope = _filled(4, [3000, 2000, 2500, 10], 4096, page=128)
    d, _ = _filled(4, [50, 60, 70, 80], 4096)
    q1, q2 = _q(4, 64, seed=1), _q(4, 128, seed=2)
    cu = _cu([1, 1, 1, 1])
    want = [_attn(c, q, cu, max_new=1)[:2] for q in (q1, q2)]
    kv, ik, cu_d = torch.randn(800, 576, device=DEV), torch.randn(800, 128, device=DEV), _cu([200, 200, 200, 200])
    err, streams = _err(), [torch.cuda.Stream() for _ in range(3)]
    got = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in want]
    ws = [csa2.chunk_attn_workspace(4, H, 4) for H in (64, 128)]
    torch.cuda.synchronize()
    for _ in range(10):
        csa2.kv_append_ragged(d, cu_d, rope, kv=kv, idx_key=ik, err=err, stream=streams[2])
        for i, q in enumerate((q1, q2)):
            csa2.chunk_attn(c, q, cu, got[i][0], got[i][1], ws[i], 1 / math.sqrt(576), max_new=1, err=err, stream=streams[i])
    torch.cuda.synchronize()
    assert int(err) == 0 and d.n_tokens.tolist() == [2050, 2060, 2070, 2080]
    for (o, l), (wo, wl_) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl_)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_chunk_attn_masked_nonfinite(bad):
    """A bf16 window holds infinities and NaN as they come: the rows that see such a token are NaN, the
    others (earlier ones, later than 127 tokens, in the same row tiles) know nothing of it."""
    c, rope = _filled(2, [90, 20], 512, swa=csa2.SWA_BF16)
    n, at, H = [200, 3], 30, 16
    cu, total = _cu(n), sum(n)
    win = csa2.chunk_window(c, total)
    g = torch.Generator(device=DEV).manual_seed(6)
    kv, ik = torch.randn(total, 576, generator=g, device=DEV), torch.randn(total, 128, generator=g, device=DEV)
    kv[at, 77] = bad
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, max_new=200, win=win)
    q = _q(total, H)
    sees = torch.zeros(total, dtype=torch.bool, device=DEV)
    sees[at:at + 128] = True
    out, lse, e = _attn(c, q, cu, win, max_new=200)
    assert e == 0 and out[sees].isnan().all() and lse[sees].isnan().all()
    clean = csa2.ChunkWindow(win.codes.clone(), win.scales)
    clean.codes[128 + at] = 0  # (the plain form would multiply it by zero)
    ru.attn_within(out[~sees], lse[~sees], [t[~sees] for t in ru.chunk_attn(c, q, cu, 1 / math.sqrt(576), clean)])


def test_chunk_attn_nonfinite_query_and_sink():
    """A query that is not finite spoils its own row; a sink of +inf takes all the weight, one of -inf none."""
    c, _ = _filled(3, [2000, 150, 1], 2048)
    H, cu = 32, _cu([1, 1, 1])
    q = _q(3, H)
    plain, pl, _ = _attn(c, q, cu, max_new=1)
    bad = q.clone()
    bad[0, 3, 100], bad[1, 31, 570], bad[2, 0, 0] = math.nan, math.inf, -math.inf
    out, lse, e = _attn(c, bad, cu, max_new=1)
    hit = torch.zeros(3, H, dtype=torch.bool, device=DEV)
    hit[0, 3] = hit[1, 31] = hit[2, 0] = True
    assert e == 0 and torch.equal(out[~hit], plain[~hit]) and torch.equal(lse[~hit], pl[~hit])
    assert out[0, 3].isnan().all() and lse[0, 3].isnan()
    sink = torch.zeros(H, device=DEV)
    sink[0], sink[1] = math.inf, -math.inf
    out, lse, e = _attn(c, q, cu, sink=sink, max_new=1)
    assert e == 0 and not out[:, 0].any() and (lse[:, 0] == math.inf).all()
    ez = 2.0 ** -20  # the sums are the same up to their last bits
    assert ((out[:, 1] - plain[:, 1]).abs() <= ez * plain[:, 1].abs()).all() and ((lse - pl)[:, 1].abs() <= ez * (1 + pl[:, 1].abs())).all()


def test_empty_calls():
    """No rows at all, and no sequence with any."""
    c, rope = _filled(2, [10, 5], 128)
    before = {n: getattr(c, n).clone() for n in ("n_tokens", "lat_codes", "swa_codes")}
    e = lambda *s, **k: torch.empty(0, *s, device=DEV, **k)
    cu, err = _cu([0, 0]), _err()
    csa2.kv_append_ragged(c, cu, rope, kv=e(576), idx_key=e(128), err=err)
    csa2.kv_read(c, cu, out_main=e(576), out_key=e(128), start=torch.zeros(2, dtype=torch.int64, device=DEV), err=err)
    csa2.chunk_attn(c, e(64, 576, dtype=torch.bfloat16), cu, e(64, 512), e(64), csa2.chunk_attn_workspace(0, 64, 2), 0.1, err=err)
    kv, ik = torch.randn(3, 576, device=DEV), torch.randn(3, 128, device=DEV)
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, err=err)
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, win=csa2.chunk_window(c, 3), err=err)
    out, lse, bits = _attn(c, _q(3, 64), cu)
    assert bits == 0 and int(err) == 0 and (out == 5).all() and (lse == 5).all()
    for n, t in before.items():
        assert torch.equal(getattr(c, n), t)
