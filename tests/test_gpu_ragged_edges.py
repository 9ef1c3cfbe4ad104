"""Edges of the ragged calls: values that are not finite where they must not matter, NaN of either sign, lists
of rows that are no lists, values of a key that lie far apart, planes of any shape."""
import math

import pytest
import torch

import ragged_util as ru
from fp4_compressed_sparse_gb300 import csa2
from test_gpu_ragged import DEV, THETA, _attn, _cache, _cu, _err, _filled, _lib, _q  # noqa: F401 (_lib: fixture)

pytestmark = pytest.mark.gpu
PLANES = ("lat_codes", "lat_scales", "rope_codes", "rope_scales", "idx_codes", "idx_scales", "swa_codes", "swa_scales")


def _same_bytes(a, b):
    """Every stored byte of two caches (of a bf16 window no scales are stored)."""
    for name in PLANES + ("cmp_buf", "n_tokens"):
        x, y = getattr(a, name), getattr(b, name)
        if x is None or (name == "swa_scales" and a.swa_dtype == csa2.SWA_BF16):
            continue
        if name == "swa_scales":  # 18 of 32 are used
            x, y = x[..., :18], y[..., :18]
        if name == "cmp_buf":
            x, y = x.view(torch.int32), y.view(torch.int32)
        assert torch.equal(x, y), name


def _r2_pair(rows, counts, swa=csa2.SWA_MXFP8, fmt=csa2.ENTRY_FP4, window=False):
    """The same ratio-2 rows appended by the ragged call (as a batch of one) and by csa2_kv_append."""
    a, b = (_cache(1, 64, ratio=2, swa=swa, fmt=fmt) for _ in range(2))
    rope, err = csa2.rope_table(THETA, 128), _err()
    bias = [torch.full((2, 704), 0.25, device=DEV), torch.full((2, 704), -0.5, device=DEV)]
    at = 0
    for n in counts:
        part = [r[at:at + n].contiguous() for r in rows]
        win = csa2.chunk_window(a, n) if window else None
        csa2.kv_append_ragged(a, _cu([n]), rope, cmp=part + bias, max_new=n, win=win, err=err)
        csa2.kv_append(b, rope_cs=rope, cmp=[r[None] for r in part] + bias, err=err)
        at += n
    assert int(err) == 0
    return a, b


def _rows4(n, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(n, 704, generator=g, device=DEV) for _ in range(4)]


@pytest.mark.parametrize("counts", [[2], [1, 1], [7]])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_r2_first_entry_has_no_predecessor(counts, bad):
    """C^b and Z^b of the first pair belong to the next entry alone, whatever they hold."""
    rows = _rows4(sum(counts))
    rows[1][0, 5::7] = bad   # C^b
    rows[3][0, 3::11] = bad  # Z^b
    rows[1][1, 4::9] = bad
    a, b = _r2_pair(rows, counts)
    _same_bytes(a, b)
    clean = [r.clone() for r in rows]
    for i in (1, 3):
        clean[i][:2] = 0.0
    c, _ = _r2_pair(clean, counts)
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    assert torch.equal(ru.main_values(a, zero), ru.main_values(c, zero))


@pytest.mark.parametrize("swa", [csa2.SWA_MXFP8, csa2.SWA_BF16])
@pytest.mark.parametrize("fmt", [csa2.ENTRY_FP4, csa2.ENTRY_FP8])
@pytest.mark.parametrize("counts,window", [([12], False), ([5, 1, 6], True), ([1] * 12, False)])
def test_r2_special_values(swa, fmt, counts, window):
    """NaN in single values, whole groups and whole rows, infinities, zeros: the bytes of csa2_kv_append."""
    rows = _rows4(12, seed=2)
    for i, t in enumerate(rows):
        t[2 + i, 64:96] = math.nan       # a group of 32, and of 16 twice
        t[3, 500:576] = math.nan         # the RoPE dims
        t[7, 600:] = math.nan            # indexer keys
        t[6, 17] = math.inf
        t[8 + i % 2] = -0.0
        t[10, ::3] = -math.inf
    rows[0][11] = math.nan
    a, b = _r2_pair(rows, counts, swa, fmt, window)
    _same_bytes(a, b)


@pytest.mark.parametrize("swa", [csa2.SWA_MXFP8, csa2.SWA_BF16])
@pytest.mark.parametrize("fmt", [csa2.ENTRY_FP4, csa2.ENTRY_FP8])
@pytest.mark.parametrize("bf16", [False, True])
def test_r1_nan_of_either_sign(swa, fmt, bf16):
    """NaN with the sign bit set, beside other values and alone in its group."""
    n = 9
    g = torch.Generator(device=DEV).manual_seed(3)
    kv, ik = (torch.randn(n, w, generator=g, device=DEV) for w in (576, 128))
    for t in (kv, ik):
        u = t.view(torch.int32)
        u[1, 5] = -1                     # 0xFFFFFFFF
        u[2, ::3] = -(1 << 22)           # 0xFFC00000
        u[3] = -1
        u[4, 32:64] = -(1 << 22)
        u[5, -20:] = -1
        u[6, ::2] = 0x7FC00000
        u[6, 1::2] = -(1 << 22)
    assert kv[1, 5].isnan() and kv[2, 3].isnan()
    if bf16:
        bits = [(t.view(torch.int32) >> 16).to(torch.int16) for t in (kv, ik)]
        kv, ik = [b.view(torch.bfloat16) for b in bits]
    rope, err = csa2.rope_table(THETA, 64), _err()
    a, b = (_cache(1, 64, swa=swa, fmt=fmt) for _ in range(2))
    csa2.kv_append_ragged(a, _cu([n]), rope, kv=kv, idx_key=ik, err=err)
    csa2.kv_append(b, kv[None], ik[None], rope, err=err)
    assert int(err) == 0
    _same_bytes(a, b)


def _list(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# lists of row bounds over 3 sequences: rows, bound on a sequence's rows, which sequences keep their rows
BROKEN = [
    ((0, 4, 4, 10), 4, 6, (0, 1)),          # the last one's rows lie behind the arrays
    ((0, 1, 2, 2), 1, 1, (0, 2)),           # the same with single tokens
    ((0, 10, 8, 18), 30, 10, (0,)),         # decreasing: the last one's rows overlap the first one's
    ((0, 4, 10, 14), 14, 5, (0, 2)),        # over the bound
    ((0, 300, 10, 400), 400, 400, (0,)),    # decreasing far: the last one's older tokens would fall among the first one's
    ((-3, 2, 4, 5), 5, 5, (1, 2)),          # a negative start
    ((0, 0, 5, 3), 8, 8, ()),               # decreasing at the end: no list at all for the middle one
    ((0, 1, 0, 1), 1, 1, (0,)),              # two claim the same row: the first one's
]


@pytest.mark.parametrize("bounds,total,mx,kept", BROKEN)
@pytest.mark.parametrize("ratio", [1, 2])
@pytest.mark.parametrize("window", [False, True])
def test_append_broken_lists(bounds, total, mx, kept, ratio, window):
    """Every broken list raises INDEX; a sequence that cannot be told its rows is left alone, the others are
    appended as by themselves."""
    def fresh(batch, start):
        c = _cache(batch, 512, ratio=ratio)
        g = torch.Generator(device=DEV).manual_seed(1)
        c.swa_codes.copy_(torch.randint(0, 100, c.swa_codes.shape, generator=g, device=DEV, dtype=torch.uint8)[:1].expand_as(c.swa_codes))
        c.n_tokens.fill_(start)
        return c
    start, rope = 6, csa2.rope_table(THETA, 1100)
    g = torch.Generator(device=DEV).manual_seed(2)
    rows = [torch.randn(total, w, generator=g, device=DEV) for w in ((576, 128) if ratio == 1 else (704,) * 4)]
    bias = [torch.zeros(2, 704, device=DEV)] * 2
    def append(c, cu, rows, mx, win, err):
        kw = dict(kv=rows[0], idx_key=rows[1]) if ratio == 1 else dict(cmp=rows + bias)
        csa2.kv_append_ragged(c, cu, rope, max_new=mx, win=win, err=err, **kw)
    c, err = fresh(3, start), _err()
    win = csa2.chunk_window(c, total) if window else None
    append(c, _list(*bounds), rows, mx, win, err)
    assert int(err) == csa2.DEVERR_INDEX
    for b in range(3):
        lo, hi = bounds[b], bounds[b + 1]
        one, e1 = fresh(1, start), _err()
        n = hi - lo if b in kept else 0
        if n > 0:
            w1 = csa2.chunk_window(one, n) if window else None
            append(one, _list(0, n), [r[lo:hi].contiguous() for r in rows], n, w1, e1)
            if window:
                r0 = lo + 128 * b
                assert torch.equal(win.codes[r0:r0 + n + 128], w1.codes)
        assert int(e1) == 0 and int(c.n_tokens[b]) == start + n
        for name in ("lat_codes", "lat_scales", "rope_codes", "swa_codes") + (("cmp_buf",) if ratio == 2 else ()):
            assert torch.equal(getattr(c, name)[b], getattr(one, name)[0]), (b, name)


@pytest.mark.parametrize("bounds,total,mx,kept", BROKEN)
def test_attn_broken_lists(bounds, total, mx, kept):
    """The same for the attention."""
    c, _ = _filled(3, [450, 460, 470], 512)
    q = _q(total, 16)
    win = csa2.chunk_window(c, total)
    g = torch.Generator(device=DEV).manual_seed(6)
    win.codes.copy_(torch.randint(0x20, 0x40, win.codes.shape, generator=g, device=DEV, dtype=torch.uint8))  # 2^-3 .. 2
    win.scales.fill_(127)
    out, lse, bits = _attn(c, q, _list(*bounds), win, max_new=mx)
    assert bits == csa2.DEVERR_INDEX
    live = torch.zeros(total, dtype=torch.bool, device=DEV)
    for b in kept:
        lo, hi = bounds[b], bounds[b + 1]
        if hi <= lo:
            continue
        live[lo:hi] = True
        n = hi - lo
        w1 = csa2.ChunkWindow(win.codes[lo + 128 * b:hi + 128 * (b + 1)], win.scales[lo + 128 * b:hi + 128 * (b + 1)])
        one = csa2.Cache.from_planes(1, 512, {k: getattr(c, k)[b:b + 1] for k in PLANES + ("n_tokens",)})
        ref = ru.chunk_attn(one, q[lo:hi], _cu([n]), 1 / math.sqrt(576), w1)
        ru.attn_within(out[lo:hi], lse[lo:hi], ref)
    assert (out[~live] == 5).all() and (lse[~live] == 5).all()


@pytest.mark.parametrize("bounds,total,mx,kept", [x for x in BROKEN if x[0] != (0, 4, 10, 14)])  # (reads have no bound)
@pytest.mark.parametrize("listed", [False, True])
def test_read_broken_lists(bounds, total, mx, kept, listed):
    """The same for reads: INDEX, and the rows of a sequence that cannot be told them are left as they were."""
    c, _ = _filled(3, [450, 460, 470], 512)
    out, key = torch.full((total, 576), 7.0, device=DEV), torch.full((total, 128), 7.0, device=DEV)
    want, wkey = out.clone(), key.clone()
    pos = torch.arange(total, device=DEV).to(torch.int32)
    start = torch.tensor([3, 1, 2], device=DEV)
    err = _err()
    csa2.kv_read(c, _list(*bounds), out_main=out, out_key=key, pos=pos if listed else None,
                 start=None if listed else start, err=err)
    assert int(err) == csa2.DEVERR_INDEX
    for b in kept:
        lo, hi = bounds[b], bounds[b + 1]
        if hi > lo:
            ent = pos[lo:hi].long() if listed else start[b] + torch.arange(hi - lo, device=DEV)
            want[lo:hi] = ru.main_values(c, ru.phys(c, b, ent)).float()
            wkey[lo:hi] = ru.key_values(c, b, ent).float()
    assert torch.equal(out, want) and torch.equal(key, wkey)


def test_from_planes_of_any_shape():
    """Flat planes, and longer ones than needed: the helpers that show entries see the shapes of a cache."""
    for page in (None, 128):
        c, _ = _filled(2, [200, 70], 256, page=page)
        flat = {n: torch.cat([getattr(c, n).reshape(-1), torch.full((32,), 9, dtype=torch.uint8, device=DEV)]) for n in PLANES}
        flat["n_tokens"] = c.n_tokens
        d = csa2.Cache.from_planes(2, 256, flat, page_entries=page, n_pages=c.n_pages or None, block_table=c.block_table)
        for n in PLANES[:4]:
            assert torch.equal(d.plane(n), c.plane(n))
        for x, y in zip(d.idx_entries(), c.idx_entries()):
            assert torch.equal(x, y)
        assert torch.equal(d.swa_codes, c.swa_codes) and torch.equal(d.swa_scales, c.swa_scales)


def _within_values(out, lse, ref, q, scale, s=1.0):
    """ru.attn_within() for keys whose values the operands hold to 2^-25 s (fp16's step is 2^-24; s is 1 for keys
    of a largest magnitude of 1 to 2^16, which go in as they are), and 2^-34 s more for a block of values whose
    codes are rounded to E4M3's step of 2^-9 at 2^-24 first: D.  The outputs, weighted means of the values, move by D
    at most, a logit by scale sum |q| D."""
    o, l, mag, dot, small = ref
    D = (2.0 ** -25 + 2.0 ** -34) * s
    ez = 40 * 2.0 ** -23 * dot + 2.0 ** -22 * (1 + l.abs()) + scale * q.double().abs().sum(-1) * D
    assert ((lse.double() - l).abs() <= ez).all()
    tol = (2.0 ** -11 + 2.0 ** -16 + 2 * ez[..., None]) * mag + 2.0 ** -29 * small + 2.0 ** -30 + D
    err = (out.double() - o).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("fmt,swa", [(csa2.ENTRY_FP8, csa2.SWA_MXFP8), (csa2.ENTRY_FP8, csa2.SWA_BF16),
                                     (csa2.ENTRY_FP4, csa2.SWA_MXFP8)])
@pytest.mark.parametrize("prior,new", [(500, 3), (0, 200), (40, 1)])
def test_attn_small_blocks_beside_large_ones(fmt, swa, prior, new):
    """Blocks of 32 dims far below the key's largest magnitude, whose scale fp16 does not have."""
    c, rope = _cache(1, 640, swa=swa, fmt=fmt), csa2.rope_table(THETA, 640)
    g = torch.Generator(device=DEV).manual_seed(4)
    kv = torch.randn(prior + new, 576, generator=g, device=DEV)
    for blk, e in ((1, -17), (2, -19), (3, -23), (4, -27), (5, -40), (9, -16), (15, -12)):
        # 2^e to 2^(e + 1), one sign: the mean is as large
        kv[:, 32 * blk:32 * blk + 32] = (1 + torch.rand(prior + new, 32, generator=g, device=DEV)) * 2.0 ** e
    kv[:, 540:570] *= 2.0 ** -18  # RoPE dims too
    ik, err = torch.zeros(prior + new, 128, device=DEV), _err()
    if prior:
        csa2.kv_append_ragged(c, _cu([prior]), rope, kv=kv[:prior], idx_key=ik[:prior], err=err)
    win, cu, scale = csa2.chunk_window(c, new), _cu([new]), 1 / math.sqrt(576)
    csa2.kv_append_ragged(c, cu, rope, kv=kv[prior:], idx_key=ik[prior:], win=win, err=err)
    q = _q(new, 64)
    out, lse, bits = _attn(c, q, cu, win)
    assert bits == 0 and int(err) == 0
    _within_values(out, lse, ru.chunk_attn(c, q, cu, scale, win), q, scale)


def test_attn_v4_entry_with_nan_rope():
    """A V4 entry's RoPE dims are bf16 and may be NaN: the rows that see the entry are NaN, the others know
    nothing of it."""
    n, at, H = 300, 100, 16
    c, rope = _cache(1, 320, swa=csa2.SWA_MXFP8, fmt=csa2.ENTRY_FP8), csa2.rope_table(THETA, 320)
    g = torch.Generator(device=DEV).manual_seed(6)
    kv, ik = torch.randn(n, 576, generator=g, device=DEV), torch.randn(n, 128, generator=g, device=DEV)
    kv[at, 530] = math.nan
    cu, win = _cu([n]), csa2.chunk_window(c, n)
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, win=win)
    assert c.rope_codes[0, at].view(torch.bfloat16).isnan().any()
    q = _q(n, H)
    out, lse, e = _attn(c, q, cu, win)
    assert e == 0 and out[at + 1:].isnan().all() and lse[at + 1:].isnan().all()
    c.rope_codes[0, at] = 0  # (the plain form would multiply it by zero)
    ref = ru.chunk_attn(c, q, cu, 1 / math.sqrt(576), win)
    ru.attn_within(out[:at + 1], lse[:at + 1], [t[:at + 1] for t in ref])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_the_least_values(dtype):
    """MXFP8 blocks down to the least scale: exact in fp32; in bf16 rounded to its step of 2^-133."""
    c, rope = _cache(1, 64, fmt=csa2.ENTRY_FP8), csa2.rope_table(THETA, 64)
    g = torch.Generator(device=DEV).manual_seed(6)
    kv = torch.randn(20, 576, generator=g, device=DEV)
    for i in range(20):
        kv[i, :512] *= 2.0 ** (-133 + i)
    kv[:, 512:] = 0.0
    csa2.kv_append_ragged(c, _cu([20]), rope, kv=kv, idx_key=torch.zeros(20, 128, device=DEV))
    main, win = torch.empty(20, 576, dtype=dtype, device=DEV), torch.empty(1, 128, 576, dtype=dtype, device=DEV)
    csa2.kv_read(c, _cu([20]), out_main=main, start=torch.zeros(1, dtype=torch.int64, device=DEV))
    csa2.window_read(c, win)
    want = ru.main_values(c, torch.arange(20, device=DEV))
    assert (want[:, :512] != 0).any() and torch.equal(want, want.float().double())
    if dtype == torch.bfloat16:
        want = (want * 2.0 ** 133).round() * 2.0 ** -133
    for got in (main, win[0, -20:]):
        assert torch.equal(got[:, :512].double(), want[:, :512])


@pytest.mark.parametrize("fmt,swa", [(csa2.ENTRY_FP8, csa2.SWA_BF16), (csa2.ENTRY_FP8, csa2.SWA_MXFP8)])
def test_attn_latents_beside_large_rope_dims(fmt, swa):
    """RoPE dims of about 2^18 beside latents of about 1: s is 2^-8 of the power of two below the key's largest."""
    n, H = 200, 16
    c, rope = _cache(1, 320, swa=swa, fmt=fmt), csa2.rope_table(THETA, 320)
    g = torch.Generator(device=DEV).manual_seed(8)
    kv, ik = torch.randn(n, 576, generator=g, device=DEV), torch.zeros(n, 128, device=DEV)
    kv[:, 512:] *= 2.0 ** 18
    cu, win, scale = _cu([n]), csa2.chunk_window(c, n), 1 / math.sqrt(576)
    csa2.kv_append_ragged(c, cu, rope, kv=kv, idx_key=ik, win=win)
    q = _q(n, H)
    q[..., 512:] *= 2.0 ** -18
    out, lse, e = _attn(c, q, cu, win)
    assert e == 0
    top = max(float(t.abs().max()) for t in (ru.main_values(c, torch.arange(n, device=DEV)),
                                             ru.window_values(win.codes[128:], win.scales[128:], swa)))
    _within_values(out, lse, ru.chunk_attn(c, q, cu, scale, win), q, scale, 2.0 ** (math.frexp(top)[1] - 1 - 8))
