"""Host-side refusals and sizes of the ragged calls (no GPU work: every pointer is
a 16-byte aligned fake that is never touched)."""
import ctypes

import pytest

FAKE = 1 << 20
P = ctypes.c_void_p(FAKE)
ODD = ctypes.c_void_p(FAKE + 4)


@pytest.fixture(scope="module")
def lib():
    from fp4_compressed_sparse_gb300 import build_lib, csa2
    build_lib.build()
    return csa2.load()


def _cache(**kw):
    from fp4_compressed_sparse_gb300 import csa2
    st = csa2.CacheStruct(2, 256, 1, 1, *([FAKE] * 10))
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def _append(lib, st=None, **kw):
    a = dict(kv=P, kvs=576, ik=P, iks=128, dt=0, cmp=None, cu=P, total=4, mx=4, rope=P, rl=300, wc=None, ws=None)
    a.update(kw)
    st = st or _cache()
    return lib.csa2_kv_append_ragged(ctypes.byref(st), a["kv"], a["kvs"], a["ik"], a["iks"], a["dt"], a["cmp"], a["cu"],
                                     a["total"], a["mx"], a["rope"], a["rl"], a["wc"], a["ws"], None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(kv=None), 1, b"kv is NULL"), (dict(ik=ODD), 3, b"idx_key is not"), (dict(cu=None), 1, b"cu_new is NULL"),
    (dict(cu=ODD), 3, b"cu_new"), (dict(kvs=575), 2, b"kv_stride"), (dict(kvs=580), 2, b"kv_stride"),
    (dict(iks=120), 2, b"key_stride"), (dict(dt=2), 4, b"in_dtype"), (dict(total=-1), 2, b"total"),
    (dict(total=(1 << 24) + 1), 2, b"total"), (dict(mx=-1), 2, b"max_new"), (dict(rope=None), 1, b"rope_cs"),
    (dict(rl=0), 2, b"rope_len"), (dict(wc=P), 1, b"win_scales is NULL"), (dict(wc=ODD, ws=P), 3, b"win_codes"),
    (dict(total=0), 0, b""), (dict(mx=0), 0, b"")])
def test_append_refusals(lib, kw, status, text):
    assert _append(lib, **kw) == status
    if status:
        assert text in lib.csa2_last_error_detail()


def test_append_ratio_rules(lib):
    from fp4_compressed_sparse_gb300 import csa2
    cin = csa2.CompressIn(*([FAKE] * 6))
    assert _append(lib, cmp=ctypes.byref(cin)) == 4
    r2 = _cache(ratio=2)
    assert _append(lib, r2) == 1 and b"cmp is NULL" in lib.csa2_last_error_detail()
    cin.zb = FAKE + 8
    assert _append(lib, r2, cmp=ctypes.byref(cin)) == 3
    cin.zb = FAKE
    assert _append(lib, r2, cmp=ctypes.byref(cin), kv=None, ik=None, total=0) == 0
    assert _append(lib, _cache(ratio=3)) == 4 and _append(lib, _cache(batch=0)) == 2


def _read(lib, st=None, **kw):
    a = dict(cu=P, total=4, pos=None, start=P, main=P, ms=576, key=P, ks=128, dt=0)
    a.update(kw)
    st = st or _cache()
    return lib.csa2_kv_read(ctypes.byref(st), a["cu"], a["total"], a["pos"], a["start"], a["main"], a["ms"], a["key"],
                            a["ks"], a["dt"], None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(cu=None), 1, b"cu_rows"), (dict(start=None), 1, b"start"), (dict(pos=ODD), 3, b"pos"),
    (dict(main=None, key=None), 1, b"both NULL"), (dict(main=ODD), 3, b"out_main"), (dict(key=ODD), 3, b"out_key"),
    (dict(ms=568), 2, b"main_stride"), (dict(ms=577), 2, b"main_stride"), (dict(ks=127), 2, b"key_stride"),
    (dict(dt=7), 4, b"out_dtype"), (dict(total=-5), 2, b"total"), (dict(total=0), 0, b""),
    (dict(total=0, main=None, ms=0), 0, b"")])
def test_read_refusals(lib, kw, status, text):
    assert _read(lib, **kw) == status
    if status:
        assert text in lib.csa2_last_error_detail()


def test_window_read_refusals(lib):
    st = _cache()
    assert lib.csa2_window_read(ctypes.byref(st), None, 0, None) == 1
    assert lib.csa2_window_read(ctypes.byref(st), ODD, 0, None) == 3
    assert lib.csa2_window_read(ctypes.byref(st), P, 2, None) == 4
    assert lib.csa2_window_read(None, P, 0, None) == 1


def _attn(lib, st=None, **kw):
    a = dict(q=P, H=64, cu=P, total=4, mx=4, wc=None, wsc=None, sink=None, scale=0.1, out=P, dt=0, lse=P, ws=P, nb=1 << 40)
    a.update(kw)
    st = st or _cache()
    return lib.csa2_chunk_attn(ctypes.byref(st), a["q"], a["H"], a["cu"], a["total"], a["mx"], a["wc"], a["wsc"], a["sink"],
                               a["scale"], a["out"], a["dt"], a["lse"], a["ws"], a["nb"], None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(q=None), 1, b"q is NULL"), (dict(q=ODD), 3, b"q is not"), (dict(H=24), 2, b"n_heads"), (dict(H=144), 2, b"n_heads"),
    (dict(H=0), 2, b"n_heads"), (dict(cu=None), 1, b"cu_q"), (dict(total=-1), 2, b"total"), (dict(mx=-2), 2, b"max_new"),
    (dict(wc=P), 1, b"win_scales"), (dict(wc=ODD, wsc=P), 3, b"win_codes"), (dict(sink=ODD), 3, b"sink"),
    (dict(scale=float("inf")), 4, b"sm_scale"), (dict(scale=float("nan")), 4, b"sm_scale"), (dict(out=None), 1, b"out"),
    (dict(dt=-1), 4, b"out_dtype"), (dict(lse=ODD), 3, b"lse"), (dict(ws=None), 7, b"workspace"), (dict(nb=8), 7, b"workspace"),
    (dict(ws=ODD), 3, b"ws is not"), (dict(total=0), 0, b""), (dict(mx=0), 0, b"")])
def test_attn_refusals(lib, kw, status, text):
    assert _attn(lib, **kw) == status
    if status:
        assert text in lib.csa2_last_error_detail()


def test_sizes(lib):
    assert lib.csa2_chunk_window_bytes(3, 10, 1, 0) == (10 + 3 * 128) * 576
    assert lib.csa2_chunk_window_bytes(3, 10, 0, 0) == (10 + 3 * 128) * 1152
    assert lib.csa2_chunk_window_bytes(3, 10, 1, 1) == (10 + 3 * 128) * 32
    assert lib.csa2_chunk_window_bytes(0, 10, 1, 0) == 0 and lib.csa2_chunk_window_bytes(1, 1, 1, 2) == 0
    assert lib.csa2_chunk_attn_workspace_size(1, 1, 16) >= 16
