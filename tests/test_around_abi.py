"""Host-side refusals and sizes of the calls around the attention: pages, slots, queries,
values, 4-bit matrices (no GPU work: every pointer is a 16-byte aligned fake that is never
touched)."""
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


def _paged(**kw):
    from fp4_compressed_sparse_gb300 import csa2
    st = csa2.CacheStruct(2, 256, 1, 1, *([FAKE] * 11), 128, 2, 4, 0)
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def _resize(lib, st=None, pool=(FAKE, FAKE, FAKE), **kw):
    from fp4_compressed_sparse_gb300 import csa2
    a = dict(target=P, cu=None, total=4, mx=4, granted=None)
    a.update(kw)
    st = st or _paged()
    ps = csa2.PoolStruct(*pool) if pool else None
    return lib.csa2_pages_resize(ctypes.byref(st), ctypes.byref(ps) if ps else None, a["target"], a["cu"], a["total"], a["mx"],
                                 a["granted"], None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(pool=None), 1, b"pool is NULL"), (dict(pool=(None, FAKE, FAKE)), 1, b"free is NULL"), (dict(pool=(FAKE, FAKE + 4, FAKE)), 3, b"n_free"),
    (dict(pool=(FAKE, FAKE, None)), 1, b"held"), (dict(target=ODD), 3, b"target"), (dict(target=None, cu=ODD), 3, b"cu_new"),
    (dict(cu=P), 4, b"both given"), (dict(granted=ODD), 3, b"granted"), (dict(total=-1), 2, b"total"),
    (dict(total=(1 << 24) + 1), 2, b"total"), (dict(mx=-1), 2, b"max_new")])
def test_resize_refusals(lib, kw, status, text):
    assert _resize(lib, **kw) == status and text in lib.csa2_last_error_detail()


def test_resize_wants_a_paged_cache(lib):
    assert _resize(lib, _paged(block_table=None)) == 1 and b"dense" in lib.csa2_last_error_detail()
    assert _resize(lib, _paged(capacity=300)) == 2 and _resize(lib, _paged(page_entries=100)) == 2


def _slots(lib, **kw):
    a = dict(cu=P, total=4, mx=4, slots=P, pos=P)
    a.update(kw)
    return lib.csa2_slot_map(ctypes.byref(_paged()), a["cu"], a["total"], a["mx"], a["slots"], a["pos"], None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(cu=None), 1, b"cu_new"), (dict(cu=ODD), 3, b"cu_new"), (dict(total=-1), 2, b"total"), (dict(mx=-3), 2, b"max_new"),
    (dict(slots=None, pos=None), 1, b"both NULL"), (dict(slots=ODD), 3, b"slots"), (dict(pos=ODD), 3, b"pos"), (dict(total=0), 0, b"")])
def test_slot_map_refusals(lib, kw, status, text):
    assert _slots(lib, **kw) == status
    if status:
        assert text in lib.csa2_last_error_detail()


def _query(lib, **kw):
    a = dict(q=P, qs=4 * 192, total=3, H=4, dim=128, w=P, ws=128 * 512, pos=P, rope=P, rl=10, out=P)
    a.update(kw)
    return lib.csa2_query_latent(a["q"], a["qs"], a["total"], a["H"], a["dim"], a["w"], a["ws"], a["pos"], a["rope"], a["rl"], a["out"],
                                 None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(q=None), 1, b"q is NULL"), (dict(q=ODD), 3, b"q is not"), (dict(qs=760), 2, b"q_stride"), (dict(qs=770), 2, b"q_stride"),
    (dict(total=-1), 2, b"total"), (dict(total=(1 << 24) + 1), 2, b"total"), (dict(H=0), 2, b"n_heads"), (dict(H=129), 2, b"n_heads"),
    (dict(dim=8), 2, b"dim"), (dict(dim=24), 2, b"dim"), (dict(dim=144), 2, b"dim"), (dict(w=None), 1, b"w_uk"), (dict(w=ODD), 3, b"w_uk"),
    (dict(ws=128 * 512 - 8), 2, b"w_stride"), (dict(ws=128 * 512 + 4), 2, b"w_stride"), (dict(pos=None), 1, b"pos"), (dict(pos=ODD), 3, b"pos"),
    (dict(rope=None), 1, b"rope_cs"), (dict(rl=0), 2, b"rope_len"), (dict(out=None), 1, b"out"), (dict(out=ODD), 3, b"out"),
    (dict(total=0, q=None, pos=None, out=None), 0, b"")])
def test_query_refusals(lib, kw, status, text):
    assert _query(lib, **kw) == status
    if status:
        assert text in lib.csa2_last_error_detail()


def _value(lib, **kw):
    a = dict(o=P, os=4 * 512, dt=0, total=3, H=4, dim=128, w=P, ws=128 * 512, out=P, ots=512)
    a.update(kw)
    return lib.csa2_value_project(a["o"], a["os"], a["dt"], a["total"], a["H"], a["dim"], a["w"], a["ws"], a["out"], a["ots"], None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(o=None), 1, b"o is NULL"), (dict(o=ODD), 3, b"o is not"), (dict(os=2040), 2, b"o_stride"), (dict(os=2052), 2, b"o_stride"),
    (dict(dt=2), 4, b"in_dtype"), (dict(dt=-1), 4, b"in_dtype"), (dict(total=-1), 2, b"total"), (dict(H=0), 2, b"n_heads"),
    (dict(H=200), 2, b"n_heads"), (dict(dim=0), 2, b"dim"), (dict(dim=130), 2, b"dim"), (dict(w=None), 1, b"w_uv"), (dict(w=ODD), 3, b"w_uv"),
    (dict(ws=512), 2, b"w_stride"), (dict(out=None), 1, b"out"), (dict(out=ODD), 3, b"out"), (dict(ots=504), 2, b"out_stride"),
    (dict(ots=516), 2, b"out_stride"), (dict(total=0, o=None, out=None), 0, b"")])
def test_value_refusals(lib, kw, status, text):
    assert _value(lib, **kw) == status
    if status:
        assert text in lib.csa2_last_error_detail()


def _m(rows=4, cols=96, fmt=0, tiles=FAKE, rs=FAKE):
    from fp4_compressed_sparse_gb300 import csa2
    return csa2.Fp4Struct(rows, cols, fmt, tiles, rs)


@pytest.mark.parametrize("m,status,text", [
    (dict(rows=-1), 2, b"rows"), (dict(rows=(1 << 24) + 1), 2, b"rows"), (dict(cols=0), 2, b"cols"), (dict(cols=(1 << 17) + 1), 2, b"cols"),
    (dict(fmt=2), 4, b"format"), (dict(tiles=None), 1, b"plane is NULL"), (dict(rs=None), 1, b"plane is NULL"),
    (dict(tiles=FAKE + 8), 3, b"plane"), (dict(rs=FAKE + 4), 3, b"plane"), (dict(rows=0, tiles=None, rs=None), 0, b"")])
def test_matrix_refusals(lib, m, status, text):
    """The same matrix checks in every call that takes one."""
    a, ok = _m(**m), _m(rows=m.get("rows", 4) if m.get("rows", 4) >= 0 else 4)
    calls = [lambda: lib.csa2_fp4_quant(ctypes.byref(a), P, 1 << 20, 0, None, None), lambda: lib.csa2_fp4_read(ctypes.byref(a), P, 1 << 20, 0, None)]
    if status:
        calls += [lambda: lib.csa2_fp4_product(ctypes.byref(a), ctypes.byref(ok), P, 1 << 25, 0, None, None),
                  lambda: lib.csa2_fp4_product(ctypes.byref(ok), ctypes.byref(a), P, 1 << 25, 0, None, None)]
        calls[2:] = [c for c in calls[2:] if ok.rows <= 1 << 24]
    for c in calls:
        assert c() == status
        if status:
            assert text in lib.csa2_last_error_detail()
    assert lib.csa2_fp4_quant(None, P, 96, 0, None, None) == 1


@pytest.mark.parametrize("kw,status,text", [
    (dict(x=None), 1, b"x is NULL"), (dict(x=ODD), 3, b"x is not"), (dict(s=88), 2, b"x_stride"), (dict(s=100), 2, b"x_stride"), (dict(dt=3), 4, b"in_dtype")])
def test_quant_refusals(lib, kw, status, text):
    a = dict(x=P, s=96, dt=0)
    a.update(kw)
    assert lib.csa2_fp4_quant(ctypes.byref(_m()), a["x"], a["s"], a["dt"], None, None) == status
    assert text in lib.csa2_last_error_detail()
    assert lib.csa2_fp4_read(ctypes.byref(_m()), a["x"], a["s"], a["dt"], None) == status


@pytest.mark.parametrize("x,w,kw,status,text", [
    (dict(), dict(fmt=1), {}, 4, b"differ"), (dict(), dict(cols=104), {}, 2, b"columns"), (dict(), dict(rows=7), dict(out=None), 1, b"out"),
    (dict(), dict(), dict(out=ODD), 3, b"out"), (dict(), dict(rows=9), dict(s=8), 2, b"out_stride"), (dict(), dict(rows=9), dict(s=12), 2, b"out_stride"),
    (dict(), dict(), dict(dt=9), 4, b"out_dtype"), (dict(rows=0), dict(), {}, 0, b""), (dict(), dict(rows=0), {}, 0, b"")])
def test_product_refusals(lib, x, w, kw, status, text):
    a = dict(out=P, s=16, dt=1)
    a.update(kw)
    assert lib.csa2_fp4_product(ctypes.byref(_m(**x)), ctypes.byref(_m(**w)), a["out"], a["s"], a["dt"], None, None) == status
    if status:
        assert text in lib.csa2_last_error_detail()


def test_plane_sizes(lib):
    f = lib.csa2_fp4_plane_bytes
    assert f(1, 1, 0, 0) == 9216 and f(1, 1, 1, 0) == 8704 and f(1, 1, 0, 1) == 512
    assert f(129, 4104, 0, 0) == 2 * 33 * 9216 and f(129, 4104, 1, 0) == 2 * 33 * 8704 and f(129, 4104, 1, 1) == 256 * 4
    assert f(0, 64, 0, 0) == 0 and f(-1, 64, 0, 0) == 0 and f(4, 0, 0, 0) == 0 and f(4, 64, 2, 0) == 0 and f(4, 64, 0, 2) == 0
    assert f(1 << 24, 1 << 17, 0, 0) == (1 << 17) * 1024 * 9216  # (beyond 32 bits)
