"""What the Python binding of pages, slots, queries, values and 4-bit matrices refuses
before anything is launched (no GPU: stand-ins for device tensors, a recorder in place of
the library call)."""
import types

import pytest
import torch

from fp4_compressed_sparse_gb300 import csa2
from test_ragged_binding import BF16, Fake, I32, I64, U8


@pytest.fixture
def calls(monkeypatch):
    got = []
    monkeypatch.setattr(csa2, "_submit", lambda fn, dev, stream, *args: got.append((fn, dev, args)))
    return got


def _cache(dev=0, batch=2, pages=4, table=True):
    c = types.SimpleNamespace(n_tokens=Fake(batch, dtype=I64, dev=dev), batch=batch, n_pages=pages,
                              block_table=Fake(batch, 2, dtype=I32, dev=dev) if table else None, address=lambda: 64)
    return c


def _pool(dev=0, batch=2, pages=4):
    return types.SimpleNamespace(sizes=(dev, pages, batch), address=32)


def _resize(c=None, pool=None, dev=0, **kw):
    a = dict(cu_new=Fake(3, dtype=I32, dev=dev))
    a.update(kw)
    csa2.pages_resize(c or _cache(dev), pool or _pool(), **a)


def _slots(c=None, dev=0, **kw):
    a = dict(cu_new=Fake(3, dtype=I32, dev=dev), slots=Fake(5, dtype=I64, dev=dev), pos=Fake(5, dtype=I64, dev=dev))
    a.update(kw)
    csa2.slot_map(c or _cache(dev), a.pop("cu_new"), **a)


def _query(dev=0, H=4, dim=128, T=3, **kw):
    a = dict(q=Fake(T, H * (dim + 64), dtype=BF16, dev=dev), w_uk=Fake(H, dim, 512, dtype=BF16, dev=dev), pos=Fake(T, dtype=I64, dev=dev),
             rope_cs=Fake(9, 32, 2, dev=dev), out=Fake(T, H, 576, dtype=BF16, dev=dev))
    a.update(kw)
    csa2.query_latent(**a)


def _value(dev=0, H=4, dim=128, T=3, **kw):
    a = dict(o=Fake(T, H, 512, dev=dev), w_uv=Fake(H, dim, 512, dtype=BF16, dev=dev), out=Fake(T, H * dim, dtype=BF16, dev=dev))
    a.update(kw)
    csa2.value_project(**a)


def _matrix(rows=3, cols=96, fmt=csa2.FP4_NV, dev=0):
    return types.SimpleNamespace(rows=rows, cols=cols, fmt=fmt, tiles=Fake(9216, dtype=U8, dev=dev), address=16)


def _quant(dev=0, **kw):
    a = dict(m=_matrix(dev=dev), x=Fake(3, 96, dev=dev))
    a.update(kw)
    csa2.fp4_quant(**a)


def _product(dev=0, **kw):
    a = dict(x=_matrix(dev=dev), w=_matrix(rows=5, dev=dev), out=Fake(3, 5, dtype=BF16, dev=dev, stride=(8, 1)))
    a.update(kw)
    csa2.fp4_product(**a)


CALLS = [_resize, _slots, _query, _value, _quant, _product]


@pytest.mark.parametrize("call", CALLS)
def test_plain_calls_pass_and_the_error_word(calls, call):
    """An error word that the device cannot write to: in host memory, on another device, of another type, empty."""
    for bad in (Fake(1, dtype=I32, dev=-1), Fake(1, dtype=I32, dev=1), Fake(1, dtype=I64), Fake(0, dtype=I32)):
        with pytest.raises(ValueError, match="err"):
            call(err=bad)
    assert not calls
    call(err=Fake(1, dtype=I32, ptr=4096))
    call()
    assert len(calls) == 2 and 4096 in calls[0][2] and 4096 not in calls[1][2] and all(c[1] == 0 for c in calls)


@pytest.mark.parametrize("call", [_slots, _query, _value, _quant, _product])
def test_host_memory(calls, call):
    """Everything in host memory agrees on a device too, but not on one that the kernels can read."""
    with pytest.raises(ValueError):
        call(dev=-1)
    assert not calls


@pytest.mark.parametrize("call,kw", [
    (_resize, dict(c=_cache(table=False))), (_resize, dict(pool=_pool(pages=5))), (_resize, dict(pool=_pool(batch=3))), (_resize, dict(pool=_pool(dev=1))),
    (_resize, dict(cu_new=Fake(4, dtype=I32))), (_resize, dict(cu_new=Fake(3, dtype=I64))), (_resize, dict(cu_new=Fake(3, dtype=I32, dev=1))),
    (_resize, dict(cu_new=None, target=Fake(3, dtype=I64))), (_resize, dict(cu_new=None, target=Fake(2, dtype=I32))), (_resize, dict(granted=Fake(3, dtype=I32))),
    (_resize, dict(granted=Fake(2, dtype=I64))), (_resize, dict(cu_new=Fake(3, dtype=I32, stride=(2,)))),
    (_slots, dict(slots=None, pos=None)), (_slots, dict(slots=Fake(4, dtype=I64))), (_slots, dict(pos=Fake(5, dtype=I32))), (_slots, dict(cu_new=None)),
    (_slots, dict(pos=Fake(5, dtype=I64, dev=1))), (_slots, dict(cu_new=Fake(2, dtype=I32))),
    (_query, dict(q=Fake(3, 767, dtype=BF16))), (_query, dict(q=Fake(4, 768, dtype=BF16))), (_query, dict(q=Fake(3, 768))), (_query, dict(q=Fake(3, 768, dtype=BF16, stride=(768, 2)))),
    (_query, dict(q=Fake(3, 768, dtype=BF16, stride=(700, 1)))), (_query, dict(w_uk=Fake(4, 128, 511, dtype=BF16))), (_query, dict(w_uk=Fake(4, 128, 512))),
    (_query, dict(w_uk=Fake(4, 128, 512, dtype=BF16, dev=1))), (_query, dict(w_uk=Fake(4, 128, 512, dtype=BF16, stride=(128 * 512, 1024, 1)))),
    (_query, dict(w_uk=Fake(4, 128, 512, dtype=BF16, stride=(512, 512, 1)))), (_query, dict(w_uk=Fake(512, 512, dtype=BF16))), (_query, dict(pos=Fake(2, dtype=I64))),
    (_query, dict(pos=Fake(3, dtype=I32))), (_query, dict(rope_cs=Fake(9, 64, 2))), (_query, dict(rope_cs=Fake(9, 32, 2, dtype=BF16))), (_query, dict(out=Fake(3, 4, 512, dtype=BF16))),
    (_query, dict(out=Fake(3, 4, 576))), (_query, dict(out=Fake(3, 4, 576, dtype=BF16, stride=(4 * 600, 600, 1)))),
    (_value, dict(o=Fake(3, 4, 576))), (_value, dict(o=Fake(3, 4, 512, dtype=torch.float16))), (_value, dict(o=Fake(2, 4, 512))), (_value, dict(o=Fake(3, 4, 512, dev=1))),
    (_value, dict(o=Fake(3, 4, 512, stride=(4 * 520, 520, 1)))), (_value, dict(o=Fake(3, 4, 512, stride=(2000, 512, 1)))),
    (_value, dict(o=Fake(3, 4, 512, stride=(4096, 1024, 2)))), (_value, dict(o=Fake(3, 512))), (_value, dict(out=Fake(3, 512))), (_value, dict(out=Fake(3, 500, dtype=BF16))), (_value, dict(w_uv=Fake(3, 128, 512, dtype=BF16))),
    (_quant, dict(x=Fake(3, 95))), (_quant, dict(x=Fake(2, 96))), (_quant, dict(x=Fake(3, 96, dtype=torch.float64))), (_quant, dict(x=Fake(3, 96, dev=1))),
    (_quant, dict(x=Fake(3, 96, stride=(1, 3)))), (_quant, dict(x=Fake(3, 96, stride=(40, 1)))), (_quant, dict(x=Fake(288))),
    (_product, dict(out=Fake(3, 6, dtype=BF16))), (_product, dict(out=Fake(3, 5, dtype=I32))), (_product, dict(w=_matrix(rows=5, dev=1))), (_product, dict(out=Fake(5, 3, dtype=BF16)))])
def test_refusals(calls, call, kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert not calls


def test_a_single_row_of_any_stride(calls):
    """A single row needs no row stride: the call gets one that the library takes."""
    _quant(m=_matrix(rows=1, cols=90), x=Fake(1, 90, stride=(90, 1)))
    _product(x=_matrix(rows=1), w=_matrix(rows=5), out=Fake(1, 5, stride=(5, 1)))
    _query(T=1, q=Fake(1, 768, dtype=BF16, stride=(3, 1)))
    assert calls[0][2][2] == 96 and calls[1][2][3] == 8 and calls[2][2][1] == 768


def test_empty_calls_submit_nothing(calls):
    _slots(slots=Fake(0, dtype=I64), pos=Fake(0, dtype=I64))
    _query(T=0)
    _value(T=0)
    _quant(m=_matrix(rows=0), x=Fake(0, 96))
    _product(x=_matrix(rows=0), out=Fake(0, 5, dtype=BF16))
    _product(w=_matrix(rows=0), out=Fake(3, 0, dtype=BF16))
    assert not calls


def test_matrix_and_pool_constructors():
    for bad in ((-1, 8, 0), (1 << 25, 8, 0), (1, 0, 0), (1, 1 << 18, 0), (1, 8, 2)):
        with pytest.raises(ValueError):
            csa2.Fp4Matrix(*bad, device="cpu")
    m = csa2.Fp4Matrix(130, 200, csa2.FP4_MX, device="cpu")
    assert m.tiles.numel() == 4 * 8704 and m.row_scales.numel() == 256
    with pytest.raises(ValueError, match="CUDA"):
        csa2.fp4_quant(m, torch.zeros(130, 200))
    with pytest.raises(ValueError, match="dense"):
        csa2.PagePool(_cache(table=False))
    with pytest.raises(ValueError, match="together"):
        csa2.PagePool(_cache(), free=Fake(4, dtype=I32))


@pytest.mark.parametrize("call,kw", [(c, {k: None}) for c, names in ((_query, ("q", "w_uk", "pos", "rope_cs", "out")), (_value, ("o", "w_uv", "out")),
                                                                     (_quant, ("x",)), (_product, ("out",))) for k in names]
                         + [(_query, dict(out=Fake(dtype=BF16))), (_query, dict(rope_cs=Fake())), (_query, dict(pos=Fake(dtype=I64), T=1)),
                            (_value, dict(out=Fake(dtype=BF16))), (_slots, dict(pos=Fake(5, 1, dtype=I64))), (_resize, dict(granted=Fake(2, 1, dtype=I32)))])
def test_no_tensor_or_one_of_other_dimensions(calls, call, kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert not calls
