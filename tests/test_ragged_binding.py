"""What the Python binding of the ragged calls refuses before anything is launched (no GPU: stand-ins for
device tensors, and a recorder in place of the library call)."""
import types

import pytest
import torch

from fp4_compressed_sparse_gb300 import csa2


class Fake:
    """What the binding reads of a tensor."""

    def __init__(self, *shape, dtype=torch.float32, dev=0, stride=None, ptr=1 << 20):
        self.shape, self.dtype, self.dev, self.ptr = torch.Size(shape), dtype, dev, ptr
        dense = [1]
        for n in reversed(shape[1:]):
            dense.insert(0, dense[0] * n)
        self.dense, self.strides = tuple(dense[:len(shape)]), tuple(stride or dense[:len(shape)])

    device = property(lambda self: f"cuda:{self.dev}" if self.dev >= 0 else "cpu")
    is_cuda = property(lambda self: self.dev >= 0)
    get_device = lambda self: self.dev
    dim = lambda self: len(self.shape)
    numel = lambda self: self.shape.numel()
    stride = lambda self, d=None: self.strides if d is None else self.strides[d]
    is_contiguous = lambda self: all(n == 1 or a == b for n, a, b in zip(self.shape, self.strides, self.dense))
    data_ptr = lambda self: self.ptr
    view = lambda self, *shape: Fake(*shape, dtype=self.dtype, dev=self.dev, ptr=self.ptr) if shape != (-1,) else self
    __getitem__ = lambda self, at: self


I32, I64, BF16, U8 = torch.int32, torch.int64, torch.bfloat16, torch.uint8


@pytest.fixture
def calls(monkeypatch):
    got = []
    monkeypatch.setattr(csa2, "_call", lambda fn, cache, dev, stream, *args: got.append((fn, dev, args)))
    return got


def _cache(dev=0, batch=2):
    return types.SimpleNamespace(n_tokens=Fake(batch, dtype=I64, dev=dev), batch=batch, ratio=1, swa_dtype=csa2.SWA_MXFP8)


def _append(c, dev=0, **kw):
    a = dict(kv=Fake(3, 576, dev=dev), idx_key=Fake(3, 128, dev=dev), err=None)
    a.update(kw)
    csa2.kv_append_ragged(c, Fake(3, dtype=I32, dev=dev), Fake(64, 32, 2, dev=dev), **a)


def _read(c, dev=0, **kw):
    a = dict(out_main=Fake(3, 576, dev=dev), start=Fake(2, dtype=I64, dev=dev), err=None)
    a.update(kw)
    csa2.kv_read(c, Fake(3, dtype=I32, dev=dev), **a)


def _attn(c, dev=0, **kw):
    csa2.chunk_attn(c, Fake(3, 64, 576, dtype=BF16, dev=dev), Fake(3, dtype=I32, dev=dev), Fake(3, 64, 512, dev=dev),
                    Fake(3, 64, dev=dev), Fake(1 << 20, dtype=U8, dev=dev), 0.1, **kw)


CALLS = [_append, _read, _attn]


@pytest.mark.parametrize("call", CALLS)
def test_the_error_word_is_a_device_int32(calls, call):
    """An error word that the device cannot write to: in host memory, on another device, of another type, empty."""
    for bad in (Fake(1, dtype=I32, dev=-1), Fake(1, dtype=I32, dev=1), Fake(1, dtype=I64), Fake(0, dtype=I32)):
        with pytest.raises(ValueError, match="err"):
            call(_cache(), err=bad)
    assert not calls
    call(_cache(), err=Fake(1, dtype=I32, ptr=4096))
    call(_cache())
    assert len(calls) == 2 and 4096 in calls[0][2] and 4096 not in calls[1][2]


@pytest.mark.parametrize("call", CALLS + [lambda c, dev: csa2.window_read(c, Fake(2, 128, 576, dev=dev))])
def test_a_cache_in_host_memory(calls, call):
    """Everything in host memory agrees on a device too, but not on one that the kernels can read."""
    with pytest.raises(ValueError):
        call(_cache(dev=-1), dev=-1)
    assert not calls


@pytest.mark.parametrize("rows", [1, 2])
def test_rows_are_contiguous_within(calls, rows):
    """Every second column of a wider tensor, also for a single row; a single row of any row stride is fine."""
    c, cu, rope = _cache(), Fake(3, dtype=I32), Fake(64, 32, 2)
    every2 = lambda w: Fake(rows, w, stride=(2 * w, 2))
    start = Fake(2, dtype=I64)
    for bad in (lambda: csa2.kv_append_ragged(c, cu, rope, kv=every2(576), idx_key=Fake(rows, 128)),
                lambda: csa2.kv_append_ragged(c, cu, rope, kv=Fake(rows, 576), idx_key=every2(128)),
                lambda: csa2.kv_read(c, cu, out_main=every2(576), start=start),
                lambda: csa2.kv_read(c, cu, out_key=every2(128), start=start)):
        with pytest.raises(ValueError, match="contiguous"):
            bad()
    assert not calls
    if rows == 1:
        csa2.kv_append_ragged(c, cu, rope, kv=Fake(1, 576, stride=(1, 1)), idx_key=Fake(1, 128, stride=(7, 1)))
        csa2.kv_read(c, cu, out_main=Fake(1, 576, stride=(0, 1)), start=start)
        assert len(calls) == 2 and calls[0][2][1] == 576 and calls[0][2][3] == 128


PLANES = dict(lat_codes=256 * 256, lat_scales=32 * 256, rope_codes=32 * 256, rope_scales=4 * 256, idx_codes=2 * 8192,
              idx_scales=2 * 512, swa_codes=2 * 128 * 576, swa_scales=2 * 128 * 32)


@pytest.fixture(scope="module")
def lib():
    from fp4_compressed_sparse_gb300 import build_lib
    build_lib.build()
    return csa2.load()


def _planes(ratio=1):
    """Planes of 2 sequences of 128 entries (dense, or two pages)."""
    p = {k: Fake(n, dtype=U8) for k, n in PLANES.items()}
    p["n_tokens"] = Fake(2, dtype=I64)
    if ratio == 2:
        p["cmp_buf"] = Fake(2, 4, 4, 704)
    return p


@pytest.mark.parametrize("ratio", [1, 2])
def test_from_planes_on_one_device(lib, ratio):
    """A plane or a block table on another device than the token counts: every plane in turn."""
    paged = dict(page_entries=128, n_pages=2)
    table = Fake(2, 1, dtype=I32)
    csa2.Cache.from_planes(2, 128, _planes(ratio), ratio=ratio)
    csa2.Cache.from_planes(2, 128, _planes(ratio), ratio=ratio, block_table=table, **paged)
    for name in _planes(ratio):
        p = _planes(ratio)
        p[name].dev = 1
        with pytest.raises(ValueError):
            csa2.Cache.from_planes(2, 128, p, ratio=ratio)
    with pytest.raises(ValueError, match="block_table"):
        csa2.Cache.from_planes(2, 128, _planes(ratio), ratio=ratio, block_table=Fake(2, 1, dtype=I32, dev=1), **paged)
    p = _planes(ratio)
    del p["n_tokens"]
    with pytest.raises(ValueError, match="n_tokens"):
        csa2.Cache.from_planes(2, 128, p, ratio=ratio)
