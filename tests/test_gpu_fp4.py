"""4-bit block-scaled matrices on the GPU: csa2_fp4_quant and csa2_fp4_read against
the definition in 64 bits (equal), csa2_fp4_product against a 64-bit product of the
stored values."""
import math

import pytest
import torch

import fp4_util as fu
from fp4_compressed_sparse_gb300 import csa2

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = [csa2.FP4_NV, csa2.FP4_MX]
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp4_compressed_sparse_gb300 import build_lib
    build_lib.build()
    csa2.load()


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _rows(rows, cols, dtype, seed=0):
    """N(0,1) rows of several magnitudes, groups of zeros, a row of zeros, rows of grid midpoints."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = x * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g, device=DEV).float())
    x[1::5] *= torch.exp2(torch.randint(-8, 8, (x[1::5].shape[0], cols), generator=g, device=DEV).float())
    x[2::7, :40] = 0.0
    x[3::11] = 0.0
    # small multiples of 1/4 with the group's largest value among 6, 12, .. : quotients at the midpoints
    mid = torch.randint(-24, 25, (rows, cols), generator=g, device=DEV).float() / 4
    mid[:, ::16] = 6.0 * torch.randint(1, 8, mid[:, ::16].shape, generator=g, device=DEV).float()
    x[4::6] = mid[4::6]
    return x.to(dtype)


def _packed(x, fmt, err=None):
    m = csa2.Fp4Matrix(*x.shape, fmt)
    csa2.fp4_quant(m, x, err=err)
    return m


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 136), (17, 31), (130, 520), (129, 4104), (2000, 264), (1300, 2056), (1217, 130), (1400, 6000), (1290, 17000),
                                       (7, 8192), (9, 8200), (2, 20000), (5, 2049), (3, 6144), (1221, 500),
                                       (1220, 1000), (1300, 4096), (1219, 4100), (1225, 8192), (1218, 8200), (1219, 10400),
                                       (1221, 5), (1250, 8), (1231, 20003), (1229, 2050), (4900, 136), (4871, 2050), (4866, 3001), (5003, 4099), (4865, 14200), (1221, 13990), (1219, 28605)])
def test_quant_is_the_definition(fmt, dtype, rows, cols):
    """Codes and scales as values, equal; read back in both types; strided rows; columns behind the
    last one of the tile are zeros."""
    wide = torch.full((rows, -(-cols // 8) * 8 + 16), float("nan"), dtype=dtype, device=DEV)
    wide[:, :cols] = _rows(rows, cols, dtype, rows + cols)
    x, err = wide[:, :cols], _err()
    m = csa2.Fp4Matrix(rows, cols, fmt)
    m.tiles.fill_(0x5A)
    csa2.fp4_quant(m, x, err=err)
    want = fu.quantised(x, fmt)
    assert int(err) == 0
    got = fu.values(m)
    assert torch.equal(got, want)
    full = fu.values(type("M", (), dict(vars(m), cols=-(-cols // 128) * 128)))
    assert not full[:, cols:].any()
    for out_t in TYPES:
        out = torch.full((rows, -(-cols // 8) * 8 + 8), 7.0, dtype=out_t, device=DEV)
        csa2.fp4_read(m, out[:, :cols])
        assert torch.equal(out[:, :cols].double(), want) and (out[:, cols:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_nv_codes_at_every_midpoint(dtype):
    """x at T s, and one step of its type beside it, for every scale s and midpoint T of the grid."""
    s = torch.arange(8, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    at = (s[:, None] * t).to(dtype)
    up, down = (torch.nextafter(at, torch.full_like(at, v)) for v in (math.inf, 0.0))
    x = torch.zeros(s.numel() + 1, 32, dtype=dtype)
    x[:-1, :16] = torch.cat([at, -up, torch.zeros_like(at[:, :1]), (6 * s)[:, None].to(dtype)], -1)
    x[:-1, 16:] = torch.cat([-at, down, torch.zeros_like(at[:, :1]), (6 * s)[:, None].to(dtype)], -1)
    # one row of 2688 beside each fixes the row's power of two at 1
    y = torch.zeros(s.numel() + 1, 48, dtype=dtype)
    y[:, :32], y[:, 40] = x, 2688.0
    y = y.to(DEV)
    m = _packed(y, csa2.FP4_NV)
    assert (m.row_scales[:y.shape[0]] == 1).all()
    assert torch.equal(fu.values(m), fu.quantised(y, csa2.FP4_NV))


@pytest.mark.parametrize("fmt", FMTS)
def test_quant_extreme_rows(fmt):
    """The largest and least magnitudes, and rows of infinities and NaN: NaN wholly, the others untouched."""
    x = torch.randn(5001, 96, device=DEV)
    x[0] *= 2.0 ** 60
    x[1] *= 2.0 ** -100
    x[2] *= 2.0 ** -140
    x[3, 5], x[4, 90], x[5, 33] = math.inf, -math.inf, math.nan
    x[6] = 2688.0 * 2.0 ** 62
    x[7] = torch.nextafter(torch.tensor(2688.0 * 2.0 ** 62), torch.tensor(math.inf)).item()
    x[8] = torch.finfo(torch.float32).max
    x[9] = 2.0 ** -149
    for rows in (12, 1500, 5001):
        err, y = _err(), x[:rows]
        m = _packed(y, fmt, err)
        want = fu.quantised(y, fmt)
        got = fu.values(m)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())
        nan = {3, 4, 5} | ({7, 8} if fmt == csa2.FP4_NV else set())
        assert set(torch.isnan(got).all(-1).nonzero().flatten().tolist()) == nan and int(err) == csa2.DEVERR_NAN
        out = torch.empty(rows, 96, device=DEV)
        csa2.fp4_read(m, out)
        assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out.double().nan_to_num(), want.nan_to_num())


def test_rows_behind_the_last_are_not_written():
    for fmt in FMTS:
        m = csa2.Fp4Matrix(5, 256, fmt)
        m.tiles.fill_(0xA5)
        m.row_scales.fill_(-3.0)
        csa2.fp4_quant(m, torch.ones(5, 256, device=DEV))
        rec = m.tiles.view(2, -1)
        codes = rec[:, :8192].reshape(2, 4, 128, 16)
        assert (codes[:, :, 5:] == 0xA5).all() and not (codes[:, :, :5] == 0xA5).any()
        sc = rec[:, 8192:].reshape(-1, 32, 4, 4)
        assert (sc[:, 5:] == 0xA5).all() and (sc[:, :5, 1:] == 0xA5).all() and (m.row_scales[5:] == -3).all()


def _within(out, x, w):
    """out against the 64-bit product of the stored values.

    Products with their block scales are exact in the MMA, which adds 64 of them to the
    sum per step: each step is off by at most one unit of fp32, 2^-23 of the magnitudes
    added up so far, and so are the joins of up to 8 partial sums.  bf16 adds half a step."""
    xv, wv = fu.values(x), fu.values(w)
    want, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    tol = (-(-x.cols // 64) + 10) * 2.0 ** -23 * mag
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    err = (out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).nan_to_num().max())


SHAPES = [(1, 8, 128), (1, 700, 4096), (5, 129, 40), (16, 256, 1000), (17, 130, 384), (33, 1000, 2048), (64, 96, 128),
          (65, 704, 640), (128, 128, 8192), (129, 1, 256), (300, 2056, 136), (1, 1, 1), (501, 704, 4104), (2, 12288, 512),
          (1000, 4100, 264), (2049, 2500, 520), (70, 900, 3000), (250, 700, 1100), (96, 6200, 300), (1, 300, 20000),
          (65, 8200, 128), (200, 96, 5000)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(fmt, dtype, M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + N)
    x, w = (torch.randn(r, K, generator=g, device=DEV) * torch.exp2(torch.randint(-9, 9, (r, 1), generator=g, device=DEV).float())
            for r in (M, N))
    pad = -(-K // 8) * 8
    xs, ws = (torch.zeros(t.shape[0], pad, device=DEV) for t in (x, w))
    xs[:, :K], ws[:, :K] = x, w
    mx, mw, err = _packed(xs[:, :K], fmt), _packed(ws[:, :K], fmt), _err()
    out = torch.full((M + 1, -(-N // 8) * 8 + 8), 3.0, dtype=dtype, device=DEV)
    csa2.fp4_product(mx, mw, out[:M, :N], err=err)
    assert int(err) == 0
    _within(out[:M, :N], mx, mw)
    assert (out[M] == 3).all() and (out[:, N:] == 3).all()
    again = torch.empty_like(out)
    csa2.fp4_product(mx, mw, again[:M, :N], err=err)
    assert torch.equal(out[:M, :N], again[:M, :N])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N", [(3, 200), (100, 50), (400, 300), (2600, 3000)])
def test_product_of_small_integers_is_exact(fmt, M, N):
    """Values of the grid under scales that are powers of two: every sum fits fp32."""
    g = torch.Generator(device=DEV).manual_seed(1)
    t = torch.tensor(fu.GRID + [-v for v in fu.GRID], device=DEV)
    x, w = (t[torch.randint(0, 16, (r, 1160), generator=g, device=DEV)] for r in (M, N))
    x[:, ::16] = 6.0
    w[:, ::16] = -6.0
    mx, mw = _packed(x, fmt), _packed(w, fmt)
    assert torch.equal(fu.values(mx), x.double()) and torch.equal(fu.values(mw), w.double())
    out = torch.empty(M, -(-N // 8) * 8, device=DEV)[:, :N]  # (row strides are multiples of 8)
    csa2.fp4_product(mx, mw, out)
    assert torch.equal(out.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("M", [30, 700, 2100])
def test_a_matrix_with_itself(M):
    m = _packed(_rows(M, 264, torch.float32, 3).clamp(-1e3, 1e3), csa2.FP4_NV)
    out = torch.empty(M, -(-M // 8) * 8, device=DEV)[:, :M]
    csa2.fp4_product(m, m, out)
    _within(out, m, m)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_of_nonfinite_rows(fmt):
    """A row with an infinity or NaN makes its row (column) NaN and nothing else; zero rows are zeros."""
    for M, N in ((20, 300), (2600, 3000)):
        x, w = torch.randn(M, 192, device=DEV), torch.randn(N, 192, device=DEV)
        x[3, 100], w[200, 0], x[7] = math.nan, math.inf, 0.0
        out = torch.empty(M, -(-N // 8) * 8, device=DEV)[:, :N]
        csa2.fp4_product(_packed(x, fmt), _packed(w, fmt), out)
        nan = torch.isnan(out)
        assert nan[3].all() and nan[:, 200].all() and int(nan.sum()) == M + N - 1
        out[3] = 0
        out[:, 200] = 0
        assert not out[7].any()


@pytest.mark.parametrize("M", [1, 40, 2600])
def test_streams_graphs_and_two_calls_at_once(M):
    """A captured quantisation and product replayed on new inputs, another stream than the tensors' own,
    two products at once over one weight."""
    N, K = 2600, 520
    w = _packed(torch.randn(N, K, device=DEV), csa2.FP4_NV)
    x, y = torch.randn(M, K, device=DEV), torch.randn(M, K, device=DEV)
    m, n = csa2.Fp4Matrix(M, K), csa2.Fp4Matrix(M, K)
    o, p = torch.empty(M, N, device=DEV), torch.empty(M, N, device=DEV)
    want = []
    for t in (x, y):
        csa2.fp4_quant(m, t)
        csa2.fp4_product(m, w, o)
        want.append(o.clone())
    torch.cuda.synchronize()
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    buf = x.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        csa2.fp4_quant(m, buf)
        csa2.fp4_product(m, w, o)
    for t, v in ((x, want[0]), (y, want[1])):
        buf.copy_(t)
        graph.replay()
        csa2.fp4_quant(n, y, stream=other)
        csa2.fp4_product(n, w, p, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(o, v) and torch.equal(p, want[1])


@pytest.mark.parametrize("M,stride", [(20, (1 << 27) + 8), (2600, (1 << 20) + 8)])
def test_rows_far_apart(M, stride):
    """Row offsets that pass 32 bits: rows in, values out and sums out, against rows that lie together."""
    N, K = 2600, 264
    x = _rows(M, K, torch.bfloat16, 5).clamp(-1e3, 1e3)
    w = _packed(_rows(N, K, torch.bfloat16, 6).clamp(-1e3, 1e3), csa2.FP4_NV)
    wide = torch.empty((M - 1) * stride + N, dtype=torch.bfloat16, device=DEV)
    far = wide.as_strided((M, K), (stride, 1))
    far.copy_(x)
    m, n = _packed(far, csa2.FP4_NV), _packed(x, csa2.FP4_NV)
    v = torch.empty_like(x)
    csa2.fp4_read(n, v)
    far.zero_()
    csa2.fp4_read(m, far)
    assert torch.equal(far, v)
    sums, far = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), wide.as_strided((M, N), (stride, 1))
    csa2.fp4_product(n, w, sums)
    csa2.fp4_product(m, w, far)
    assert torch.equal(far, sums)


def test_calls_behind_one_another():
    """Calls whose launches overlap: each reads what the one before has just written, over the same memory
    again and again, as with the stream emptied in between."""
    M, N = 40, 264
    w = _packed(torch.randn(N, N, device=DEV) / 8, csa2.FP4_MX)
    x0 = torch.randn(M, N, device=DEV)
    ends = []
    for wait in (True, False):
        x, m = x0.clone(), csa2.Fp4Matrix(M, N, csa2.FP4_MX)
        seen = []
        for i in range(60):
            for call in (lambda: csa2.fp4_quant(m, x), lambda: csa2.fp4_product(m, w, x), lambda: csa2.fp4_quant(m, x),
                         lambda: csa2.fp4_read(m, x)):
                call()
                if wait:
                    torch.cuda.synchronize()
            if i % 20 == 19:
                seen.append(x.clone())
        ends.append(seen)
    assert all(torch.equal(a, b) for a, b in zip(*ends))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N", [(20, 300), (300, 264), (2600, 1496), (2600, 1501)])
def test_product_rows_in_the_middle_of_a_sector(M, N, dtype):
    """Output rows that begin 16 bytes behind a multiple of 32, all or every second one: the same bits, nothing beside them."""
    x, w = (_packed(torch.randn(r, 392, device=DEV), csa2.FP4_NV) for r in (M, N))
    wide = -(-N // 32) * 32
    want = torch.empty(M, wide, dtype=dtype, device=DEV)[:, :N]
    csa2.fp4_product(x, w, want)
    for off, stride in ((0, wide + 8), (16 // want.element_size(), wide + 32), (16 // want.element_size(), wide + 40)):
        out = torch.full((M, stride), 5.0, dtype=dtype, device=DEV)
        csa2.fp4_product(x, w, out[:, off:off + N])
        assert torch.equal(out[:, off:off + N], want)
        assert (out[:, :off] == 5).all() and (out[:, off + N:] == 5).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(3, 100), (37, 1000), (2500, 1288)])
def test_read_rows_in_the_middle_of_a_sector(rows, cols, dtype):
    """Output rows that begin 16 bytes behind a multiple of 32, all or every second one."""
    m = _packed(_rows(rows, cols + cols % 8, torch.float32, 9)[:, :cols], csa2.FP4_MX)
    wide = -(-cols // 32) * 32
    want = fu.values(m)
    for off, stride in ((0, wide), (0, wide + 8), (16 // dtype.itemsize, wide + 32), (16 // dtype.itemsize, wide + 40)):
        out = torch.full((rows, stride), 5.0, dtype=dtype, device=DEV)
        csa2.fp4_read(m, out[:, off:off + cols])
        assert torch.equal(out[:, off:off + cols].double(), want)
        assert (out[:, :off] == 5).all() and (out[:, off + cols:] == 5).all()


def test_quant_from_two_host_threads():
    """Narrow and wide matrices of one kernel, first used by two host threads at once, then the wide ones again."""
    import threading
    for dtype, narrow, wide in ((torch.bfloat16, 1100, 13990), (torch.float32, 600, 6400), (torch.float32, 14100, 28000)):
        for fmt in FMTS:
            xs = [torch.randn(1300, -(-c // 8) * 8, device=DEV).to(dtype)[:, :c] for c in (narrow, wide)]
            ms = [csa2.Fp4Matrix(*x.shape, fmt) for x in xs]
            torch.cuda.synchronize()
            gate, failed = threading.Barrier(2), []

            def run(x, m):
                try:
                    s = torch.cuda.Stream()
                    gate.wait()
                    csa2.fp4_quant(m, x, stream=s)
                    s.synchronize()
                except Exception as e:
                    failed.append(e)
            threads = [threading.Thread(target=run, args=a) for a in zip(xs, ms)]
            [t.start() for t in threads]
            [t.join() for t in threads]
            assert not failed
            csa2.fp4_quant(ms[1], xs[1])
            for x, m in zip(xs, ms):
                assert torch.equal(fu.values(m), fu.quantised(x, fmt))


def _codes(m):
    """The E2M1 codes of an Fp4Matrix, [rows, cols], from its records."""
    rt, ct = -(-m.rows // 128), -(-m.cols // 128)
    rec = m.tiles.view(rt, ct, -1)[..., :8192]
    b = rec.reshape(rt, ct, 4, 128, 16).permute(0, 3, 1, 2, 4).reshape(rt * 128, ct * 64)
    return torch.stack([b & 15, b >> 4], -1).flatten(1)[:m.rows, :m.cols]


@pytest.mark.parametrize("rows,cols", [(5, 264), (1300, 520), (1300, 4104), (4900, 520), (1230, 20008)])
@pytest.mark.parametrize("fmt", FMTS)
def test_codes_keep_the_sign(fmt, rows, cols):
    """The sign bit of a code is the value's, also where it rounds to zero and of -0; bf16 rows and the same rows
    in fp32 give the same bytes.  (A group of zeros is zeros: its scale, or its values, leave nothing to sign.)"""
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-24, 1, x.shape, generator=g, device=DEV).float())  # down to 2^-13 of a code and below
    x[:, ::16] = 6.0
    x[:, 3::16] = -0.0
    x[:, 5::16] = 0.0
    x = x.to(torch.bfloat16)
    m, n = _packed(x, fmt), _packed(x.float(), fmt)
    sign = torch.signbit(x)
    for k in (m, n):
        assert torch.equal((_codes(k) & 8) != 0, sign)
        assert torch.equal(fu.values(k), fu.quantised(x, fmt))
    assert torch.equal(_codes(m), _codes(n)) and ((_codes(m) & 7) == 0).any()
    out = torch.empty(rows, cols, device=DEV)
    csa2.fp4_read(m, out)
    assert torch.equal(torch.signbit(out), sign)
