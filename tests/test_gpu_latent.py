"""csa2_query_latent and csa2_value_project on the GPU against 64-bit products."""
import math

import pytest
import torch

from fp4_compressed_sparse_gb300 import csa2

pytestmark = pytest.mark.gpu
DEV = "cuda"
THETA = 10000.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp4_compressed_sparse_gb300 import build_lib
    build_lib.build()
    csa2.load()


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _weights(H, dim, g):
    """W_UK and W_UV as slices of one [H, 2 dim, 512]."""
    w = (torch.randn(H, 2 * dim, 512, generator=g, device=DEV) / math.sqrt(512)).to(torch.bfloat16)
    return w[:, :dim], w[:, dim:]


def _near(out, want, mag, steps, lost=0.0):
    """bf16 out against 64 bits: the sum of `steps` MMA steps, each off by at most one unit of fp32 (2^-23
    of the magnitudes added up), what the operands lost, and half a step of bf16."""
    tol = (steps * 2.0 ** -23 + lost) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    err = (out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).nan_to_num().max())


QUERY = [(1, 64, 128), (2, 1, 16), (127, 16, 64), (128, 128, 128), (129, 5, 48), (500, 64, 128), (33, 128, 112), (1500, 32, 32), (3001, 16, 128),
         (700, 20, 48), (400, 40, 80), (900, 17, 16), (1, 128, 128), (16, 8, 96), (4, 128, 64), (5, 128, 128), (16, 128, 32), (32, 64, 64), (33, 64, 64)]


@pytest.mark.parametrize("T,H,D", QUERY)
def test_query_latent(T, H, D):
    """Strided rows and heads; rows of negative positions left alone; RoPE dims bit for bit."""
    g = torch.Generator(device=DEV).manual_seed(T)
    w, _ = _weights(H, D, g)
    wide = torch.randn(T + 2, H * (D + 64) + 24, generator=g, device=DEV).to(torch.bfloat16)
    q = wide[:, :H * (D + 64)]
    rope, err = csa2.rope_table(THETA, 5000), _err()
    pos = torch.randint(0, 5000, (T + 2,), generator=g, device=DEV)
    pos[0], pos[T // 2] = 4999, -1
    pos[T:] = -7
    out = torch.full((T + 2, H, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    csa2.query_latent(q, w, pos, rope, out, err=err)
    assert int(err) == 0
    live = pos >= 0
    assert (out[~live] == 9).all()
    x = q.view(T + 2, H, D + 64)[live].double() if q.is_contiguous() else q.reshape(T + 2, H, D + 64)[live].double()
    wd = w.double()
    want, mag = torch.einsum("thk,hkc->thc", x[..., :D], wd), torch.einsum("thk,hkc->thc", x[..., :D].abs(), wd.abs())
    _near(out[live][..., :512], want, mag, D // 16 + 1)
    c, s = rope[pos[live]][:, None, :, 0].double(), rope[pos[live]][:, None, :, 1].double()
    a, b = x[..., D::2], x[..., D + 1::2]
    f = lambda v: v.float().double()
    rot = torch.stack([f(a * c - f(b * s)), f(b * c + f(a * s))], -1).flatten(-2)
    assert torch.equal(out[live][..., 512:], rot.float().to(torch.bfloat16))


def test_query_rope_errors():
    rope, err = csa2.rope_table(THETA, 100), _err()
    g = torch.Generator(device=DEV).manual_seed(0)
    w, _ = _weights(4, 32, g)
    q = torch.randn(3, 4 * 96, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.full((3, 4, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    csa2.query_latent(q, w, torch.tensor([99, 100, 2 ** 40], device=DEV), rope, out, err=err)
    assert int(err) == csa2.DEVERR_ROPE and (out[1:] == 9).all() and not (out[0] == 9).all()


def test_position_zero_and_far_rows():
    """Position 0 leaves the RoPE dims as they are; offsets beyond 2^31 elements of q and out."""
    T, H, D = 60000, 128, 128
    rope = csa2.rope_table(THETA, 4)
    g = torch.Generator(device=DEV).manual_seed(1)
    w, _ = _weights(H, D, g)
    q = torch.empty(T, H * (D + 64), dtype=torch.bfloat16, device=DEV)
    assert T * H * 576 > 2 ** 31
    at = torch.tensor([0, 1, T // 2 - 1, T - 130, T - 2, T - 1], device=DEV)
    q[at] = torch.randn(6, H * (D + 64), generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    pos[at] = 0
    out = torch.zeros(T, H, 576, dtype=torch.bfloat16, device=DEV)
    csa2.query_latent(q, w, pos, rope, out)
    x = q[at].view(6, H, D + 64)
    assert torch.equal(out[at][..., 512:], x[..., D:])
    wd, xd = w.double(), x[..., :D].double()
    _near(out[at][..., :512], torch.einsum("thk,hkc->thc", xd, wd), torch.einsum("thk,hkc->thc", xd.abs(), wd.abs()), 9)
    assert not out[2:T // 2 - 2].any()


VALUE = [(1, 64, 128), (2, 1, 16), (127, 16, 64), (128, 128, 128), (129, 5, 48), (300, 64, 128), (33, 128, 112), (1500, 32, 32), (3001, 16, 128),
         (700, 20, 48), (400, 40, 80), (900, 17, 16), (1, 128, 128), (16, 8, 96), (32, 64, 128), (17, 128, 128), (64, 64, 128), (256, 16, 64), (8192, 1, 16), (20011, 1, 16)]


@pytest.mark.parametrize("T,H,D", VALUE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_value_project(T, H, D, dtype):
    g = torch.Generator(device=DEV).manual_seed(T)
    _, w = _weights(H, D, g)
    o, err = torch.randn(T, H * 512 + 24, generator=g, device=DEV).to(dtype)[:, :H * 512].view(T, H, 512), _err()
    out = torch.full((T + 1, H * D + 8), 9.0, dtype=torch.bfloat16, device=DEV)
    csa2.value_project(o, w, out[:T, :H * D], err=err)
    assert int(err) == 0 and (out[T:] == 9).all() and (out[:, H * D:] == 9).all()
    od, wd = o.double(), w.double()
    want, mag = torch.einsum("thc,hjc->thj", od, wd), torch.einsum("thc,hjc->thj", od.abs(), wd.abs())
    f32 = dtype == torch.float32
    _near(out[:T, :H * D].reshape(T, H, D), want, mag, (64 if f32 else 32) + 1, 2.0 ** -16 if f32 else 0.0)


@pytest.mark.parametrize("T", [20, 1100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_value_nonfinite_rows(T, dtype):
    """An infinite or NaN latent reaches the values of its own token and head, and no other."""
    g = torch.Generator(device=DEV).manual_seed(3)
    _, w = _weights(4, 64, g)
    o = torch.randn(T, 4, 512, generator=g, device=DEV).to(dtype)
    clean, out = (torch.empty(T, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    csa2.value_project(o, w, clean)
    o[3, 1, 77], o[T - 10, 2, 500] = math.inf, math.nan
    csa2.value_project(o, w, out)
    want = o[3, 1, 77].float() * w[1, :, 77].float()
    assert torch.equal(out[3, 64:128].float(), want) and torch.isnan(out[T - 10, 128:192]).all()
    out[3, 64:128], out[T - 10, 128:192] = clean[3, 64:128], clean[T - 10, 128:192]
    assert torch.equal(out, clean)


def test_rows_in_other_batches():
    """A row of a smaller batch: the same bits where the form is the same, else within both roundings."""
    g = torch.Generator(device=DEV).manual_seed(4)
    k, v = _weights(16, 128, g)
    rope = csa2.rope_table(THETA, 5000)
    q = torch.randn(2000, 16 * 192, generator=g, device=DEV).to(torch.bfloat16)
    o = torch.randn(2000, 16, 512, generator=g, device=DEV)
    pos = torch.arange(2000, device=DEV)

    def run(lo, hi):
        a = torch.empty(hi - lo, 16, 576, dtype=torch.bfloat16, device=DEV)
        b = torch.empty(hi - lo, 16 * 128, dtype=torch.bfloat16, device=DEV)
        csa2.query_latent(q[lo:hi], k, pos[lo:hi].clone(), rope, a)
        csa2.value_project(o[lo:hi], v, b)
        return a, b
    full, few = run(0, 2000), run(0, 32)  # (up to 32 rows of 16 heads take the form for few)
    for (lo, hi), ref in (((0, 1), few), ((17, 18), few), ((1, 30), few), ((300, 2000), full), ((100, 500), full)):
        for x, y in zip(run(lo, hi), ref):
            assert torch.equal(x, y[lo:hi])
    for x, y in zip(few, full):
        y = y[:32].double()
        assert ((x.double() - y).abs() <= 2.0 ** -7 * y.abs() + 2.0 ** -12).all()


@pytest.mark.parametrize("T", [200, 1500])
def test_unaligned_to_32_bytes(T):
    """Outputs on 16-byte boundaries (and row strides that are odd multiples of 16 bytes)."""
    g = torch.Generator(device=DEV).manual_seed(5)
    k, v = _weights(3, 32, g)
    rope = csa2.rope_table(THETA, 1500)
    q, o = torch.randn(T, 3 * 96, generator=g, device=DEV).to(torch.bfloat16), torch.randn(T, 3, 512, generator=g, device=DEV)
    pos = torch.arange(T, device=DEV)
    a = torch.empty(T, 3, 576, dtype=torch.bfloat16, device=DEV)
    b = torch.empty(T * 3 * 576 + 8, dtype=torch.bfloat16, device=DEV)[8:].view(T, 3, 576)
    c = torch.empty(T, 96, dtype=torch.bfloat16, device=DEV)
    d = torch.empty(T, 104, dtype=torch.bfloat16, device=DEV)[:, 8:]
    assert b.data_ptr() % 32 == 16
    csa2.query_latent(q, k, pos, rope, a)
    csa2.query_latent(q, k, pos, rope, b)
    csa2.value_project(o, v, c)
    csa2.value_project(o, v, d)
    assert torch.equal(a, b) and torch.equal(c, d)


@pytest.mark.parametrize("T", [1, 400])
def test_streams_and_graphs(T):
    g = torch.Generator(device=DEV).manual_seed(6)
    k, v = _weights(64, 128, g)
    rope = csa2.rope_table(THETA, 1000)
    xs = [(torch.randn(T, 64 * 192, generator=g, device=DEV).to(torch.bfloat16), torch.randn(T, 64, 512, generator=g, device=DEV),
           torch.randint(0, 1000, (T,), generator=g, device=DEV)) for _ in range(2)]
    out = lambda: (torch.zeros(T, 64, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(T, 64 * 128, dtype=torch.bfloat16, device=DEV))
    want = []
    for q, o, p in xs:
        a, b = out()
        csa2.query_latent(q, k, p, rope, a)
        csa2.value_project(o, v, b)
        want.append((a, b))
    buf, res, res2 = [t.clone() for t in xs[0]], out(), out()
    torch.cuda.synchronize()
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        csa2.query_latent(buf[0], k, buf[2], rope, res[0])
        csa2.value_project(buf[1], v, res[1])
    for x, w in zip(xs, want):
        for t, s in zip(buf, x):
            t.copy_(s)
        graph.replay()
        csa2.query_latent(x[0], k, x[2], rope, res2[0], stream=other)
        csa2.value_project(x[1], v, res2[1], stream=other)
        torch.cuda.synchronize()
        for r in (res, res2):
            assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])


@pytest.mark.parametrize("T,stride", [(20, (1 << 27) + 8), (1100, (1 << 21) + 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_far_apart(T, stride, dtype):
    """Row offsets that pass 32 bits, in and out, against rows that lie together."""
    H, D = 3, 48
    g = torch.Generator(device=DEV).manual_seed(7)
    wk, wv = _weights(H, D, g)
    o = torch.randn(T, H, 512, generator=g, device=DEV).to(dtype)
    wide = torch.empty((T - 1) * stride + H * 512, dtype=dtype, device=DEV)
    far = wide.as_strided((T, H, 512), (stride, 512, 1))
    far.copy_(o)
    near = torch.empty(T, H * D, dtype=torch.bfloat16, device=DEV)
    csa2.value_project(o, wv, near)
    out = torch.empty(T, H * D, dtype=torch.bfloat16, device=DEV)
    csa2.value_project(far, wv, out)
    assert torch.equal(out, near)
    if dtype == torch.float32:
        return
    q = torch.randn(T, H * (D + 64), generator=g, device=DEV).to(dtype)
    far = wide.as_strided((T, H * D), (stride, 1))
    csa2.value_project(o, wv, far)
    assert torch.equal(far, near)
    far = wide.as_strided(q.shape, (stride, 1))
    far.copy_(q)
    rope, pos = csa2.rope_table(THETA, 2000), torch.arange(T, device=DEV)
    a, b = (torch.empty(T, H, 576, dtype=dtype, device=DEV) for _ in range(2))
    csa2.query_latent(q, wk, pos, rope, a)
    csa2.query_latent(far, wk, pos, rope, b)
    assert torch.equal(a, b)


def test_query_rows_behind_32_bits():
    """More than 2^31 elements of queries: the last rows as in a call of their own."""
    T, H, D = 30100, 128, 16
    g = torch.Generator(device=DEV).manual_seed(8)
    w, _ = _weights(H, D, g)
    q = torch.randn(T, H * (D + 64), generator=g, device=DEV).to(torch.bfloat16)
    rope, pos = csa2.rope_table(THETA, 40000), torch.arange(T, device=DEV)
    out, few = (torch.zeros(n, H, 576, dtype=torch.bfloat16, device=DEV) for n in (T, 300))
    csa2.query_latent(q, w, pos, rope, out)
    csa2.query_latent(q[-300:], w, pos[-300:].clone(), rope, few)
    assert torch.equal(out[-300:], few) and out[::1000].any(-1).all()


@pytest.mark.parametrize("T,H", [(1, 4), (20, 4), (130, 64), (1000, 16)])
def test_query_rows_left_alone(T, H):
    """Every row idle: nothing is written and nothing reported; a row behind the RoPE table among others:
    reported, left alone, the others as without it."""
    rope, err = csa2.rope_table(THETA, 2000), _err()
    g = torch.Generator(device=DEV).manual_seed(T)
    w, _ = _weights(H, 48, g)
    q = torch.randn(T, H * 112, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.full((T, H, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    csa2.query_latent(q, w, torch.full((T,), -5, device=DEV), rope, out, err=err)
    assert (out == 9).all() and int(err) == 0
    want = torch.empty_like(out)
    pos = torch.arange(T, device=DEV)
    csa2.query_latent(q, w, pos, rope, want, err=err)
    assert int(err) == 0
    pos[T // 2] = 2000
    csa2.query_latent(q, w, pos, rope, out, err=err)
    assert int(err) == csa2.DEVERR_ROPE and (out[T // 2] == 9).all()
    out[T // 2] = want[T // 2]
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [5, 20, 1100])
@pytest.mark.parametrize("scale", [0, 100, -100])
def test_value_keeps_all_bits_of_fp32(T, scale):
    """A value less its own first 16 bits, under a weight that is a power of two: what is left has 8 bits,
    every sum on the way fits fp32, and so does the result bf16: equal."""
    H, D = 4, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    p = (1.0 + torch.randint(0, 1 << 23, (T, H), generator=g, device=DEV) * 2.0 ** -23) * 2.0 ** scale
    p *= torch.randint(0, 2, (T, H), generator=g, device=DEV) * 2.0 - 1
    first = (p.view(torch.int32) & -256).view(torch.float32)
    o = torch.zeros(T, H, 512, device=DEV)
    at = torch.randint(0, 256, (2, T, H, 1), generator=g, device=DEV)
    o.scatter_(2, at[0], p[..., None])
    o.scatter_(2, 256 + at[1], -first[..., None])
    w = torch.exp2(torch.randint(-3, 4, (H, D, 1), generator=g, device=DEV).float()).expand(H, D, 512).to(torch.bfloat16).contiguous()
    out = torch.empty(T, H * D, dtype=torch.bfloat16, device=DEV)
    csa2.value_project(o, w, out)
    want = (p.double() - first.double())[..., None] * w[None, :, :, 0].double()
    assert (want != 0).any() and torch.equal(out.view(T, H, D).double(), want)


@pytest.mark.parametrize("T", [5, 20, 1100])
def test_value_of_the_largest_fp32(T):
    """Finite latents above bf16's largest number stay finite; a NaN whose payload bf16 cuts off stays a NaN."""
    H, D = 4, 64
    o = torch.zeros(T, H, 512, device=DEV)
    top = torch.finfo(torch.float32).max
    o[..., 33], o[1::2, :, 33] = top, -top
    o[2, 1, 33] = torch.nextafter(torch.tensor(top), torch.tensor(0.0)).item()
    w = torch.full((H, D, 512), 0.125, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(T, H * D, dtype=torch.bfloat16, device=DEV)
    csa2.value_project(o, w, out)
    assert torch.equal(out.view(T, H, D), (o[..., 33:34] * 0.125).to(torch.bfloat16).expand(T, H, D)) and torch.isfinite(out).all()
    nan = torch.tensor([0x7F800001, -8388607], dtype=torch.int32, device=DEV).view(torch.float32)
    o[3, 0, 500], o[T - 1, 2, 7] = nan[0], nan[1]
    csa2.value_project(o, w, out)
    is_nan = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    is_nan[3, 0] = is_nan[T - 1, 2] = True
    assert torch.equal(torch.isnan(out.view(T, H, D)), is_nan[..., None].expand(T, H, D))


@pytest.mark.parametrize("T", [32, 100, 1000])
def test_value_sums_of_fp32_are_fp32_sums(T):
    """The outputs that differ from the rounded 64-bit ones (sums close to a border of bf16, and off by more): not
    more than twice as many as of torch's product in fp32.  An output changes sides where its sum is off by more than
    its distance from the border, so their number is the sums' mean error, whatever its distribution."""
    H, D = 64, 128
    g = torch.Generator(device=DEV).manual_seed(T)
    _, w = _weights(H, D, g)
    o = torch.randn(T, H, 512, generator=g, device=DEV)
    out = torch.empty(T, H * D, dtype=torch.bfloat16, device=DEV)
    csa2.value_project(o, w, out)
    want = torch.einsum("thc,hjc->thj", o.double(), w.double()).reshape(T, -1).float().to(torch.bfloat16)
    assert not torch.backends.cuda.matmul.allow_tf32
    plain = torch.matmul(o.transpose(0, 1), w.float().transpose(1, 2)).transpose(0, 1).reshape(T, -1).to(torch.bfloat16)
    n = int((plain != want).sum())
    assert n >= 20 and int((out != want).sum()) <= 2 * n
