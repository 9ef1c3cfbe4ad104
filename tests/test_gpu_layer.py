"""A dense attention layer over a paged cache, all of it in the library's calls: pages
for the step, 4-bit projections of the hidden rows, append, queries into the latent
space, attention, values, 4-bit output projection.  Every call against a 64-bit form of
its own inputs; then the same as a captured graph."""
import math

import pytest
import torch

import fp4_util as fu
import ragged_util as ru
from fp4_compressed_sparse_gb300 import csa2

pytestmark = pytest.mark.gpu
DEV = "cuda"
HID, H, DIM, PAGE, PER, N_PAGES, B = 520, 16, 128, 128, 8, 20, 4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp4_compressed_sparse_gb300 import build_lib
    build_lib.build()
    csa2.load()


class Layer:
    def __init__(self, total, fmt, max_new, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.total, self.max_new = total, max_new
        self.c = csa2.Cache(B, PER * PAGE, page_entries=PAGE, n_pages=N_PAGES)
        self.pool, self.rope, self.err = csa2.PagePool(self.c), csa2.rope_table(1e4, PER * PAGE), torch.zeros(1, dtype=torch.int32, device=DEV)
        self.w = {}
        for name, n, k in (("q", H * (DIM + 64), HID), ("kv", 704, HID), ("o", HID, H * DIM)):
            self.w[name] = csa2.Fp4Matrix(n, k, fmt)
            csa2.fp4_quant(self.w[name], torch.randn(n, k, generator=g, device=DEV) * (2.0 / math.sqrt(k)), err=self.err)
        up = (torch.randn(H, 2 * DIM, 512, generator=g, device=DEV) / math.sqrt(512)).to(torch.bfloat16)
        self.uk, self.uv = up[:, :DIM], up[:, DIM:]
        e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
        self.cu, self.slots, self.pos = e(B + 1, dt=torch.int32), e(total, dt=torch.int64), e(total, dt=torch.int64)
        self.granted = e(B, dt=torch.int32)
        self.x4, self.v4 = csa2.Fp4Matrix(total, HID, fmt), csa2.Fp4Matrix(total, H * DIM, fmt)
        self.q, self.kv, self.lat = e(total, H * (DIM + 64)), e(total, 704, dt=torch.float32), e(total, H, 576)
        self.att, self.lse, self.val, self.out = e(total, H, 512), e(total, H, dt=torch.float32), e(total, H * DIM), e(total, HID)
        self.ws = csa2.chunk_attn_workspace(total, H, B)
        self.win = csa2.chunk_window(self.c, total)
        self.scale = 1 / math.sqrt(DIM + 64)

    def step(self, x):
        c, cu, mx, err = self.c, self.cu, self.max_new, self.err
        csa2.pages_resize(c, self.pool, cu_new=cu, max_new=mx, granted=self.granted, err=err)
        csa2.slot_map(c, cu, self.slots, self.pos, max_new=mx, err=err)
        csa2.fp4_quant(self.x4, x, err=err)
        csa2.fp4_product(self.x4, self.w["q"], self.q, err=err)
        csa2.fp4_product(self.x4, self.w["kv"], self.kv, err=err)
        csa2.kv_append_ragged(c, cu, self.rope, kv=self.kv[:, :576], idx_key=self.kv[:, 576:], max_new=mx, win=self.win, err=err)
        csa2.query_latent(self.q, self.uk, self.pos, self.rope, self.lat, err=err)
        csa2.chunk_attn(c, self.lat, cu, self.att, self.lse, self.ws, self.scale, max_new=mx, win=self.win, err=err)
        csa2.value_project(self.att, self.uv, self.val, err=err)
        csa2.fp4_quant(self.v4, self.val, err=err)
        csa2.fp4_product(self.v4, self.w["o"], self.out, err=err)


def _product_within(out, x, w):
    xv, wv = fu.values(x), fu.values(w)
    want, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    tol = (-(-x.cols // 64) + 10) * 2.0 ** -23 * mag  # (a unit of fp32 per MMA step and join, then the output's rounding)
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert ((out.double() - want).abs() <= tol).all()


STEPS = [[200, 1, 90, 0], [0, 300, 7, 129], [4, 4, 4, 4], [1, 1, 1, 1], [250, 1, 1, 1]]


@pytest.mark.parametrize("fmt", [csa2.FP4_NV, csa2.FP4_MX])
def test_layer_steps(fmt):
    total = 436 + 4  # (four rows of no sequence behind the largest step's)
    y = Layer(total, fmt, 300)
    g = torch.Generator(device=DEV).manual_seed(9)
    for step, counts in enumerate(STEPS):
        if step == 4:  # sequence 0 ends and a new prompt takes its place (and its pages)
            y.c.n_tokens[0] = 0
        n, before = sum(counts), y.c.n_tokens.clone()
        y.cu.copy_(torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist()))
        x = torch.randn(total, HID, generator=g, device=DEV).to(torch.bfloat16)
        y.lat[n:] = 5.0
        y.step(x)
        assert int(y.err) == 0 and y.granted.tolist() == [1] * B
        # pages: as many as the lengths need, each held once
        held = [-(-(int(b) + k) // PAGE) for b, k in zip(before, counts)]
        assert y.pool.held.tolist() == held and int(y.pool.n_free) == N_PAGES - sum(held)
        used = [p for b in range(B) for p in y.c.block_table[b, :held[b]].tolist()]
        assert len(set(used)) == len(used) and sorted(used + y.pool.free[:N_PAGES - sum(held)].tolist()) == list(range(N_PAGES))
        # projections
        assert torch.equal(fu.values(y.x4), fu.quantised(x, fmt))
        _product_within(y.q, y.x4, y.w["q"])
        _product_within(y.kv, y.x4, y.w["kv"])
        # the append wrote where the slots say
        main = torch.empty(n, 576, device=DEV)
        csa2.kv_read(y.c, y.cu, out_main=main, start=before)
        assert torch.equal(main.double(), ru.main_values(y.c, y.slots[:n])) and (y.slots[n:] == -1).all() and (y.pos[n:] == -1).all()
        # queries
        q = y.q[:n].double().view(n, H, DIM + 64)
        wd = y.uk.double()
        want, mag = torch.einsum("thk,hkc->thc", q[..., :DIM], wd), torch.einsum("thk,hkc->thc", q[..., :DIM].abs(), wd.abs())
        tol = 9 * 2.0 ** -23 * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        assert ((y.lat[:n, :, :512].double() - want).abs() <= tol).all() and (y.lat[n:] == 5).all()
        # attention, values, output
        ru.attn_within(y.att[:n], y.lse[:n], ru.chunk_attn(y.c, y.lat[:n], y.cu, y.scale, y.win))
        o, wd = y.att[:n].double(), y.uv.double()
        want, mag = torch.einsum("thc,hjc->thj", o, wd).reshape(n, -1), torch.einsum("thc,hjc->thj", o.abs(), wd.abs()).reshape(n, -1)
        tol = 33 * 2.0 ** -23 * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        assert ((y.val[:n].double() - want).abs() <= tol).all()
        _product_within(y.out, y.v4, y.w["o"])


def test_layer_as_a_graph():
    """Captured once, replayed with other lengths and rows: the bits of the eager calls."""
    total = 12
    a, b = Layer(total, csa2.FP4_NV, 9), Layer(total, csa2.FP4_NV, 9)
    x = torch.zeros(total, HID, dtype=torch.bfloat16, device=DEV)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    b.step(x)  # (no new tokens: attributes that are set once)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        b.step(x)
    for counts in ([9, 0, 1, 2], [1, 1, 1, 1], [0, 8, 0, 4], [3, 3, 3, 3]):
        n = sum(counts)
        x.copy_(torch.randn(total, HID, device=DEV))
        for y in (a, b):
            y.cu.copy_(torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist()))
        a.step(x)
        graph.replay()
        torch.cuda.synchronize()
        assert int(a.err) == 0 and int(b.err) == 0
        for p, q in ((a.c.block_table, b.c.block_table), (a.c.n_tokens, b.c.n_tokens), (a.lat[:n], b.lat[:n]), (a.att[:n], b.att[:n]), (a.out[:n], b.out[:n])):
            assert torch.equal(p, q)


def test_calls_of_all_kinds_at_once():
    """Queries, values, quantisations and products of several sizes on five streams at once: the bits of the
    same calls one after the other."""
    g = torch.Generator(device=DEV).manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    H, D = 16, 64
    w = (rand(H, 2 * D, 512) / 20).to(torch.bfloat16)
    rope = csa2.rope_table(10000.0, 4000)
    jobs = []
    for T in (3, 300, 1500):
        q, pos, out = rand(T, H * (D + 64)).to(torch.bfloat16), torch.arange(T, device=DEV), torch.zeros(T, H, 576, dtype=torch.bfloat16, device=DEV)
        jobs.append((out, lambda s, q=q, pos=pos, out=out: csa2.query_latent(q, w[:, :D], pos, rope, out, stream=s)))
    for T, dtype in ((3, torch.float32), (700, torch.float32), (1500, torch.bfloat16)):
        o, out = rand(T, H, 512).to(dtype), torch.zeros(T, H * D, dtype=torch.bfloat16, device=DEV)
        jobs.append((out, lambda s, o=o, out=out: csa2.value_project(o, w[:, D:], out, stream=s)))
    for M, N, K, fmt in ((1, 2000, 1040, csa2.FP4_NV), (50, 1400, 520, csa2.FP4_MX), (400, 600, 2056, csa2.FP4_NV), (2500, 2600, 264, csa2.FP4_MX),
                         (1500, 304, 4104, csa2.FP4_NV)):
        x, b, m, out = rand(M, K), csa2.Fp4Matrix(N, K, fmt), csa2.Fp4Matrix(M, K, fmt), torch.zeros(M, N, device=DEV)
        csa2.fp4_quant(b, rand(N, K))

        def step(s, x=x, b=b, m=m, out=out):
            csa2.fp4_quant(m, x, stream=s)
            csa2.fp4_product(m, b, out, stream=s)
        jobs.append((out, step))
    want = []
    for out, job in jobs:
        job(None)
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    for _ in range(30):
        for i, (_, job) in enumerate(jobs):
            job(streams[i % 5])
    torch.cuda.synchronize()
    assert all(torch.equal(out, v) for (out, _), v in zip(jobs, want))
