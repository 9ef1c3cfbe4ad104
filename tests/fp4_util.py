"""64-bit forms of the 4-bit block-scaled matrices: quantisation by definition, and
values from the planes' bytes (torch; used by the GPU tests of those calls)."""
import torch

from fp4_compressed_sparse_gb300 import csa2

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e2m1(v):
    grid = torch.tensor(GRID, dtype=torch.float64, device=v.device)
    a = v.abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    mid = (grid[hi - 1] + grid[hi]) / 2
    return torch.copysign(torch.where((a > mid) | ((a == mid) & (hi % 2 == 0)), grid[hi], grid[hi - 1]), v)


def e4m3(v):
    ex = torch.floor(torch.log2(torch.where(v > 0, v, 1.0))).clamp(min=-6)
    return (torch.round(v / torch.exp2(ex - 3)) * torch.exp2(ex - 3)).clamp(max=448.0)


def quantised(x, fmt):
    """[rows, cols] fp64: what the matrix of x stands for; NaN rows as documented."""
    rows, cols = x.shape
    size = 16 if fmt == csa2.FP4_NV else 32
    x = torch.nn.functional.pad(x.double(), (0, -cols % size))
    top = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    x = torch.where(bad, 0.0, x)
    if fmt == csa2.FP4_NV:
        bad |= top > 2688.0 * 2.0 ** 62
        top = torch.where(bad, 0.0, top)
        f, e = torch.frexp(top)
        r = torch.where(top > 0, e - 12 + (f > 2688 / 4096).int(), 0).clamp(min=-62).double().exp2()
        g = (x / r).reshape(rows, -1, size)
        s = e4m3((g.abs().amax(-1, keepdim=True) / 6.0).float().double())
        v = torch.where(s > 0, e2m1((g / torch.where(s > 0, s, 1.0)).float().double()) * s, 0.0) * r[..., None]
    else:
        g = x.reshape(rows, -1, size)
        t = g.abs().amax(-1, keepdim=True)
        s = torch.exp2((torch.frexp(t)[1].double() - 3).clamp(-127, 127))
        v = torch.where(t > 0, e2m1(g / s) * s, 0.0)
    return torch.where(bad, float("nan"), v.reshape(rows, -1))[:, :cols]


def values(m):
    """[rows, cols] fp64 from the planes of an Fp4Matrix."""
    nv = m.fmt == csa2.FP4_NV
    rt, ct = -(-m.rows // 128), -(-m.cols // 128)
    dev = m.tiles.device
    t = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=dev)
    rec = m.tiles.view(rt, ct, 9216 if nv else 8704)
    b = rec[..., :8192].reshape(rt, ct, 4, 128, 16).permute(0, 3, 1, 2, 4).reshape(rt * 128, ct * 64).int()
    v = torch.stack([t[b & 15], t[b >> 4]], -1).flatten(1)
    n = 2 if nv else 1
    sc = rec[..., 8192:].reshape(rt, ct, n, 32, 4, 4).permute(0, 4, 3, 1, 2, 5).reshape(rt * 128, ct * n * 4)  # row 32 i + l
    if nv:
        s = torch.arange(256, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()[sc.int()]
    else:
        s = torch.exp2(sc.double() - 127)
    v = v * s.repeat_interleave(16 if nv else 32, -1) * m.row_scales.double()[:, None]
    return v[:m.rows, :m.cols]
