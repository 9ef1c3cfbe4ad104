"""Plain 64-bit forms of the ragged cache calls, from the planes' bytes and the
definitions alone (torch; used by the GPU tests of the ragged calls)."""
import math

import torch

from fp4_compressed_sparse_gb300 import csa2

HALVES = [0, 1, 2, 3, 4, 6, 8, 12]
WIN = 128


def _e4m3(dev):
    return torch.arange(256, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()


def _nibbles(b):
    t = torch.tensor([v / 2 for v in HALVES] + [-v / 2 for v in HALVES], dtype=torch.float64, device=b.device)
    b = b.int()
    return torch.stack([t[b & 15], t[b >> 4]], -1).flatten(-2)


def _e8m0(s):
    return torch.ldexp(torch.ones((), dtype=torch.float64, device=s.device), s.int() - 127)


def phys(c, b, ent):
    """Physical entry rows of entries `ent` (int64) of sequence b."""
    if not c.page_entries:
        return b * c.capacity + ent
    return c.block_table[b].long()[ent // c.page_entries] * c.page_entries + ent % c.page_entries


def main_values(c, at):
    """[n, 576] fp64 values of physical entries `at`."""
    flat = lambda t: t.reshape(-1, t.shape[-1])
    if c.entry_format == csa2.ENTRY_FP8:
        lat = _e4m3(at.device)[flat(c.lat_codes)[at].int()]
        lat = lat * _e8m0(flat(c.lat_scales)[at]).repeat_interleave(32, -1)
        return torch.cat([lat, flat(c.rope_codes)[at].contiguous().view(torch.bfloat16).double()], -1)
    tab = _e4m3(at.device)
    lat = _nibbles(flat(c.lat_codes)[at]) * tab[flat(c.lat_scales)[at].int()].repeat_interleave(16, -1)
    rope = _nibbles(flat(c.rope_codes)[at]) * tab[flat(c.rope_scales)[at].int()].repeat_interleave(16, -1)
    return torch.cat([lat, rope], -1)


def key_values(c, b, ent):
    """[n, 128] fp64 values of the indexer keys of entries `ent` of sequence b."""
    if c.page_entries:
        at = phys(c, b, ent)
        tile, m = at // 128, at % 128
    else:
        tile, m = b * c.idx_tiles + ent // 128, ent % 128
    codes = c.idx_codes.reshape(-1, 4, 128, 16)[tile, :, m].flatten(1)
    scales = c.idx_scales.reshape(-1, 32, 4, 4)[tile, m % 32, m // 32]
    return _nibbles(codes) * _e8m0(scales).repeat_interleave(32, -1)


def window_values(codes, scales, swa):
    if swa == csa2.SWA_MXFP8:
        return _e4m3(codes.device)[codes.int()] * _e8m0(scales[..., :18]).repeat_interleave(32, -1)
    return codes.contiguous().view(torch.bfloat16).double()


def chunk_attn(c, q, cu, scale, win=None, sink=None):
    """out, lse in fp64, and per output element the sum of p |c| (what a relative
    error of the weights is multiplied by), per row the sum of |z| terms, and per
    output element what the small weights' absolute error is multiplied by (see
    attn_within): W sum |c| 2^-sigma, W = max p 2^sigma over the keys a row sees."""
    cu, outs, lses, mags, dots, smalls = cu.tolist(), [], [], [], [], []
    dev = q.device
    for b in range(c.batch):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        nt = int(c.n_tokens[b])
        P = nt - n
        T = (nt - 1) // c.ratio
        k = main_values(c, phys(c, b, torch.arange(T, device=dev)))
        if win is not None:
            r0 = cu[b] + WIN * b
            w = window_values(win.codes[r0:r0 + WIN + n], win.scales[r0:r0 + WIN + n], c.swa_dtype)
            tok = torch.arange(P - WIN, nt, device=dev)
        else:
            tok = torch.arange(nt - WIN, nt, device=dev)
            w = window_values(c.swa_codes[b][tok % WIN], c.swa_scales[b][tok % WIN], c.swa_dtype)
        k = torch.cat([k, w])
        pos = torch.arange(P, nt, device=dev)[:, None]
        see = torch.cat([torch.arange(T, device=dev)[None] < pos // c.ratio,
                         (tok[None] >= 0) & (tok[None] <= pos) & (tok[None] > pos - WIN)], -1)
        k = torch.where(see.any(0)[:, None], k, 0.0)
        top = k.abs().amax(-1)
        e = torch.frexp(top)[1].double() - 1  # 2^e <= top < 2^(e+1)
        sigma = torch.where((top == 0) | ((e >= 0) & (e <= 15)), 0.0, (e - 8).clamp(-24, 120))
        if c.entry_format == csa2.ENTRY_FP4:
            sigma[:T] = 0
        qd = q[cu[b]:cu[b + 1]].double()
        z = torch.einsum("qhd,td->qht", qd, k) * scale
        z = z.masked_fill(~see[:, None], -math.inf)
        m = z.amax(-1, keepdim=True)
        if sink is not None:
            m = torch.maximum(m, sink.double()[None, :, None])
        e = torch.exp(z - m)
        den = e.sum(-1, keepdim=True)
        if sink is not None:
            den = den + torch.exp(sink.double()[None, :, None] - m)
        p = e / den
        outs.append(torch.einsum("qht,td->qhd", p, k[:, :512]))
        mags.append(torch.einsum("qht,td->qhd", p, k[:, :512].abs()))
        lses.append((m + den.log())[..., 0])
        s2 = torch.exp2(sigma)
        W = (p * s2).amax(-1)
        smalls.append(W[..., None] * torch.einsum("qt,td->qd", see.double(), k[:, :512].abs() / s2[:, None])[:, None])
        dots.append(torch.einsum("qhd,td->qht", qd.abs(), k.abs()).masked_fill(~see[:, None], 0.0).amax(-1) * abs(scale))
    return torch.cat(outs), torch.cat(lses), torch.cat(mags), torch.cat(dots), torch.cat(smalls)


def attn_within(out, lse, ref, live=None):
    """Check a chunk attention against chunk_attn().

    The operands' values are exact.  A logit is a sum of 36 blocks of 16 exact
    products accumulated in fp32: off by at most 40 * 2^-23 of the sum of its
    terms' magnitudes (each fp32 addition by one unit at most), and so is lse,
    plus 2^-22 relative for the sum and the logarithm.  The weights (times a power
    of two 2^sigma of their key, whose values are divided by it) are rounded to
    fp16 on a scale on which the largest is 2^4 at least: 2^-11 relative, or below
    2^-14, where fp16's step is 2^-24, an absolute 2^-25.  That is 2^-25 / 2^4 =
    2^-29 of the largest weighted weight W per key, times |c| 2^-sigma, summed.
    They carry the logits' error; a bf16 output adds 2^-8 of its value."""
    o, l, mag, dot, small = ref
    if live is not None:
        out, lse = out[live], lse[live]
    ez = 40 * 2.0 ** -23 * dot + 2.0 ** -22 * (1 + l.abs())
    assert torch.isfinite(out.float()).all()
    assert ((lse.double() - l).abs() <= ez).all(), float(((lse.double() - l).abs() / ez).max())
    tol = (2.0 ** -11 + 2.0 ** -16 + 2 * ez[..., None]) * mag + 2.0 ** -29 * small + 2.0 ** -30
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs()
    err = (out.double() - o).abs()
    assert (err <= tol).all(), float((err / tol).max())
