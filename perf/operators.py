"""What the ragged cache operators of libcsa2 are measured on: writing new tokens
into the quantised cache and reading them back, reading cached entries back, and
dense attention of a chunk of new tokens over the (paged) cache.

A case is a dict of plain values:
  op      "append" | "read" | "attn"
  batch   sequences
  ctx     entries (append, read: tokens) of the longest sequence before the call
  new     new tokens (append, attn) or rows read (read) of the longest sequence
  ragged  sequences of different lengths, some with no new token; else all alike
  page    entries per physical page (a shuffled pool), 0 = dense planes
  fmt     "fp4" (the 288 B + 36 B record) | "fp8" (E4M3 latent, bf16 RoPE dims)
  swa     "mxfp8" | "bf16": the sliding window's storage
  heads   query heads (attn)
  ratio   tokens per entry (attn: 1 or 2; append, read: 1)
  dtype   "bf16" | "f32": the new rows (append) and what is read back (read)
  pick    read: "range" (a contiguous stretch per sequence) | "list" (positions in
          any order, some of them empty)

Everything here is elementary torch; where `own` is true `run` calls libcsa2."""
import math

import numpy as np
import torch

own = False

LAT, ROPE, DQK, DI, WIN = 512, 64, 576, 128, 128
DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
THETA = 10000.0


# ------------------------------------------------------------------------------ cases
def _c(name, op, **kw):
    d = dict(name=name, op=op, batch=1, ctx=0, new=1, ragged=False, page=0, fmt="fp4", swa="mxfp8", heads=64, ratio=1,
             dtype="bf16", pick="range")
    d.update(kw)
    return d


def listed():
    return [
        # one decode step's tokens of 32 sequences, paged: written, then the records read back (latency)
        _c("append_decode_b32", "append", batch=32, ctx=65536, new=1, page=256),
        # a prefill batch: chunks of unequal lengths (some sequences idle), fp32 rows, odd offsets
        _c("append_chunks_ragged", "append", batch=7, ctx=4099, new=4096, ragged=True, page=128, swa="bf16", dtype="f32"),
        # a long prompt written in one call in the comparison format
        _c("append_prompt_fp8", "append", batch=2, ctx=1000, new=16384, fmt="fp8"),
        # the 512 selected entries of each of 32 sequences, dequantised for inspection or another kernel
        _c("read_selected_b32", "read", batch=32, ctx=65536, new=512, page=256, pick="list"),
        # whole prefixes read back as a GEMM operand (unabsorbed prefill, cache export)
        _c("read_prefix_ragged", "read", batch=6, ctx=65536, new=65536, ragged=True, page=1024),
        # the same from the comparison format, in fp32
        _c("read_prefix_fp8_f32", "read", batch=1, ctx=30011, new=30011, fmt="fp8", dtype="f32"),
        # one new token over a short dense context: the latency of the smallest call
        _c("attn_decode_b1_short", "attn", batch=1, ctx=1000, new=1, heads=64),
        # a decode batch whose sequences are short enough for every entry to be attended
        _c("attn_decode_b32_t8192", "attn", batch=32, ctx=8192, new=1, heads=64, page=256),
        # the long end of dense decode, ragged lengths, the bf16 window
        _c("attn_decode_b16_ragged", "attn", batch=16, ctx=65536, new=1, ragged=True, heads=64, page=1024, swa="bf16"),
        # four drafted tokens per sequence, few heads, two tokens per entry
        _c("attn_draft4_h16_r2", "attn", batch=8, ctx=16384, new=4, heads=16, ratio=2, page=128),
        # a mixed batch: chunks of unequal lengths over a paged cache
        _c("attn_chunks_ragged", "attn", batch=4, ctx=8192, new=500, ragged=True, heads=64, page=256),
        # a chunk of a prompt over its prefix in the comparison format
        _c("attn_chunk_1024_fp8", "attn", batch=1, ctx=15000, new=1024, heads=64, fmt="fp8"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn"])
    c = dict(op=op, ragged=rng.random() < 0.5, page=rng.choice([0, 128, 256, 1024]), fmt=rng.choice(["fp4", "fp4", "fp8"]),
             swa=rng.choice(["mxfp8", "bf16"]), heads=64, ratio=1, dtype=rng.choice(["bf16", "f32"]), pick="range")
    if op == "append":
        c["batch"] = _logint(rng, 1, 32)
        c["new"] = _logint(rng, 1, 32768 // c["batch"])
        c["ctx"] = _logint(rng, 1, 16384)
    elif op == "read":
        c["batch"] = _logint(rng, 1, 32)
        c["ctx"] = _logint(rng, 16, 200000 // c["batch"])
        c["pick"] = rng.choice(["range", "list"])
        c["new"] = _logint(rng, 1, c["ctx"])
    else:
        c["dtype"] = "bf16"
        c["heads"] = rng.choice([16, 32, 48, 64, 128])
        c["ratio"] = rng.choice([1, 1, 2])
        if rng.random() < 0.5:
            c["batch"], c["new"] = _logint(rng, 1, 32), rng.choice([1, 1, 2, 4, 7])
            c["ctx"] = _logint(rng, 1, min(65536, 400000 // c["batch"]))
        else:
            c["batch"], c["new"] = rng.randint(1, 3), _logint(rng, 16, 700)
            c["ctx"] = _logint(rng, 1, 800000 // (c["batch"] * c["new"]) * 64 // c["heads"] + 1)
            c["ctx"] = min(c["ctx"], 12000)
    return c


def lengths(case):
    """Per sequence: tokens before the call, new tokens (append, attn) or rows read (read)."""
    B, ctx, new = case["batch"], case["ctx"] * case["ratio"], case["new"]
    if not case["ragged"]:
        return [ctx] * B, [new] * B
    before = [max(0, ctx * (B - b) // B - 13 * b) for b in range(B)]
    if case["op"] == "read":
        return before, [min(before[b], max(0, new * (B - b) // B)) for b in range(B)]
    fresh = [max(1, new * (1 + (b * 5) % B) // B) for b in range(B)]
    if B > 2 and case["op"] == "append":
        fresh[1] = 0  # an idle sequence of the batch
    return before, fresh


def _capacity(case):
    before, fresh = lengths(case)
    need = max((p + (0 if case["op"] == "read" else n)) // case["ratio"] for p, n in zip(before, fresh))
    step = case["page"] or 128
    return max(1, -(-(need + 1) // step)) * step


# ------------------------------------------------------------------------------ plain formats
def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _e2m1_codes(y):
    a = y.abs()
    c = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (c + 8 * torch.signbit(y).int()).to(torch.uint8)


def _nvfp4(x):
    """Groups of 16 with an E4M3 scale: codes (one per byte) and scale bytes."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    s8 = (g.abs().amax(-1).double() / 6.0).float().clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    y = (g.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[..., None]).float()
    codes = torch.where((s > 0)[..., None], _e2m1_codes(y), torch.zeros_like(y, dtype=torch.uint8))
    return codes.reshape(x.shape), s8.view(torch.uint8)


def _mx_exponent(g, top):
    amax = g.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 1 - top).clamp(-127, 127).int()
    return torch.where(amax > 0, e, torch.full_like(e, -127)), amax > 0


def _mxfp4(x):
    g = x.reshape(*x.shape[:-1], -1, 32)
    e, some = _mx_exponent(g, 2)
    codes = torch.where(some[..., None], _e2m1_codes(g * _pow2(-e)[..., None]), torch.zeros_like(g, dtype=torch.uint8))
    return codes.reshape(x.shape), (e + 127).to(torch.uint8)


def _mxfp8(x):
    g = x.reshape(*x.shape[:-1], -1, 32)
    e, some = _mx_exponent(g, 8)
    y = torch.where(some[..., None], g * _pow2(-e)[..., None], torch.zeros_like(g)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape), (e + 127).to(torch.uint8)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(b):
    return torch.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def _e2m1_values(codes):
    t = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
    return t[codes.int()]


def _val_nvfp4(codes, scales):
    v = _e2m1_values(codes)
    return (v.reshape(*v.shape[:-1], -1, 16) * scales.view(torch.float8_e4m3fn).float()[..., None]).reshape(v.shape)


def _val_mxfp4(codes, scales):
    v = _e2m1_values(codes)
    return (v.reshape(*v.shape[:-1], -1, 32) * _pow2(scales.int() - 127)[..., None]).reshape(v.shape)


def _val_mxfp8(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.reshape(*v.shape[:-1], -1, 32) * _pow2(scales.int() - 127)[..., None]).reshape(v.shape)


def _encode_entry(x, fmt):
    """Rotated fp32 rows [n, 576] -> the four record planes of the format."""
    if fmt == "fp4":
        c, s = _nvfp4(x)
        return [_pack(c[:, :LAT]), s[:, :32], _pack(c[:, LAT:]), s[:, 32:]]
    c, s = _mxfp8(x[:, :LAT])
    return [c, s, x[:, LAT:].to(torch.bfloat16).view(torch.uint8), None]


def _decode_entry(lc, ls, rc, rs, fmt):
    if fmt == "fp4":
        return torch.cat([_val_nvfp4(_unpack(lc), ls), _val_nvfp4(_unpack(rc), rs)], -1)
    return torch.cat([_val_mxfp8(lc, ls), rc.contiguous().view(torch.bfloat16).float()], -1)


def _encode_window(x, swa):
    if swa == "mxfp8":
        c, s = _mxfp8(x)
        return c, torch.nn.functional.pad(s, (0, 14))
    return x.to(torch.bfloat16).view(torch.uint8), torch.zeros(x.shape[0], 32, dtype=torch.uint8, device=x.device)


def _decode_window(c, s, swa):
    return _val_mxfp8(c, s[..., :18]) if swa == "mxfp8" else c.contiguous().view(torch.bfloat16).float()


def _rotate(x, cs):
    """RoPE on the last 64 dims, pairs interleaved: x' = fma(x, c, -(y s)), y' = fma(y, c, x s)."""
    a, b = x[:, LAT::2], x[:, LAT + 1::2]
    c, s = cs[:, 0::2], cs[:, 1::2]
    ra = (a.double() * c.double() - (b * s).double()).float()
    rb = (b.double() * c.double() + (a * s).double()).float()
    return torch.cat([x[:, :LAT], torch.stack([ra, rb], -1).reshape(x.shape[0], ROPE)], -1)


def _rope_rows(pos):
    """The table's rows at these positions: cos, sin interleaved, evaluated in double."""
    inv = THETA ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=pos.device) / ROPE)
    ang = pos.double()[:, None] * inv
    return torch.stack([ang.cos(), ang.sin()], -1).reshape(pos.shape[0], ROPE).float()


# ------------------------------------------------------------------------------ state
def _rows(n, width, g, dtype=torch.float32):
    """N(0,1) rows, one in sixteen eight times larger, some groups all zero."""
    x = torch.randn(n, width, generator=g, device=DEV)
    x[5::16] *= 8.0
    if n > 3:
        x[3, :16] = 0.0
    return x.to(dtype)


def _empty_cache(case, g):
    B, cap, page, fmt = case["batch"], _capacity(case), case["page"], case["fmt"]
    n_pages = 0
    if page:
        per = cap // page
        n_pages = B * per + 3
        table = torch.randperm(n_pages, generator=g, device=DEV)[:B * per].to(torch.int32).view(B, per)
        rows = n_pages * page
    else:
        table, rows = None, B * cap
    widths = [256, 32, 32, 4] if fmt == "fp4" else [512, 16, 128, 0]
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    st = {"table": table, "cap": cap, "n_pages": n_pages,
          "planes": [u8(rows, w) if w else None for w in widths] + [u8(rows // 128, 8192), u8(rows // 128, 512)],
          "swa_codes": u8(B, WIN, 576 if case["swa"] == "mxfp8" else 1152), "swa_scales": u8(B, WIN, 32)}
    return st


def _phys(st, case, seq, ent):
    """Physical entry row of entry `ent` of sequence `seq` (tensors alike)."""
    if not case["page"]:
        return seq * st["cap"] + ent
    return st["table"].long()[seq, ent // case["page"]] * case["page"] + ent % case["page"]


def _ragged(counts):
    """(sequence, index within it) of every row of ragged sequences packed one after the other."""
    n = torch.tensor(counts, device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(counts), device=DEV), n)
    return seq, torch.arange(int(n.sum()), device=DEV) - (torch.cumsum(n, 0) - n)[seq]


def _cu(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)


def _fill(st, case, counts, g, keys):
    """Records of `counts[b]` entries per sequence, from N(0,1) rows."""
    for b, n in enumerate(counts):
        for e0 in range(0, n, 131072):
            m = min(131072, n - e0)
            ent = torch.arange(e0, e0 + m, device=DEV)
            row = _phys(st, case, torch.full_like(ent, b), ent)
            for p, v in zip(st["planes"], _encode_entry(_rows(m, DQK, g), case["fmt"])):
                if p is not None:
                    p[row] = v
            if keys:
                c, s = _mxfp4(_rows(m, DI, g))
                st["planes"][4].view(-1, 4, 128, 16)[row // 128, :, row % 128] = _pack(c).view(m, 4, 16)
                st["planes"][5].view(-1, 32, 4, 4)[row // 128, row % 32, row % 128 // 32] = s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    before, fresh = lengths(case)
    st = _empty_cache(case, g)
    st["case"], B = case, case["batch"]
    total = sum(fresh)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    st["max_new"] = max(fresh)
    st["cu"], st["err"] = _cu(fresh), torch.zeros(1, dtype=torch.int32, device=DEV)
    if case["op"] == "append":
        # the sequences' windows (their older entries are not touched), the new rows, the RoPE table
        c, s = _encode_window(_rows(B * WIN, DQK, g), case["swa"])
        st["swa_codes"].copy_(c.view(B, WIN, -1))
        st["swa_scales"].copy_(s.view(B, WIN, 32))
        st["n0"] = torch.tensor(before, dtype=torch.int64, device=DEV)
        st["n_tokens"] = st["n0"].clone()
        st["kv"], st["key"] = _rows(total, DQK, g, dt), _rows(total, DI, g, dt)
        st["rope"] = _rope_rows(torch.arange(max(p + n for p, n in zip(before, fresh)), device=DEV))
        st["main"] = torch.empty(total, DQK, dtype=torch.bfloat16, device=DEV)
        st["keys"] = torch.empty(total, DI, dtype=torch.bfloat16, device=DEV)
        st["window"] = torch.empty(B, WIN, DQK, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "read":
        _fill(st, case, before, g, True)
        st["n_tokens"] = torch.tensor(before, dtype=torch.int64, device=DEV)
        seq, i = _ragged(fresh)
        span = st["n_tokens"] - torch.tensor(fresh, device=DEV)
        if case["pick"] == "list":
            pos = torch.minimum((torch.rand(total, generator=g, device=DEV) * st["n_tokens"][seq]).long(), st["n_tokens"][seq] - 1)
            st["pos"] = torch.where(torch.rand(total, generator=g, device=DEV) < 0.03, -1, pos).to(torch.int32)
            st["start"] = None
        else:
            st["pos"], st["start"] = None, (torch.rand(B, generator=g, device=DEV) * (span + 1)).long()
        st["main"] = torch.empty(total, DQK, dtype=dt, device=DEV)
        st["keys"] = torch.empty(total, DI, dtype=dt, device=DEV)
    else:
        H, r = case["heads"], case["ratio"]
        n = [p + k for p, k in zip(before, fresh)]
        _fill(st, case, [t // r for t in n], g, False)
        st["n_tokens"] = torch.tensor(n, dtype=torch.int64, device=DEV)
        # the chunk's window rows: per sequence the 128 tokens before the chunk, then its own
        c, s = _encode_window(_rows(total + WIN * B, DQK, g), case["swa"])
        st["win_codes"], st["win_scales"] = c, s
        seq, i = _ragged([WIN] * B)
        tok = st["n_tokens"][seq] - WIN + i  # the ring: the last 128 tokens, token t in slot t % 128
        row = st["cu"].long()[seq + 1] + WIN * seq + i
        ok = tok >= 0
        st["swa_codes"][seq[ok], tok[ok] % WIN] = c[row[ok]]
        st["swa_scales"][seq[ok], tok[ok] % WIN] = s[row[ok]]
        q = torch.randn(total, H, DQK, generator=g, device=DEV)
        st["q"] = (q * (0.5 + 2.5 * torch.rand(H, 1, generator=g, device=DEV))).to(torch.bfloat16)
        st["sink"] = torch.randn(H, generator=g, device=DEV)
        st["scale"] = 1.0 / math.sqrt(DQK)
        st["out"] = torch.empty(total, H, LAT, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.empty(total, H, device=DEV)
        st["max_ent"] = max(t // r for t in n)  # the longest sequence, for the padded plain form
    return st


# ------------------------------------------------------------------------------ run
def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    return _plain_append(st) if op == "append" else _plain_read(st) if op == "read" else _plain_attn(st)


def _handle(st):
    """The program's cache handle over its planes, and its workspace: made once, kept with them."""
    from fp4_compressed_sparse_gb300 import csa2
    if "cache" not in st:
        case = st["case"]
        names = ("lat_codes", "lat_scales", "rope_codes", "rope_scales", "idx_codes", "idx_scales")
        planes = dict(zip(names, st["planes"]), swa_codes=st["swa_codes"], swa_scales=st["swa_scales"],
                      n_tokens=st["n_tokens"])
        if case["ratio"] == 2:
            planes["cmp_buf"] = torch.zeros(case["batch"], 4, 4, 704, device=DEV)
        st["cache"] = csa2.Cache.from_planes(
            case["batch"], st["cap"], planes, ratio=case["ratio"],
            swa_dtype=csa2.SWA_MXFP8 if case["swa"] == "mxfp8" else csa2.SWA_BF16,
            page_entries=case["page"] or None, n_pages=st["n_pages"] or None, block_table=st["table"],
            entry_format=csa2.ENTRY_FP4 if case["fmt"] == "fp4" else csa2.ENTRY_FP8)
        if case["op"] == "attn":
            st["ws"] = csa2.chunk_attn_workspace(st["q"].shape[0], case["heads"], case["batch"])
            st["win"] = csa2.ChunkWindow(st["win_codes"], st["win_scales"])
    return csa2, st["cache"]


def _run_own(st):
    csa2, c = _handle(st)
    op, err = st["case"]["op"], st["err"]
    if op == "append":
        c.n_tokens.copy_(st["n0"])  # back to the state before the call, so that the pass can be repeated
        csa2.kv_append_ragged(c, st["cu"], st["rope"], kv=st["kv"], idx_key=st["key"], max_new=st["max_new"], err=err)
        csa2.kv_read(c, st["cu"], start=st["n0"], out_main=st["main"], out_key=st["keys"], err=err)
        csa2.window_read(c, st["window"])
        return {"main": st["main"], "key": st["keys"], "window": st["window"], "n_tokens": c.n_tokens}
    if op == "read":
        csa2.kv_read(c, st["cu"], start=st["start"], pos=st["pos"], out_main=st["main"], out_key=st["keys"], err=err)
        return {"main": st["main"], "key": st["keys"]}
    one = st["case"]["new"] == 1  # single tokens: the cache's own window ring holds all they need
    csa2.chunk_attn(c, st["q"], st["cu"], st["out"], st["lse"], st["ws"], st["scale"], max_new=st["max_new"],
                    win=None if one else st["win"], sink=st["sink"], err=err)
    return {"out": st["out"], "lse": st["lse"]}


def _plain_append(st):
    case, n0 = st["case"], st["n0"]
    cu = st["cu"].long()
    n_new = cu[1:] - cu[:-1]
    row = torch.arange(st["kv"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    tok = n0[seq] + row - cu[seq]
    x = _rotate(st["kv"].float(), st["rope"][tok])
    rec = _encode_entry(x, case["fmt"])
    main = _decode_entry(*rec, case["fmt"]).to(torch.bfloat16)
    kc, ks = _mxfp4(st["key"].float())
    at = _phys(st, case, seq, tok)
    for p, v in zip(st["planes"], rec):
        if p is not None:
            p[at] = v
    st["planes"][4].view(-1, 4, 128, 16)[at // 128, :, at % 128] = _pack(kc).view(-1, 4, 16)
    st["planes"][5].view(-1, 32, 4, 4)[at // 128, at % 32, at % 128 // 32] = ks
    # the window: each sequence's last 128 tokens, older ones from its ring
    n = n0 + n_new
    last = tok >= n[seq] - WIN
    wc, ws = _encode_window(x[last], case["swa"])
    st["swa_codes"][seq[last], tok[last] % WIN] = wc
    st["swa_scales"][seq[last], tok[last] % WIN] = ws
    t = n[:, None] - WIN + torch.arange(WIN, device=DEV)
    b = torch.arange(case["batch"], device=DEV)[:, None]
    w = _decode_window(st["swa_codes"][b, t % WIN], st["swa_scales"][b, t % WIN], case["swa"])
    w = torch.where((t >= 0)[..., None], w, torch.zeros_like(w))
    st["n_tokens"].copy_(n)
    return {"main": main, "key": _val_mxfp4(kc, ks).to(torch.bfloat16), "window": w.to(torch.bfloat16), "n_tokens": st["n_tokens"]}


def _gather(st, at):
    rec = [p[at] if p is not None else None for p in st["planes"][:4]]
    return _decode_entry(*rec, st["case"]["fmt"])


def _plain_read(st):
    cu = st["cu"].long()
    row = torch.arange(st["main"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    ent = st["pos"].long() if st["pos"] is not None else st["start"][seq] + row - cu[seq]
    some = (ent >= 0)[:, None]
    at = _phys(st, st["case"], seq, ent.clamp(min=0))
    main = torch.where(some, _gather(st, at), 0.0)
    kc = st["planes"][4].view(-1, 4, 128, 16)[at // 128, :, at % 128].reshape(-1, 64)
    ks = st["planes"][5].view(-1, 32, 4, 4)[at // 128, at % 32, at % 128 // 32]
    key = torch.where(some, _val_mxfp4(_unpack(kc), ks), 0.0)
    return {"main": main.to(st["main"].dtype), "key": key.to(st["keys"].dtype)}


def _plain_attn(st):
    """Every sequence padded to the longest: logits over the visible entries and the window, one softmax."""
    case, cu, n = st["case"], st["cu"].long(), st["n_tokens"]
    B, H, N, T = case["batch"], case["heads"], st["max_new"], st["max_ent"]
    b = torch.arange(B, device=DEV)[:, None]
    i = torch.arange(N, device=DEV)
    n_new = cu[1:] - cu[:-1]
    qpos = (n - n_new)[:, None] + i  # [B, N]
    row = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][row].float().reshape(B, N * H, DQK)
    ent = torch.arange(T, device=DEV)
    held = (ent[None] < (n // case["ratio"])[:, None])
    k = _gather(st, _phys(st, case, b.expand(B, T), torch.where(held, ent[None], 0)))
    wi = torch.arange(WIN + N, device=DEV)
    wrow = (cu[:-1, None] + WIN * b + wi).clamp(max=st["win_codes"].shape[0] - 1)
    k = torch.cat([k, _decode_window(st["win_codes"][wrow], st["win_scales"][wrow], case["swa"])], 1)
    s = torch.matmul(q, k.transpose(1, 2)).view(B, N, H, T + WIN + N) * st["scale"]
    wtok = (n - n_new)[:, None] - WIN + wi  # [B, WIN + N]
    see = torch.cat([ent[None, None] < (qpos // case["ratio"])[..., None],
                     (wtok[:, None] >= 0) & (wtok[:, None] <= qpos[..., None]) & (wtok[:, None] > (qpos - WIN)[..., None])], -1)
    s.masked_fill_(~see[:, :, None], -math.inf)
    m = torch.maximum(s.amax(-1), st["sink"])
    p = s.sub_(m[..., None]).exp_()
    den = p.sum(-1) + (st["sink"] - m).exp()
    o = torch.matmul(p.view(B, N * H, -1), k[..., :LAT]).view(B, N, H, LAT) / den[..., None]
    live = i[None] < n_new[:, None]
    return {"out": o[live].to(torch.bfloat16), "lse": (m + den.log())[live]}


# ------------------------------------------------------------------------------ work
def work(case):
    before, fresh = lengths(case)
    rec = 392 if case["fmt"] == "fp4" else 724
    main = rec - 68
    wrow = 594 if case["swa"] == "mxfp8" else 1152
    total, B, size = sum(fresh), case["batch"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        # rows in, RoPE rows, records written and read back as bf16, the window written and read back
        wrote = sum(min(n, WIN) for n in fresh)
        return {"bytes": total * (704 * size + 256 + rec + 704 * 2) + wrote * wrow + B * WIN * (wrow + DQK * 2), "flops": total * 704 * 4}
    if case["op"] == "read":
        return {"bytes": total * (rec + 704 * size + (4 if case["pick"] == "list" else 0)), "flops": total * 704}
    H, r = case["heads"], case["ratio"]
    keys = by = 0
    for p, n in zip(before, fresh):
        keys += sum((p + i) // r + min(p + i + 1, WIN) for i in range(n))
        if n:
            by += (p + n - 1) // r * main + min(p + n, WIN - 1 + n) * wrow
    return {"bytes": by + total * H * (DQK * 2 + LAT * 2 + 4), "flops": keys * H * 2 * (DQK + LAT)}


# ------------------------------------------------------------------------------ 64 bits
def _x_e2m1(v):
    """Nearest grid value, ties to the even code, on float64 numpy values."""
    grid = np.array(E2M1)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, 7)
    lo = hi - 1
    mid = (grid[lo] + grid[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return np.copysign(np.where(up, grid[hi], grid[lo]), v)


def _x_e4m3(v):
    a = np.minimum(np.abs(v), 448.0)
    ex = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    ulp = 2.0 ** (ex - 3)
    return np.copysign(np.minimum(np.rint(a / ulp) * ulp, 448.0), v)


def _x_group(v, n, kind):
    """One row block through a format, as the values it stands for (float64)."""
    g = v.reshape(v.shape[0], -1, n)
    amax = np.abs(g).max(-1, keepdims=True)
    if kind == "nvfp4":
        s = _x_e4m3((amax / 6.0).astype(np.float32).astype(np.float64))
        q = (g / np.where(s > 0, s, 1.0)).astype(np.float32).astype(np.float64)
        return np.where(s > 0, _x_e2m1(q) * s, 0.0).reshape(v.shape)
    s = 2.0 ** (np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - (2 if kind == "mxfp4" else 8))
    return ((_x_e2m1 if kind == "mxfp4" else _x_e4m3)(g / s) * s).reshape(v.shape)


def _x_bf16(v):
    return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).double().numpy()


def _exact_append(case, st):
    before, fresh = lengths(case)
    kv, key = st["kv"].double().cpu().numpy(), st["key"].double().cpu().numpy()
    tok = np.concatenate([np.arange(p, p + n) for p, n in zip(before, fresh)])
    cs = st["rope"].cpu().numpy()[tok].astype(np.float64)
    f32 = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    x = kv.copy()  # the table's fp32 values; products and sums rounded to fp32 as the definition says
    a, b, c, s = kv[:, LAT::2], kv[:, LAT + 1::2], cs[:, 0::2], cs[:, 1::2]
    x[:, LAT::2], x[:, LAT + 1::2] = f32(a * c - f32(b * s)), f32(b * c + f32(a * s))
    if case["fmt"] == "fp4":
        main = _x_group(x, 16, "nvfp4")
    else:
        main = np.concatenate([_x_group(x[:, :LAT], 32, "mxfp8"), _x_bf16(x[:, LAT:])], -1)
    wv = _x_group(x, 32, "mxfp8") if case["swa"] == "mxfp8" else _x_bf16(x)
    old = st["swa_codes"].cpu()
    if case["swa"] == "mxfp8":
        tab = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        sc = 2.0 ** (st["swa_scales"].cpu().numpy()[..., :18].astype(np.float64) - 127)
        old = tab[old.numpy()] * np.repeat(sc, 32, -1)
    else:
        old = old.view(torch.bfloat16).double().numpy()
    window, at = np.zeros((case["batch"], WIN, DQK)), np.cumsum([0] + fresh)
    for q, (p, n) in enumerate(zip(before, fresh)):
        for i in range(WIN):
            t = p + n - WIN + i
            if t >= p:
                window[q, i] = wv[at[q] + t - p]
            elif t >= 0:
                window[q, i] = old[q, t % WIN]
    return {"main": main, "key": _x_group(key, 32, "mxfp4"), "window": window,
            "n_tokens": np.array([p + n for p, n in zip(before, fresh)], dtype=np.int64)}


def _x_records(st, case, b, ent):
    """Records of entries `ent` (an int64 tensor) of sequence b, as float64, from the bytes."""
    page, cap = case["page"], st["cap"]
    at = b * cap + ent if not page else st["table"][b].long()[torch.div(ent, page, rounding_mode="floor")] * page + torch.remainder(ent, page)
    tab = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    if case["fmt"] == "fp8":
        lat = tab[st["planes"][0][at].int()] * torch.exp2(st["planes"][1][at].double() - 127).repeat_interleave(32, -1)
        return torch.cat([lat, st["planes"][2][at].view(torch.bfloat16).double()], -1), at
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device=DEV) / 2
    codes = torch.cat([st["planes"][0][at], st["planes"][2][at]], -1).int()
    v = torch.empty(codes.shape[0], DQK, dtype=torch.float64, device=DEV)
    v[:, 0::2], v[:, 1::2] = half[codes % 16], half[codes // 16]
    return v * tab[torch.cat([st["planes"][1][at], st["planes"][3][at]], -1).int()].repeat_interleave(16, -1), at


def _exact_read(case, st):
    cu, main, key = st["cu"].tolist(), [], []
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device=DEV) / 2
    for b in range(case["batch"]):
        r = torch.arange(cu[b], cu[b + 1], device=DEV)
        ent = st["pos"][r].long() if st["pos"] is not None else st["start"][b] + r - cu[b]
        gone = ent < 0
        v, at = _x_records(st, case, b, torch.where(gone, 0, ent))
        tile, m = torch.div(at, 128, rounding_mode="floor"), torch.remainder(at, 128)
        codes = st["planes"][4][tile[:, None, None], (torch.arange(4, device=DEV) * 2048)[None, :, None] + (m * 16)[:, None, None] + torch.arange(16, device=DEV)].reshape(-1, 64).int()
        sc = st["planes"][5][tile[:, None], (16 * (m % 32) + 4 * torch.div(m, 32, rounding_mode="floor"))[:, None] + torch.arange(4, device=DEV)]
        k = torch.empty(codes.shape[0], DI, dtype=torch.float64, device=DEV)
        k[:, 0::2], k[:, 1::2] = half[codes % 16], half[codes // 16]
        k *= torch.exp2(sc.double() - 127).repeat_interleave(32, -1)
        v[gone], k[gone] = 0.0, 0.0
        main.append(v)
        key.append(k)
    return {"main": torch.cat(main), "key": torch.cat(key)}


def _exact_attn(case, st):
    before, fresh = lengths(case)
    H, r = case["heads"], case["ratio"]
    tab = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    outs, lses, at = [], [], 0
    for b, (p, n) in enumerate(zip(before, fresh)):
        k, _ = _x_records(st, case, b, torch.arange((p + n - 1) // r, device=DEV))
        rows = slice(at + WIN * b, at + WIN * b + WIN + n)
        if case["swa"] == "mxfp8":
            w = tab[st["win_codes"][rows].int()] * torch.exp2(st["win_scales"][rows, :18].double() - 127).repeat_interleave(32, -1)
        else:
            w = st["win_codes"][rows].view(torch.bfloat16).double()
        for i0 in range(0, n, 64):
            i1 = min(n, i0 + 64)
            q = st["q"][at + i0:at + i1].double()
            pos = torch.arange(p + i0, p + i1, device=DEV)[:, None]
            z = torch.cat([torch.einsum("qhd,td->qht", q, k), torch.einsum("qhd,td->qht", q, w)], -1) * st["scale"]
            t = torch.arange(p - WIN, p + n, device=DEV)[None]
            ok = torch.cat([torch.arange(k.shape[0], device=DEV)[None] < torch.div(pos, r, rounding_mode="floor"),
                            (t >= 0) & (t <= pos) & (pos - t < WIN)], -1)
            z = torch.cat([torch.where(ok[:, None], z, -math.inf), st["sink"].double()[None, :, None].expand(i1 - i0, H, 1)], -1)
            lse = torch.logsumexp(z, -1)
            pr = torch.exp(z - lse[..., None])
            outs.append(torch.einsum("qht,td->qhd", pr[..., :k.shape[0]], k[:, :LAT])
                        + torch.einsum("qht,td->qhd", pr[..., k.shape[0]:-1], w[:, :LAT]))
            lses.append(lse)
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    if case["op"] == "attn" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn}[case["op"]](case, st)
