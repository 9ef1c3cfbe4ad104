"""What the operators around the attention of libcsa2 are measured on: the pages of a
paged cache handed out on the GPU, the products that lead into the latent space and
out of it, and 4-bit block-scaled matrices (quantisation, reading back, product).

A case is a dict of plain values:
  op      "pages" | "query" | "value" | "quant" | "product"
pages:  the block table and free list for each sequence's length after a step, then
        the physical slot and the position of every new token
  batch   sequences
  ctx     tokens of the longest sequence before the step
  new     new tokens of the sequence that brings most
  churn   some sequences end (their pages come back), some bring prompts, others a token
  page    entries per physical page
  ratio   tokens per entry
query:  q_latent = q_nope W_UK per head beside the rotated 64 RoPE dims
value:  o = o_latent W_UV^T per head
  tokens  rows; heads; dim  the head's q_nope / value width
  idle    rows behind the last sequence (query: left as they were)
  dtype   value: type of the latent rows, "bf16" | "f32"
quant:  a matrix quantised and read back as the values it stands for
product: x quantised, then out = x W^T with W held in the same 4-bit format
  rows, cols (K), n (product: rows of W); fmt "nv" (E2M1, an E4M3 scale per 16, a power
  of two per row) | "mx" (E2M1, an E8M0 scale per 32); dtype of x; out: type of the result

Everything here is elementary torch; where `own` is true `run` calls libcsa2."""
import math

import numpy as np
import torch

own = False

LAT, ROPE, DQK = 512, 64, 576
DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
THETA = 10000.0


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest step: 32 sequences append a token each, now and then one needs a page
        dict(name="pages_decode_b32", op="pages", batch=32, ctx=65536, new=1, churn=False, page=256, ratio=1),
        # a scheduler's step: requests end, prompts come in, most sequences append a token
        dict(name="pages_churn_b512", op="pages", batch=512, ctx=32768, new=4096, churn=True, page=128, ratio=2),
        # one decoded token's heads into the latent space
        dict(name="query_b1", op="query", tokens=1, heads=64, dim=128, idle=0),
        # a decode batch in a buffer with room for more rows
        dict(name="query_decode_b32", op="query", tokens=32, heads=128, dim=128, idle=8),
        # a prefill batch of ragged chunks
        dict(name="query_chunks_4001", op="query", tokens=4001, heads=64, dim=128, idle=95),
        # a decode batch's latents (fp32 from the sparse attention) to values
        dict(name="value_decode_b32", op="value", tokens=32, heads=64, dim=128, dtype="f32"),
        # the same for a prefill batch, bf16 from the chunk attention
        dict(name="value_chunks_4001", op="value", tokens=4001, heads=64, dim=128, dtype="bf16"),
        # activations of a decode batch, written and read back
        dict(name="quant_x_b32", op="quant", rows=32, cols=4096, fmt="mx", dtype="bf16"),
        # a weight laid out when a model is loaded, read back for a check
        dict(name="quant_weight", op="quant", rows=12288, cols=4096, fmt="nv", dtype="bf16"),
        # one token's query projection: the weight's bytes
        dict(name="product_b1", op="product", rows=1, cols=4096, n=12288, fmt="nv", dtype="bf16", out="bf16"),
        # a ragged batch's latent row and indexer key in one projection, fp32 results for the append
        dict(name="product_501_kv", op="product", rows=501, cols=4104, n=704, fmt="mx", dtype="f32", out="f32"),
        # a prefill batch's query projection
        dict(name="product_prefill", op="product", rows=8192, cols=4096, n=12288, fmt="nv", dtype="bf16", out="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "query", "value", "quant", "product", "product"])
    c = dict(op=op)
    if op == "pages":
        c["batch"] = _logint(rng, 1, 1024)
        c["page"], c["ratio"], c["churn"] = rng.choice([128, 256, 1024]), rng.choice([1, 2]), rng.random() < 0.5
        c["ctx"] = _logint(rng, 1, min(262144, 16777216 // c["batch"]))
        c["new"] = _logint(rng, 1, 4096) if c["churn"] else rng.choice([1, 1, 4, 7])
    elif op in ("query", "value"):
        c["heads"], c["dim"] = rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
        c["tokens"] = _logint(rng, 1, 262144 // c["heads"])
        if op == "query":
            c["idle"] = rng.choice([0, 1, 13, 200])
        else:
            c["dtype"] = rng.choice(["bf16", "f32"])
    else:
        c["fmt"], c["dtype"] = rng.choice(["nv", "mx"]), rng.choice(["bf16", "f32"])
        c["rows"] = _logint(rng, 1, 8192)
        c["cols"] = 8 * _logint(rng, 2, 1024)
        if op == "product":
            c["n"], c["out"] = _logint(rng, 16, 12288), rng.choice(["bf16", "f32"])
            c["rows"] = max(1, min(c["rows"], 8192 * 4096 * 12288 // (c["cols"] * c["n"])))
        else:
            c["rows"] = min(c["rows"], 12288 * 4096 // c["cols"])
    return c


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def lengths(case):
    """Per sequence: tokens before the step, new tokens, and whether it ends with the step."""
    B, ctx, new = case["batch"], case["ctx"], case["new"]
    before = [max(0, ctx - (ctx * 7 * b // (8 * B)) - 3 * b) for b in range(B)]
    if not case["churn"]:
        return before, [new] * B, [False] * B
    ends = [b % 10 == 3 for b in range(B)]
    prompt = [b % 8 == 5 and not ends[b] for b in range(B)]
    before = [0 if prompt[b] else before[b] for b in range(B)]
    fresh = [0 if ends[b] else max(1, new * (B - b) // B) if prompt[b] else 1 for b in range(B)]
    return before, fresh, ends


# ------------------------------------------------------------------------------ plain formats
def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _e2m1_codes(y):
    a = y.abs()
    c = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (c + 8 * torch.signbit(y).int()).to(torch.uint8)


def _exponent(a):
    """floor(log2 a) of a > 0, 0 for 0."""
    return torch.where(a > 0, torch.frexp(a)[1] - 1, 0).int()


def _row_exponent(x):
    """The power of two that brings a row's largest magnitude to 448 x 6 at most."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1)
    return torch.where(a > 0, e - 12 + (m > 2688.0 / 4096).int(), 0).clamp(min=-62).int()


def _quant(x, fmt):
    """Rows (fp32) to codes (one per byte, whole groups), scale bytes and the rows' powers of two."""
    rows, cols = x.shape
    size = 16 if fmt == "nv" else 32
    pad = -cols % size
    x = torch.nn.functional.pad(x, (0, pad)) if pad else x
    if fmt == "nv":
        r = _pow2(_row_exponent(x))
        g = (x / r[:, None]).reshape(rows, -1, size)
        s8 = (g.abs().amax(-1).double() / 6.0).float().clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float()
        y = (g.double() / torch.where(s > 0, s, 1.0).double()[..., None]).float()
        codes = torch.where((s > 0)[..., None], _e2m1_codes(y), 0)
        return codes.reshape(rows, -1).to(torch.uint8), s8.view(torch.uint8), r
    g = x.reshape(rows, -1, size)
    amax = g.abs().amax(-1)
    e = torch.where(amax > 0, (_exponent(amax) - 2).clamp(-127, 127), -127)
    codes = torch.where((amax > 0)[..., None], _e2m1_codes(g * _pow2(-e)[..., None]), 0)
    return codes.reshape(rows, -1).to(torch.uint8), (e + 127).to(torch.uint8), None


def _values(codes, scales, r, fmt, cols):
    t = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
    size = 16 if fmt == "nv" else 32
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nv" else _pow2(scales.int() - 127)
    v = (t[codes.int()].reshape(codes.shape[0], -1, size) * s[..., None]).reshape(codes.shape)[:, :cols]
    return v if r is None else v * r[:, None]


# ------------------------------------------------------------------------------ state
def _matrix(rows, cols, g, scale=1.0):
    """N(0,1) rows, one in sixteen eight times larger, some groups all zero, a zero row."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x[5::16] *= 8.0
    x[3::7, :16] = 0.0
    if rows > 40:
        x[40] = 0.0
    return x * scale


def _rope_rows(n):
    inv = THETA ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=DEV) / ROPE)
    ang = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.stack([ang.cos(), ang.sin()], -1).float()  # [n, 32, 2]


def _prepare_pages(case, g):
    before, fresh, ends = lengths(case)
    B, page, ratio = case["batch"], case["page"], case["ratio"]
    after = [0 if e else p + n for p, n, e in zip(before, fresh, ends)]
    per = max(1, -(-max(max(a, p) for a, p in zip(after, before)) // (ratio * page)) + 1)
    held = [-(-(p // ratio) // page) for p in before]
    n_pages = sum(max(h, -(-(a // ratio) // page)) for h, a in zip(held, after)) + 5
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    # one blob, so that the state before the step is put back by a single copy
    sizes = [-(-n // 4) * 4 for n in (B * per, B, n_pages, 1)]
    blob = torch.zeros(sum(sizes), dtype=torch.int32, device=DEV)
    at = np.cumsum([0] + sizes).tolist()
    view = lambda i, n: blob[at[i]:at[i] + n]  # noqa: E731
    st = dict(case=case, blob=blob, per=per, n_pages=n_pages, table=view(0, B * per).view(B, per), held=view(1, B),
              free=view(2, n_pages), n_free=view(3, 1))
    h = torch.tensor(held, device=DEV)
    st["held"].copy_(h)
    col = torch.arange(per, device=DEV)
    has = col[None] < h[:, None]
    order = (torch.cumsum(has.flatten().long(), 0) - 1).view(B, per)
    st["table"].copy_(torch.where(has, perm[order.clamp(0, n_pages - 1)], -1))
    used = sum(held)
    st["free"][:n_pages - used] = perm[used:]
    st["n_free"].fill_(n_pages - used)
    st["before"] = blob.clone()
    st["n_tokens"] = torch.tensor([0 if e else p for p, e in zip(before, ends)], dtype=torch.int64, device=DEV)
    st["cu"] = torch.tensor([0] + list(np.cumsum(fresh)), dtype=torch.int32, device=DEV)
    total = sum(fresh)
    st["granted"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    st["slots"] = torch.zeros(total, dtype=torch.int64, device=DEV)
    st["pos"] = torch.zeros(total, dtype=torch.int64, device=DEV)
    st["max_new"] = max(fresh)
    return st


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "pages":
        st = _prepare_pages(case, g)
    elif op == "query":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        rows = T + case["idle"]
        st = dict(q=torch.randn(rows, H * (D + ROPE), generator=g, device=DEV).to(torch.bfloat16),
                  w=(torch.randn(H, 2 * D, LAT, generator=g, device=DEV) / math.sqrt(LAT)).to(torch.bfloat16)[:, :D],
                  pos=torch.randint(0, 65536, (rows,), generator=g, device=DEV), rope=_rope_rows(65536),
                  out=torch.zeros(rows, H, DQK, dtype=torch.bfloat16, device=DEV))
        st["pos"][T:] = -1
    elif op == "value":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        st = dict(o=torch.randn(T, H, LAT, generator=g, device=DEV).to(_dt(case["dtype"])),
                  w=(torch.randn(H, 2 * D, LAT, generator=g, device=DEV) / math.sqrt(LAT)).to(torch.bfloat16)[:, D:],
                  out=torch.empty(T, H * D, dtype=torch.bfloat16, device=DEV))
    else:
        rows, cols = case["rows"], case["cols"]
        st = dict(x=_matrix(rows, cols, g).to(_dt(case["dtype"])))
        if op == "quant":
            st["out"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
        else:
            st["weight"] = _matrix(case["n"], cols, g, 1 / math.sqrt(cols)).to(torch.bfloat16)
            st["packed"] = _quant(st["weight"].float(), case["fmt"])  # as the plain program keeps it
            wide = torch.empty(rows, -(-case["n"] // 8) * 8, dtype=_dt(case["out"]), device=DEV)
            st["out"] = wide[:, :case["n"]]
    st["case"], st["err"] = case, torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


# ------------------------------------------------------------------------------ run
def run(st):
    op = st["case"]["op"]
    if own:
        return _own[op](st)
    return {"pages": _plain_pages, "query": _plain_query, "value": _plain_value, "quant": _plain_quant,
            "product": _plain_product}[op](st)


def _own_pages(st):
    from fp4_compressed_sparse_gb300 import csa2
    case = st["case"]
    if "cache" not in st:  # the program's cache over its pool of pages, made once
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
        rows = st["n_pages"] * case["page"]
        planes = dict(lat_codes=u8(rows, 256), lat_scales=u8(rows, 32), rope_codes=u8(rows, 32), rope_scales=u8(rows, 4),
                      idx_codes=u8(rows // 128, 8192), idx_scales=u8(rows // 128, 512), swa_codes=u8(case["batch"], 128, 576),
                      swa_scales=u8(case["batch"], 128, 32), n_tokens=st["n_tokens"])
        if case["ratio"] == 2:
            planes["cmp_buf"] = torch.zeros(case["batch"], 4, 4, 704, device=DEV)
        st["cache"] = csa2.Cache.from_planes(case["batch"], st["per"] * case["page"], planes, ratio=case["ratio"],
                                             page_entries=case["page"], n_pages=st["n_pages"], block_table=st["table"])
        st["pool"] = csa2.PagePool(st["cache"], free=st["free"], n_free=st["n_free"], held=st["held"])
    st["blob"].copy_(st["before"])  # back to the state before the step, so that the pass can be repeated
    csa2.pages_resize(st["cache"], st["pool"], cu_new=st["cu"], max_new=st["max_new"], granted=st["granted"], err=st["err"])
    csa2.slot_map(st["cache"], st["cu"], st["slots"], st["pos"], max_new=st["max_new"], err=st["err"])
    return _pages_out(st)


def _own_query(st):
    from fp4_compressed_sparse_gb300 import csa2
    csa2.query_latent(st["q"], st["w"], st["pos"], st["rope"], st["out"], err=st["err"])
    return st["out"]


def _own_value(st):
    from fp4_compressed_sparse_gb300 import csa2
    csa2.value_project(st["o"], st["w"], st["out"], err=st["err"])
    return st["out"]


def _formats(csa2):
    return {"nv": csa2.FP4_NV, "mx": csa2.FP4_MX}


def _own_quant(st):
    from fp4_compressed_sparse_gb300 import csa2
    if "m" not in st:
        st["m"] = csa2.Fp4Matrix(*st["x"].shape, _formats(csa2)[st["case"]["fmt"]])
    csa2.fp4_quant(st["m"], st["x"], err=st["err"])
    csa2.fp4_read(st["m"], st["out"])
    return st["out"]


def _own_product(st):
    from fp4_compressed_sparse_gb300 import csa2
    if "w4" not in st:  # the weight laid out once, and a buffer for the activations
        f = _formats(csa2)[st["case"]["fmt"]]
        st["w4"], st["x4"] = csa2.Fp4Matrix(*st["weight"].shape, f), csa2.Fp4Matrix(*st["x"].shape, f)
        csa2.fp4_quant(st["w4"], st["weight"], err=st["err"])
    csa2.fp4_quant(st["x4"], st["x"], err=st["err"])
    csa2.fp4_product(st["x4"], st["w4"], st["out"], err=st["err"])
    return st["out"]


_own = {"pages": _own_pages, "query": _own_query, "value": _own_value, "quant": _own_quant, "product": _own_product}


def _pages_out(st):
    return {k: st[k] for k in ("table", "held", "free", "n_free", "granted", "slots", "pos")}


def _plain_pages(st):
    """Pages beyond a sequence's need go back (first sequence's first page on top), then sequences
    that need more take from the top, in order, as long as there are enough."""
    case = st["case"]
    B, per, page, ratio, n_pages = case["batch"], st["per"], case["page"], case["ratio"], st["n_pages"]
    st["blob"].copy_(st["before"])
    table, held, free = st["table"], st["held"].long(), torch.cat([st["free"], st["free"][:1]])
    cu, n0 = st["cu"].long(), st["n_free"].long()
    entries = (st["n_tokens"] + cu[1:] - cu[:-1]) // ratio
    need = (entries + page - 1) // page
    col = torch.arange(per, device=DEV)[None]
    back = (col >= need[:, None]) & (col < held[:, None])
    j = (torch.cumsum(back.flatten().long(), 0) - 1).view(B, per)
    n = n0 + back.sum()
    free.scatter_(0, torch.where(back, n - 1 - j, n_pages).flatten(), table.flatten())
    grow = (need - held).clamp(min=0)
    upto = torch.cumsum(grow, 0)
    granted = (grow == 0) | (upto <= n)
    take = (col >= held[:, None]) & (col < need[:, None]) & granted[:, None]
    k = (upto - grow)[:, None] + col - held[:, None]
    new = free[(n - 1 - k).clamp(0, n_pages - 1)]
    table.copy_(torch.where(take, new, torch.where(back, -1, table)))
    st["held"].copy_(torch.where(granted, need, held))
    st["free"].copy_(free[:n_pages])
    st["n_free"].copy_(n - torch.where(granted, grow, 0).sum())
    st["granted"].copy_(granted)
    r = torch.arange(st["slots"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], r, right=True)
    pos = st["n_tokens"][seq] + r - cu[seq]
    ent = pos // ratio
    # (the odd last token of a ratio-2 sequence has no entry yet)
    pg = torch.where(ent < entries[seq], table.long()[seq, (ent // page).clamp(max=per - 1)], -1)
    st["slots"].copy_(torch.where(pg >= 0, pg * page + ent % page, -1))
    st["pos"].copy_(pos)
    return _pages_out(st)


def _rotate(x, cs):
    """Pairs interleaved: x' = fma(x, c, -(y s)), y' = fma(y, c, x s)."""
    a, b, c, s = x[..., 0::2], x[..., 1::2], cs[..., 0], cs[..., 1]
    ra = (a.double() * c.double() - (b * s).double()).float()
    rb = (b.double() * c.double() + (a * s).double()).float()
    return torch.stack([ra, rb], -1).flatten(-2)


def _plain_query(st):
    H, D = st["case"]["heads"], st["case"]["dim"]
    q = st["q"].view(-1, H, D + ROPE).float()
    lat = torch.matmul(q[..., :D].transpose(0, 1), st["w"].float()).transpose(0, 1)
    rot = _rotate(q[..., D:], st["rope"][st["pos"].clamp(min=0)][:, None])
    full = torch.cat([lat, rot], -1).to(torch.bfloat16)
    st["out"].copy_(torch.where((st["pos"] >= 0)[:, None, None], full, st["out"]))
    return st["out"]


def _plain_value(st):
    o = torch.matmul(st["o"].float().transpose(0, 1), st["w"].float().transpose(1, 2)).transpose(0, 1)
    st["out"].copy_(o.reshape(o.shape[0], -1))
    return st["out"]


def _plain_quant(st):
    fmt, cols = st["case"]["fmt"], st["case"]["cols"]
    st["out"].copy_(_values(*_quant(st["x"].float(), fmt), fmt, cols))
    return st["out"]


def _plain_product(st):
    fmt, cols = st["case"]["fmt"], st["case"]["cols"]
    x = _values(*_quant(st["x"].float(), fmt), fmt, cols)
    w = _values(*st["packed"], fmt, cols)
    st["out"].copy_(torch.matmul(x, w.t()))
    return st["out"]


# ------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "pages":
        before, fresh, ends = lengths(case)
        B, total, ratio, page = case["batch"], sum(fresh), case["ratio"], case["page"]
        moved = 0
        for p, n, e in zip(before, fresh, ends):
            moved += abs(-(-((0 if e else p + n) // ratio) // page) - -(-(p // ratio) // page))
        # lengths, bounds and counts read, counts and grants written; pages moved between list and table; slots and positions
        return {"bytes": B * (8 + 4 + 4 + 4 + 4) + moved * 8 + total * 16, "flops": B * 8 + total * 8}
    if op in ("query", "value"):
        T, H, D = case["tokens"], case["heads"], case["dim"]
        w = H * D * LAT * 2
        if op == "query":
            return {"bytes": w + T * H * ((D + ROPE) * 2 + DQK * 2) + T * (8 + ROPE * 4), "flops": T * H * (2 * D * LAT + 3 * ROPE)}
        return {"bytes": w + T * H * (LAT * (2 if case["dtype"] == "bf16" else 4) + D * 2), "flops": T * H * 2 * D * LAT}
    rows, cols, size = case["rows"], case["cols"], 2 if case["dtype"] == "bf16" else 4
    group = 16 if case["fmt"] == "nv" else 32
    if op == "quant":
        return {"bytes": rows * cols * (size + 2) + rows * cols // 2 + rows * cols // group, "flops": rows * cols * 4}
    n, out = case["n"], 2 if case["out"] == "bf16" else 4
    return {"bytes": rows * cols * size + n * cols // 2 + n * cols // group + rows * n * out, "flops": 2 * rows * cols * n}


# ------------------------------------------------------------------------------ 64 bits
def _x_e2m1(v):
    """Nearest grid value, ties to the even code, on float64 tensors."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    a = v.abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    mid = (grid[hi - 1] + grid[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return torch.copysign(torch.where(up, grid[hi], grid[hi - 1]), v)


def _x_e4m3(v):
    """Magnitudes rounded to E4M3, ties to even, 448 at most."""
    ex = torch.floor(torch.log2(torch.where(v > 0, v, 1.0))).clamp(min=-6)
    ulp = torch.exp2(ex - 3)
    return (torch.round(v / ulp) * ulp).clamp(max=448.0)


def _x_matrix(x, fmt):
    """The values the 4-bit matrix of x stands for, by definition, in float64."""
    rows, cols = x.shape
    size = 16 if fmt == "nv" else 32
    x = torch.nn.functional.pad(x.double(), (0, -cols % size))
    r = torch.ones(rows, 1, dtype=torch.float64, device=x.device)
    if fmt == "nv":
        top = x.abs().amax(-1, keepdim=True)
        r = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, 2688.0) / 2688.0)).clamp(min=-62))
        g = (x / r).reshape(rows, -1, size)
        s = _x_e4m3((g.abs().amax(-1, keepdim=True) / 6.0).float().double())
        v = torch.where(s > 0, _x_e2m1((g / torch.where(s > 0, s, 1.0)).float().double()) * s, 0.0)
    else:
        g = x.reshape(rows, -1, size)
        top = g.abs().amax(-1, keepdim=True)
        s = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2)
        v = _x_e2m1(g / s) * s
    return (v.reshape(rows, -1) * r)[:, :cols]


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None
    st = prepare(case, seed)
    if op == "query":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        q = st["q"].double().view(-1, H, D + ROPE)
        cs = torch.view_as_complex(st["rope"].double())[st["pos"].clamp(min=0)][:, None]
        rot = torch.view_as_real(torch.view_as_complex(q[..., D:].reshape(*q.shape[:2], 32, 2).contiguous()) * cs).flatten(-2)
        out = torch.empty(q.shape[0], H, DQK, dtype=torch.float64, device=DEV)
        for h in range(H):
            out[:, h, :LAT] = q[:, h, :D] @ st["w"][h].double()
        out[..., LAT:] = rot
        out[T:] = 0.0
        return out
    if op == "value":
        o, w = st["o"], st["w"]
        return torch.cat([o[:, h].double() @ w[h].double().t() for h in range(case["heads"])], -1)
    x = _x_matrix(st["x"], case["fmt"])
    if op == "quant":
        return x
    return x @ _x_matrix(st["weight"], case["fmt"]).t()
