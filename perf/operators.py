"""The quantised key/value cache's operators as workloads: rows stored into a paged cache held in 4 or
8 bits, rows read back from it, and attention over it.

Every token row x[0..D) of a KV head is held as D whole numbers n and two bf16 parameters:
  z = the row's minimum rounded down to bf16,  s = (max - z) / (2^bits - 1) rounded to bf16
  n = (x - z) / s rounded to the nearest whole number (ties to even), 0 <= n < 2^bits
  and stands for s n + z. A row whose s would be below 2^-100 has s = 1 and n = 0.
One page of one head is one run of bytes (see `lay_out`): the keys' numbers in 16-byte pieces, piece by
piece over the page's tokens; the keys' (s, z); the values' numbers with the tokens along a channel
together, in pieces of up to 16 bytes, piece by piece over the channels; the values' (s, z).

`run` computes the operators in elementary torch operations, or, where `own` is set, through the
library's calls.
"""
import math

import numpy as np
import torch

own = False

TINY = 2.0 ** -100


# ------------------------------------------------------------------ cases
def _c(name, op, **kw):
    d = dict(op=op, seqs=1, q_heads=4, kv_heads=1, dim=128, page=64, lmin=256, lmax=256, bits=4, dtype="bf16",
             rows=1, n=1, budget=0)
    d.update(kw)
    if name:
        d["name"] = name
    return d


def listed():
    eight = dict(q_heads=32, kv_heads=8, dim=128, page=64)      # an 8B model's layer: 32 query, 8 KV heads
    return [
        # a draft step's one new row in each of 16 sequences: latency
        _c("store-draft-row", "append", seqs=16, lmin=16384, lmax=16384, n=1, **eight),
        # a prompt's next 1000 tokens in each of 64 sequences of mixed lengths
        _c("store-prompt-1000", "append", seqs=64, lmin=1000, lmax=9000, n=1000, **eight),
        # a bf16 cache's 16 x 16384 tokens quantised after the prompt, and read back
        _c("pack-16x16k", "pack", seqs=16, lmin=16384, lmax=16384, **eight),
        # a window of 500 tokens of each sequence, 8 bits (tokens moved to another cache)
        _c("read-window-500", "read", seqs=16, lmin=700, lmax=16384, n=500, bits=8, **eight),
        # everything of short mixed sequences in 16-token pages, as float32
        _c("read-all-f32", "read", seqs=48, q_heads=16, kv_heads=4, dim=64, page=16, lmin=1, lmax=4097, n=4097,
           dtype="f32"),
        # one token of one short sequence: the smallest call
        _c("attend-1x256", "attend", dim=64, page=16, lmin=256, lmax=256),
        # the float32 check model's verification rows over 8 bits
        _c("attend-f32-rows4", "attend", seqs=2, dim=64, page=16, lmin=251, lmax=777, bits=8, dtype="f32", rows=4),
        # a drafter's single rows over 16 x 16384 tokens in 4 bits
        _c("attend-16x16k", "attend", seqs=16, lmin=16384, lmax=16384, **eight),
        # verification rows over the same cache in 8 bits
        _c("attend-16x16k-rows5-b8", "attend", seqs=16, lmin=16384, lmax=16384, bits=8, rows=5, **eight),
        # 64 sequences of mixed length
        _c("attend-ragged", "attend", seqs=64, lmin=4097, lmax=32767, **eight),
        # a wide batch verifying eight drafts (40 query heads)
        _c("attend-256x8k-rows9", "attend", seqs=256, q_heads=40, kv_heads=8, lmin=8192, lmax=8192, rows=9),
        # a drafter's single rows over 64 kept pages of four long sequences
        _c("attend-pages-4x64k", "attend", seqs=4, lmin=65536, lmax=65536, budget=64, **eight),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "pack", "read", "attend", "attend", "attend"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.randint(1, 8)
    dim, page, bits = rng.choice([64, 128]), rng.choice([16, 64]), rng.choice([4, 8])
    # tokens x heads at most a quarter of the largest listed cache; less for float32, a check's type
    room = (1 << 17) if dtype == "f32" and op == "attend" else (1 << 22)
    lmax = _between(rng, 1, min(65536, room // kv_heads))
    seqs = _between(rng, 1, max(1, min(128, room // (kv_heads * lmax))))
    lmin = lmax if rng.random() < 0.3 else _between(rng, 1, lmax)
    rows, n, budget = 1, 1, 0
    if op == "attend":
        rows = min(lmin, rng.choice([1, 1, rng.randint(2, 17)]), 128 // group)
        if rng.random() < 0.25:
            budget = rng.randint(1, 1 + lmax // page)
    elif op == "append":
        n = _between(rng, 1, min(1024, lmin))
    elif op == "read":
        n = _between(rng, 1, lmax)
    return _c("", op, seqs=seqs, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, lmin=lmin, lmax=lmax,
              bits=bits, dtype=dtype, rows=rows, n=n, budget=budget)


def lengths(case):
    """The sequences' lengths: spread over lmin..lmax, both met where there are two sequences."""
    S, lo, hi = case["seqs"], case["lmin"], case["lmax"]
    at = (np.arange(S) * 0.6180339887498949) % 1.0
    L = (lo + np.floor(at * (hi - lo + 1))).astype(np.int64)
    L[-1] = hi
    return np.clip(L, lo, hi)


def _starts(case):
    """First position of a read window: the last n positions, or the beginning of a shorter sequence."""
    return np.maximum(lengths(case) - case["n"], 0)


def work(case):
    S, Hq, H, D, P = case["seqs"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    L = lengths(case)
    elt = 4 if case["dtype"] == "f32" else 2
    row = 2 * D * case["bits"] // 8 + 8                       # a token's keys and values of one head, held
    if case["op"] == "attend":
        tokens = np.minimum(L, case["budget"] * P).sum() if case["budget"] else L.sum()
        io = 2 * S * case["rows"] * Hq * D * elt + 4 * S * case["rows"] * Hq
        return {"bytes": int(tokens) * H * row + io, "flops": 4 * int(tokens) * Hq * case["rows"] * D}
    if case["op"] == "append":
        t = S * case["n"] * H
        return {"bytes": t * (2 * D * elt * 2 + row), "flops": 0}
    if case["op"] == "pack":
        t = int(L.sum()) * H
        return {"bytes": t * (2 * D * elt * 2 + row), "flops": 0}
    t = int((L - _starts(case)).sum()) * H
    return {"bytes": t * (2 * D * elt + row), "flops": 0}


# ------------------------------------------------------------------ the format
def page_bytes(D, P, bits):
    return 2 * (P * D * bits // 8) + 8 * P


def _down_bf16(x):
    """float32 rounded towards minus infinity to bf16 values."""
    y = x.bfloat16().float()
    i = y.view(torch.int32)
    lower = torch.where(y > 0, i - 65536, torch.where(y == 0, torch.full_like(i, -2147483648 + 65536), i + 65536))
    return torch.where(y > x, lower.view(torch.float32), y)


def quantise(x, bits):
    """Rows x [..., D] (float32): whole numbers (uint8) [..., D], s and z [...] (float32 of bf16 values)."""
    top = 2 ** bits - 1
    fine = torch.isfinite(x).all(-1)
    z = _down_bf16(x.amin(-1))
    s = ((x.amax(-1).double() - z.double()) / top).float().bfloat16().float()
    flat = s < TINY
    s = torch.where(flat | ~fine, torch.ones_like(s), s)
    n = torch.round((x.double() - z.double().unsqueeze(-1)) / s.double().unsqueeze(-1)).clamp(0, top)
    n = torch.where((flat | ~fine).unsqueeze(-1), torch.zeros_like(n), n).to(torch.uint8)
    return n, s, torch.where(fine, z, torch.full_like(z, math.nan))


def _pieces(n, bits, inner):
    """[A, rows, len] whole numbers -> bytes [A, piece, rows, size], `size` = min(16, len * bits / 8)."""
    b = n if bits == 8 else n[..., 0::2] | (n[..., 1::2] << 4)
    size = min(16, b.shape[-1])
    return b.reshape(b.shape[0], inner, -1, size).permute(0, 2, 1, 3).reshape(b.shape[0], -1)


def _from_pieces(b, bits, inner, length):
    """The inverse of `_pieces`: bytes [A, x] -> whole numbers (uint8) [A, inner, length]."""
    size = min(16, length * bits // 8)
    b = b.reshape(b.shape[0], -1, inner, size).permute(0, 2, 1, 3).reshape(b.shape[0], inner, -1)
    return b if bits == 8 else torch.stack((b & 15, b >> 4), -1).reshape(b.shape[0], inner, -1)


def lay_out(kn, ks, kz, vn, vs, vz, bits):
    """Pages [A, P, D] of numbers and [A, P] of parameters -> bytes [A, page_bytes]."""
    A, P, D = kn.shape
    par = lambda s, z: torch.stack((s, z), -1).bfloat16().reshape(A, 2 * P).view(torch.uint8)  # noqa: E731
    return torch.cat((_pieces(kn, bits, P), par(ks, kz), _pieces(vn.transpose(1, 2), bits, D), par(vs, vz)), 1)


def stands_for(b, D, P, bits):
    """Bytes [A, page_bytes] -> the float32 keys and values [A, P, D] that they stand for."""
    A, half = b.shape[0], P * D * bits // 8

    def par(at):
        sz = b[:, at:at + 4 * P].contiguous().view(torch.bfloat16).float().reshape(A, P, 2)
        return sz[..., 0:1], sz[..., 1:2]

    s, z = par(half)
    k = _from_pieces(b[:, :half], bits, P, D).float() * s + z
    s, z = par(2 * half + 4 * P)
    at = half + 4 * P
    v = _from_pieces(b[:, at:at + half], bits, D, P).transpose(1, 2).float() * s + z
    return k, v


# ------------------------------------------------------------------ inputs
def _rows(gen, shape, heads_at, dtype):
    """Keys or values: N(0, 1) and, per head, eight channels that move together."""
    dev = gen.device
    H, D = shape[heads_at], shape[-1]
    x = torch.randn(shape, generator=gen, device=dev)
    w = torch.zeros((H, D), device=dev)
    w.scatter_(1, torch.rand((H, D), generator=gen, device=dev).argsort(1)[:, :8],
               torch.randn((H, 8), generator=gen, device=dev) / math.sqrt(8.0))
    t = 2.0 * torch.randn(shape[:-1] + (1,), generator=gen, device=dev)
    lead = [1] * len(shape)
    lead[heads_at], lead[-1] = H, D
    return (x + t * w.reshape(lead)).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) + 1)
    S, Hq, H, D, P, bits = (case[k] for k in ("seqs", "q_heads", "kv_heads", "dim", "page", "bits"))
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    L = lengths(case)
    n_b = -(-L // P)
    width = int(n_b.max())
    total = int(n_b.sum())
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    at = np.concatenate(([0], np.cumsum(n_b)))[:-1]
    index = torch.from_numpy(np.minimum(at[:, None] + np.arange(width), total - 1)).to(dev)
    table = torch.where(torch.arange(width, device=dev) < torch.from_numpy(n_b).to(dev)[:, None], order[index],
                        torch.zeros_like(order[index]))
    st = dict(case=dict(case), table=table.contiguous(), lens=torch.from_numpy(L.astype(np.int32)).to(dev),
              scale=1.0 / math.sqrt(D), handle=None)
    nb = page_bytes(D, P, bits)
    st["pages"] = torch.zeros((total, H, nb), dtype=torch.uint8, device=dev)
    if case["op"] in ("attend", "read"):
        step = max(1, (1 << 27) // (H * P * D))
        for a in range(0, total, step):
            m = min(step, total - a)
            kn = quantise(_rows(gen, (m, H, P, D), 1, dt).float().reshape(m * H, P, D), bits)
            vn = quantise(_rows(gen, (m, H, P, D), 1, dt).float().reshape(m * H, P, D), bits)
            st["pages"][a:a + m] = lay_out(*kn, *vn, bits).reshape(m, H, nb)
    if case["op"] == "attend":
        R = case["rows"]
        st["q"] = _rows(gen, (S, R, Hq, D), 2, dt)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((S, R, Hq), dtype=torch.float32, device=dev)
        st["kept"] = None
        if case["budget"]:
            # kept pages, ascending, the newest among them; -1 behind the last
            B, at = case["budget"], torch.arange(width, device=dev)
            nb_ = torch.from_numpy(n_b).to(dev)[:, None, None]
            key = torch.rand((S, H, width), generator=gen, device=dev)
            key = torch.where(at == nb_ - 1, 2.0, torch.where(at < nb_, key, -1.0))
            top, ids = key.topk(min(B, width), dim=-1)
            ids = torch.where(top < 0, width, ids).sort(-1).values
            kept = torch.full((S, H, B), -1, dtype=torch.int32, device=dev)
            kept[:, :, :ids.shape[-1]] = torch.where(ids < width, ids, -1).to(torch.int32)
            st["kept"] = kept
    elif case["op"] == "append":
        st["k"] = _rows(gen, (S, case["n"], H, D), 2, dt)
        st["v"] = _rows(gen, (S, case["n"], H, D), 2, dt)
    elif case["op"] == "pack":
        st["k"] = _rows(gen, (total, H, P, D), 1, dt)
        st["v"] = _rows(gen, (total, H, P, D), 1, dt)
    if case["op"] != "attend":
        n = int(L.max()) if case["op"] == "pack" else case["n"]
        st["n"] = n
        first = L - n if case["op"] == "append" else np.zeros(S) if case["op"] == "pack" else _starts(case)
        st["first"] = torch.from_numpy(first.astype(np.int32)).to(dev)
        st["k_out"] = torch.zeros((S, n, H, D), dtype=dt, device=dev)
        st["v_out"] = torch.zeros((S, n, H, D), dtype=dt, device=dev)
    return st


# ------------------------------------------------------------------ the operators
def run(st):
    if own:
        return _library(st)
    c = st["case"]
    S, Hq, H, D, P, bits = (c[k] for k in ("seqs", "q_heads", "kv_heads", "dim", "page", "bits"))
    if c["op"] == "append":
        return {"k": _held(st["k"], bits), "v": _held(st["v"], bits)}
    table, lens = st["table"].long(), st["lens"].long()
    if c["op"] == "pack":
        # [S, width, H, P, D] -> the first n positions of every sequence
        there = (torch.arange(st["n"], device=lens.device) < lens[:, None])[:, :, None, None]
        return {x: torch.where(there, _held(st[x], bits)[table].permute(0, 1, 3, 2, 4).reshape(S, -1, H, D)[:, :st["n"]], 0)
                for x in ("k", "v")}
    if c["op"] == "read":
        pos = st["first"].long()[:, None] + torch.arange(st["n"], device=lens.device)
        there = pos < lens[:, None]
        pos = torch.where(there, pos, 0)
        page = table.gather(1, pos // P)
        k, v = stands_for(st["pages"].reshape(-1, st["pages"].shape[-1]), D, P, bits)
        dt = st["k_out"].dtype
        pick = lambda x: torch.where(there[:, :, None, None], x.to(dt).reshape(-1, H, P, D)[page, :, pos % P], 0)  # noqa: E731
        return {"k": pick(k), "v": pick(v)}
    G, R = Hq // H, c["rows"]
    width = table.shape[1]
    if st["kept"] is None:
        logical = torch.arange(width, device=lens.device).expand(S, H, width)
    else:
        logical = st["kept"].long()
    B = logical.shape[-1]
    phys = table[:, None].expand(S, H, width).gather(2, logical.clamp(min=0))
    held = st["pages"][phys, torch.arange(H, device=lens.device)[None, :, None]]
    k, v = stands_for(held.reshape(S * H * B, -1), D, P, bits)
    k, v = k.reshape(S * H, B * P, D), v.reshape(S * H, B * P, D)
    pos = (logical[..., None] * P + torch.arange(P, device=lens.device)).reshape(S, H, 1, B * P)
    last = (lens[:, None] - R + torch.arange(R, device=lens.device)).repeat_interleave(G, 1)      # [S, R G]
    seen = (pos >= 0) & (pos <= last[:, None, :, None])
    q = st["q"].float().reshape(S, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(S * H, R * G, D)
    x = (q @ k.transpose(1, 2)).reshape(S, H, R * G, B * P) * st["scale"]
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(S * H, R * G, B * P) @ v).reshape(S, H, R * G, D) / torch.where(total == 0, 1, total)
    back = lambda y: y.reshape(S, H, R, G, -1).permute(0, 2, 1, 3, 4).reshape(S, R, Hq, -1)  # noqa: E731
    return {"out": back(o).to(st["q"].dtype), "lse": back(top + torch.log(total)).squeeze(-1)}


def _held(x, bits):
    """The values that rows x stand for once held in `bits`, in x's type."""
    n, s, z = quantise(x.float(), bits)
    return (n.float() * s.unsqueeze(-1) + z.unsqueeze(-1)).to(x.dtype)


def _library(st):
    from self_sparse_speculative_b200 import s3r

    c = st["case"]
    h = st["handle"]
    if h is None:                                  # kept by a program: the descriptors and the workspace
        kvq = s3r.paged_kvq(st["pages"], st["table"], st["lens"], c["q_heads"], c["dim"], c["page"], c["bits"])
        size = (s3r.s3r_kvq_attn_workspace_bytes(kvq, c["dtype"], c["rows"], c["budget"]) if c["op"] == "attend"
                else s3r.s3r_kv_workspace_bytes(c["seqs"]))
        kv = (s3r.paged_kv(st["k"], st["v"], st["table"], st["lens"], c["q_heads"]) if c["op"] == "pack" else None)
        h = st["handle"] = (kvq, kv, torch.zeros(size, dtype=torch.uint8, device=st["pages"].device))
    kvq, kv, ws = h
    if c["op"] == "attend":
        s3r.s3r_kvq_attn(kvq, st["q"], c["dtype"], c["rows"], st["scale"], st["out"], st["lse"], ws,
                         pages=st["kept"], budget_pages=c["budget"])
        return {"out": st["out"], "lse": st["lse"]}
    if c["op"] == "append":
        s3r.s3r_kvq_append(kvq, st["lens"], st["k"], st["v"], c["dtype"], c["n"], c["n"], ws)
    elif c["op"] == "pack":
        s3r.s3r_kvq_pack(kv, kvq, 0, ws)
    s3r.s3r_kvq_read(kvq, st["first"], st["n"], c["dtype"], st["k_out"], st["v_out"], ws)
    return {"k": st["k_out"], "v": st["v_out"]}


# ------------------------------------------------------------------ in 64 bits, written apart
def _exact_rows(x, bits):
    """The values that rows stand for, in float64: the definition, row by row of the last axis."""
    x = x.double()
    lo, hi = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
    z = lo.float().bfloat16().double()
    # the bf16 number below z: one step of its own binade (the step below a power of two is half as wide)
    m, e = torch.frexp(z)
    step = torch.ldexp(torch.ones_like(z), e - torch.where(m == 0.5, 9, 8))
    z = torch.where(z > lo, z - step, z)
    s = ((hi - z) / (2 ** bits - 1)).float().bfloat16().double()
    n = torch.clip(torch.round((x - z) / s), 0, 2 ** bits - 1)
    return torch.where(s < TINY, z.expand_as(x), s * n + z)


def _exact_page(raw, D, P, bits):
    """One (page, head)'s bytes -> float64 keys and values [.., P, D], byte by byte from the layout."""
    dev = raw.device
    t, d = torch.meshgrid(torch.arange(P, device=dev), torch.arange(D, device=dev), indexing="ij")
    kb = d * bits // 8
    k_at = (kb // 16) * (P * 16) + t * 16 + kb % 16
    size = min(16, P * bits // 8)
    vb = t * bits // 8
    v_at = (vb // size) * (D * size) + d * size + vb % size
    half = P * D * bits // 8

    def par(at):
        w = raw[..., at:at + 4 * P].to(torch.int64).reshape(*raw.shape[:-1], P, 2, 2)
        u = ((w[..., 0] + 256 * w[..., 1]) << 16).to(torch.int32).view(torch.float32).double()
        return u[..., 0:1], u[..., 1:2]

    def number(at, base, i):
        b = raw[..., (at + base).reshape(-1)].reshape(*raw.shape[:-1], P, D).to(torch.int64)
        return (b if bits == 8 else (b >> (4 * (i % 2))) & 15).double()

    ks, kz = par(half)
    vs, vz = par(2 * half + 4 * P)
    return number(k_at, 0, d) * ks + kz, number(v_at, half + 4 * P, t) * vs + vz


def exact(case, seed):
    st = prepare(case, seed)
    S, Hq, H, D, P, bits, R = (case[k] for k in ("seqs", "q_heads", "kv_heads", "dim", "page", "bits", "rows"))
    L = lengths(case)
    dev = st["pages"].device
    if case["op"] == "append":
        return {"k": _exact_rows(st["k"], bits), "v": _exact_rows(st["v"], bits)}
    if case["op"] in ("pack", "read"):
        got = {x: torch.zeros(st[x + "_out"].shape, dtype=torch.float64, device=dev) for x in ("k", "v")}
        first = np.zeros(S, dtype=np.int64) if case["op"] == "pack" else _starts(case)
        for b in range(S):
            ids = st["table"][b, :-(-int(L[b]) // P)].long()
            if case["op"] == "pack":
                pair = [_exact_rows(st[x][ids], bits) for x in ("k", "v")]
            else:
                pair = _exact_page(st["pages"][ids], D, P, bits)
            m = min(int(L[b] - first[b]), st["n"])
            for x, y in zip(("k", "v"), pair):
                y = y.permute(0, 2, 1, 3).reshape(-1, H, D)
                got[x][b, :m] = y[int(first[b]):int(first[b]) + m]
        return got
    G = Hq // H
    out = torch.zeros((S, R, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.zeros((S, R, Hq), dtype=torch.float64, device=dev)
    for b in range(S):
        n_b = -(-int(L[b]) // P)
        for h in ([None] if st["kept"] is None else range(H)):
            heads = slice(0, H) if h is None else slice(h, h + 1)
            if h is None:
                logical = torch.arange(n_b, device=dev)
            else:
                logical = st["kept"][b, h].long()
                logical = logical[logical >= 0]
            pos = (logical[:, None] * P + torch.arange(P, device=dev)).reshape(-1)
            k, v = _exact_page(st["pages"][st["table"][b].long()[logical], heads], D, P, bits)
            k = k.transpose(0, 1).flatten(1, 2)                 # [heads, tokens, D]
            v = v.transpose(0, 1).flatten(1, 2)
            nh = k.shape[0]
            cols = slice(0, Hq) if h is None else slice(h * G, (h + 1) * G)
            q = st["q"][b, :, cols].double().reshape(R, nh, G, D)
            x = torch.einsum("rhgd,htd->hrgt", q, k) * st["scale"]
            x = torch.where((pos[None, :] <= int(L[b]) - R + torch.arange(R, device=dev)[:, None])[None, :, None, :], x, -math.inf)
            y = torch.logsumexp(x, -1)
            p = torch.where((y == -math.inf)[..., None], 0.0, torch.exp(x - torch.where(y == -math.inf, 0.0, y)[..., None]))
            out[b, :, cols] = torch.einsum("hrgt,htd->rhgd", p, v).reshape(R, nh * G, D)
            lse[b, :, cols] = y.permute(1, 0, 2).reshape(R, nh * G)
    return {"out": out, "lse": lse}
