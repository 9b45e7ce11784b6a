"""Attention over the quantised cache on the GPU against its float64 oracle:
single rows and verification rows, every head layout, lengths from one token,
odd sizes, page lists, rows that see nothing, NaN in masked places, captured
and repeated calls, caches past 32-bit offsets.

Error bound of an output (u = 2^-24, A = sum p |v| / sum p, B = sum p s_v / sum p, n at most
N = 2^bits - 1, c = N / 2, T tokens):
- a score's products are exact in float32 and are summed with at most T_k = 32 +
  D / 4 roundings of partial sums no larger than scale (s_k (N + 1) + |z_k|) sum |q|, so it is off by
  at most e = T_k u scale (s_k (N + 1) + |z_k|) sum |q|. bf16: a query is met as float16 of q 2^k, exact
  but for values so small that they round to its spacing of 2^-24, where the row's largest is at least 128:
  each of D values off by at most 2^-32 of the row's largest, times scale s_k N.
  With the base-2 exponential's 2^-21 relative error a weight is off by e + 2^-21 +
  4 u |score| of itself, which moves the output by at most twice that times A;
- bf16, 8 bits or more than 16 packed rows: a weight w = p s_v is rounded to float16: off by at most 2^-12 w + 2^-25,
  where the row's largest weight is at least 2^8; the error meets n - c, at most c + 1 in size: (c + 1) (2^-12 B + T
  2^-33 max s_v). 4 bits, up to 16 packed rows: w is rounded to 9 bits, which moves the
  output by at most 2^-9 A, and held in two e4m3 terms, off by at most 2^-15 where the row's largest is at
  least 2^6, which meets n: N T 2^-21 max s_v; a query's two terms leave at most 2^-15 of a value where the row's
  largest is at least 128: D values of 2^-22 of the row's largest, times scale s_k N. The output's rounding is 2^-8 |out|;
- sums over T tokens: at most T + 64 roundings of partial sums no larger than 2 (N + 1) B + A.
The log-sum-exp is off by at most max e + 2^-21 + (T + 64) u + 4 u |lse|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle.kv_quant as Q                                                     # noqa: E402
from self_sparse_speculative_b200 import s3r                                    # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


class Case:
    """A filled cache: host bytes and device tensors, queries, and what the oracle says."""

    def __init__(self, S, H, G, D, P, bits, lens, rows, dtype, seed=0, budget=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.S, self.H, self.G, self.D, self.P, self.bits, self.rows, self.dtype = S, H, G, D, P, bits, rows, dtype
        self.lens, self.scale = list(lens), 1.0 / np.sqrt(D)
        self.width = max(1, max(-(-max(n, 1) // P) for n in lens))
        total = S * self.width + 2
        table = rng.permutation(total)[:S * self.width].reshape(S, self.width).astype(np.int32)
        self.pages = torch.zeros((total, H, Q.page_bytes(D, P, bits)), dtype=torch.uint8, device="cuda")
        self.table, self.dlens = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kvq = s3r.paged_kvq(self.pages, self.table, self.dlens, H * G, D, P, bits)
        # the cache through the library's own writer (checked byte for byte elsewhere)
        kc = torch.from_numpy(rng.standard_normal((total, H, P, D)).astype(np.float32) * spread
                              + rng.standard_normal((total, H, P, 1)).astype(np.float32)).cuda()
        vc = torch.from_numpy(rng.standard_normal((total, H, P, D)).astype(np.float32)
                              + 0.5 * rng.standard_normal((total, H, P, 1)).astype(np.float32)).cuda()
        full = torch.full((S,), self.width * P, dtype=torch.int32, device="cuda")
        ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
        s3r.s3r_kvq_pack(s3r.paged_kv(kc, vc, self.table, full, H * G), self.kvq, 0, ws)
        assert s3r.s3r_device_status(ws) == (0, 0)
        self.host_table = table
        self.q = torch.from_numpy(rng.standard_normal((S, rows, H * G, D)).astype(np.float32)).to(DT[dtype]).cuda()
        self.out = torch.full_like(self.q, 77.0)
        self.lse = torch.full((S, rows, H * G), 77.0, device="cuda")
        self.budget, self.list = budget, None
        self.ws = torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(self.kvq, dtype, rows, budget), dtype=torch.uint8,
                              device="cuda")
        assert self.ws.numel() > 0

    def set_list(self, lists):
        """lists [S, H, budget] logical pages."""
        self.list = torch.tensor(lists, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        s3r.s3r_kvq_attn(self.kvq, self.q, self.dtype, self.rows, self.scale, self.out, self.lse, self.ws, pages=self.list,
                         budget_pages=self.budget, **kw)

    def check(self, seqs=None, skip=()):
        pages, lists = self.pages.cpu().numpy(), None if self.list is None else self.list.cpu().numpy()
        N = 2 ** self.bits - 1
        for b in range(self.S) if seqs is None else seqs:
            if b in skip:
                continue
            L = self.lens[b]
            held = Q.held_rows(pages, self.host_table[b], L, self.D, self.P, self.bits)
            pos = None
            if lists is not None:
                pos = [np.concatenate([np.arange(i * self.P, min(L, (i + 1) * self.P)) for i in lists[b, h] if i >= 0]
                                      or [np.zeros(0, dtype=np.int64)]) for h in range(self.H)]
            q = self.q[b].float().cpu().numpy()
            ref, lse, A, B = Q.attend(q, held, self.scale, self.rows, pos)
            T = L if pos is None else max(len(x) for x in pos)
            sumq = np.abs(q.astype(np.float64)).sum(-1)                         # [R, Hq]
            span = (held["sk"] * (N + 1) + np.abs(held["zk"])).max(0).repeat(self.G)   # [Hq]
            e = (32 + self.D / 4) * U * self.scale * span * sumq
            e4 = self.dtype == "bf16" and self.bits == 4 and self.G * self.rows <= 16
            if self.dtype == "bf16":
                e = e + (self.D * 2.0 ** (-22 if e4 else -32) * np.abs(q).max(-1) * self.scale * N
                         * held["sk"].max(0).repeat(self.G))
            top = np.where(np.isfinite(lse), np.abs(lse), 0.0)
            w = e + 2.0 ** -21 + 4 * U * (top + np.log(max(T, 1)) + 1)
            tol = 2 * w[..., None] * A + (T + 64) * U * (2 * (N + 1) * B[..., None] + A) + 1e-30
            big = T * held["sv"].max(0).repeat(self.G)[None, :, None]
            if self.dtype == "bf16":
                tol = tol + 1.01 * 2.0 ** -8 * np.abs(ref)
                tol = tol + 1.01 * (2.0 ** -9 * A + N * 2.0 ** -21 * big if e4
                                    else (N / 2 + 1) * (2.0 ** -12 * B[..., None] + 2.0 ** -33 * big))
            out, got = self.out[b].double().cpu().numpy(), self.lse[b].double().cpu().numpy()
            bad = np.abs(out - ref) > tol
            assert not bad.any(), (b, np.argwhere(bad)[:3], out[bad][:3], ref[bad][:3], tol[bad][:3])
            assert (np.isfinite(out)).all()
            none = lse == -np.inf
            assert (got[none] == -np.inf).all() and (out[none] == 0).all()
            ltol = w + (T + 64) * U + 4 * U * top
            bad = ~none & ~(np.abs(np.where(none, 0, got) - np.where(none, 0, lse)) <= ltol)
            assert not bad.any(), (b, np.argwhere(bad)[:3], got[bad][:3], lse[bad][:3], ltol[bad][:3])

    def ok(self):
        assert s3r.s3r_device_status(self.ws) == (0, 0)


LENGTHS = {1: [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300], 4: [4, 5, 16, 18, 64, 66, 130, 257]}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 4])
def test_lengths(D, P, bits, rows, dtype):
    lens = LENGTHS[rows]
    c = Case(len(lens), 2, 3, D, P, bits, lens, rows, dtype, seed=D + P + bits + rows)
    c.call()
    c.check()
    c.ok()


# packed rows G x rows from 1 to 128, over every row tile of the kernels
@pytest.mark.parametrize("G,rows", [(1, 1), (8, 1), (4, 2), (3, 3), (8, 2), (5, 4), (6, 4), (4, 7), (8, 4), (5, 8), (5, 9),
                                    (8, 6), (7, 8), (4, 16), (8, 8), (1, 17), (5, 13), (8, 9), (6, 17), (8, 16), (7, 17)])
@pytest.mark.parametrize("D,P,bits", [(128, 64, 4), (64, 16, 4), (128, 64, 8), (64, 64, 8)])
def test_packed_rows(D, P, bits, G, rows):
    c = Case(3, 2, G, D, P, bits, [17, 200, 131], rows, "bf16", seed=G * rows)
    c.call()
    c.check()
    c.ok()


@pytest.mark.parametrize("G,rows", [(1, 1), (8, 16), (7, 17)])
def test_packed_rows_f32(G, rows):
    c = Case(2, 2, G, 128, 64, 4, [17, 100], rows, "f32", seed=G)
    c.call()
    c.check()
    c.ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
def test_long_sequences_split_over_many_ctas(bits, dtype):
    c = Case(2, 1, 4, 128, 64, bits, [9001, 4097], 3, dtype, seed=1)
    for _ in range(3):                                   # the workspace serves the next call as it is
        c.out.fill_(77.0)
        c.lse.fill_(77.0)
        c.call()
    c.check()
    c.ok()


def test_many_short_sequences():
    lens = [int(x) for x in np.random.default_rng(0).integers(2, 60, 300)]
    c = Case(300, 2, 2, 64, 16, 4, lens, 2, "bf16", seed=2)
    c.call()
    c.check(seqs=range(0, 300, 7))
    c.ok()


def test_scores_that_grow_along_the_sequence():
    # the reference of the softmax is raised again and again (large scores, late maxima)
    for bits in (4, 8):
        c = Case(2, 1, 2, 128, 64, bits, [1500, 700], 2, "bf16", seed=3, spread=6.0)
        c.q.mul_(4)
        c.call()
        c.check()
        c.ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,P", [(128, 64), (64, 16)])
@pytest.mark.parametrize("rows", [1, 3])
def test_page_lists(D, P, rows, dtype):
    S, H, B = 4, 2, 7
    c = Case(S, H, 4, D, P, 4, [5 * P + 3, 9 * P, rows, 12 * P + 1], rows, dtype, seed=4, budget=B)
    rng = np.random.default_rng(5)
    lists = np.full((S, H, B), -1)
    for b in range(S):
        n_b = -(-c.lens[b] // P)
        for h in range(H):
            ids = rng.permutation(n_b)[:B - 2]
            lists[b, h, :len(ids)] = np.sort(ids)
    lists[0, 0] = [-1, 3, -1, 5, 0, -1, -1]              # any order, gaps
    lists[0, 1] = [2, 2, 2, 1, -1, 1, 0]                 # repeated pages count again
    lists[1, 0] = -1                                     # nothing: every row is empty
    lists[1, 1] = [8, -1, -1, -1, -1, -1, -1]
    lists[3, 0] = [12, -1, -1, -1, -1, -1, -1]           # one position: the earlier rows see none of it
    c.set_list(lists)
    for _ in range(2):
        c.call()
    c.check()
    c.ok()
    assert (c.lse[1, :, :4] == -np.inf).all() and (c.out[1, :, :4] == 0).all()
    if rows == 3:
        assert (c.lse[3, :2, :4] == -np.inf).all() and torch.isfinite(c.lse[3, 2, :4]).all()


def test_list_longer_than_the_table_and_many_units():
    c = Case(80, 4, 2, 64, 16, 4, [33] * 80, 1, "bf16", seed=6, budget=40)
    lists = np.full((80, 4, 40), -1)
    lists[:, :, 37], lists[:, :, 2] = 2, 0
    c.set_list(lists)
    c.call()
    c.check(seqs=range(0, 80, 9))
    c.ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_lengths_and_pages(dtype):
    S, P = 7, 16
    c = Case(S, 2, 2, 64, P, 4, [40, 33, 48, 20, 40, 40, 40], 3, dtype, seed=7)
    c.dlens.copy_(torch.tensor([40, 2, 49, -5, 0, 40, 2 ** 31 - 1], dtype=torch.int32))
    c.call()
    for b in (1, 2, 3, 4, 6):                            # shorter than the rows, longer than the table, no length
        assert (c.out[b] == 0).all() and (c.lse[b] == -np.inf).all()
    c.check(seqs=[0, 5])
    assert s3r.s3r_device_status(c.ws)[1] == s3r.S3R_DEV_BAD_CONTEXT_LEN
    # a bad page is left out, the others are attended to
    c = Case(S, 2, 2, 64, P, 4, [48] * S, 1, dtype, seed=8, budget=3)
    c.table[0, 1], c.table[1, 0] = -1, 10 ** 7
    lists = np.tile(np.arange(3), (S, 2, 1))
    lists[2, 0], lists[3, 1] = [0, 3, 1], [-2, 2, 2 ** 31 - 1]
    c.set_list(lists)
    c.call()
    assert s3r.s3r_device_status(c.ws)[1] == s3r.S3R_DEV_BAD_PAGE_ID
    good = lists.copy()
    good[0, :, 1] = good[1, :, 0] = -1
    good[2, 0], good[3, 1] = [0, 1, -1], [-1, 2, -1]
    c.list = torch.from_numpy(good.astype(np.int32))
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
def test_nan_rows_reach_only_the_rows_that_see_them(bits, dtype):
    S, H, G, D, P, rows = 3, 2, 3, 64, 16, 3
    lens = [30, 30, 300]
    c = Case(S, H, G, D, P, bits, lens, rows, dtype, seed=9)
    # every slot behind the sequences, whole unused pages, and one visible position of head 1 in sequence 1
    raw = c.pages.cpu().numpy()
    half = P * D * bits // 8
    nan = np.array([0x7FC0, 0x7FC0], dtype="<u2").view(np.uint8)
    used = set(c.host_table.reshape(-1).tolist())
    for b in range(S):
        for pos in range(lens[b], c.width * P):
            for par in (half, 2 * half + 4 * P):
                raw[c.host_table[b, pos // P], :, par + 4 * (pos % P):par + 4 * (pos % P) + 4] = nan
    for i in set(range(len(raw))) - used:
        raw[i] = 0xFF
    clean = raw.copy()
    # position 28 (row 1's own): rows 1 and 2 see it, row 0 does not
    for par in (half, 2 * half + 4 * P):
        raw[c.host_table[1, 1], 1, par + 4 * 12:par + 4 * 12 + 4] = nan
    # a NaN value row alone at the last position of sequence 2, head 0: row 2 alone sees it
    at = 2 * half + 4 * P + 4 * (299 % P)
    raw[c.host_table[2, 299 // P], 0, at:at + 4] = nan
    c.pages.copy_(torch.from_numpy(raw))
    c.call()
    c.ok()
    nans = torch.isnan(c.out).all(-1).cpu()
    some = torch.isnan(c.out).any(-1).cpu()
    want = torch.zeros((S, rows, H * G), dtype=torch.bool)
    want[1, 1:, G:] = True
    want[2, 2, :G] = True
    assert torch.equal(nans, want) and torch.equal(some, want)
    assert torch.isnan(c.lse[1, 1:, G:]).all() and not torch.isnan(c.lse[2]).any() and not torch.isnan(c.lse[0]).any()
    # the others are what they are without it
    out, lse = c.out.clone(), c.lse.clone()
    c.pages.copy_(torch.from_numpy(clean))
    c.call()
    c.check()
    w = want.cuda()
    assert torch.equal(out[~w], c.out[~w]) and torch.equal(lse[~w], c.lse[~w])


def test_without_lse_on_another_stream_and_repeatable():
    c = Case(3, 2, 4, 128, 64, 4, [500, 64, 1], 1, "bf16", seed=10)
    c.call()
    torch.cuda.synchronize()
    ref, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    c.out.fill_(3.0)
    c.lse.fill_(4.0)
    torch.cuda.synchronize()
    s3r.s3r_kvq_attn(c.kvq, c.q, "bf16", 1, c.scale, c.out, None, c.ws, stream=side)
    side.synchronize()
    assert torch.equal(c.out, ref) and (c.lse == 4.0).all()
    for _ in range(20):
        c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out, ref) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_other_scales(scale, bits, dtype):
    c = Case(2, 2, 4, 128, 64, bits, [333, 5], 2, dtype, seed=21)
    c.scale = scale
    c.call()
    if scale >= 0:
        c.check()
    else:                                                                      # the same rows, queries negated
        out, lse = c.out.clone(), c.lse.clone()
        c.scale, c.q = -scale, -c.q
        c.check()
        c.call()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)
    c.ok()


@pytest.mark.parametrize("bits,G,rows,dtype", [(4, 4, 2, "bf16"), (4, 4, 5, "bf16"), (8, 4, 2, "bf16"), (8, 5, 9, "bf16"),
                                               (4, 4, 2, "f32")])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite_reach_their_own_row_only(bits, G, rows, dtype, value):
    c = Case(2, 2, G, 128, 64, bits, [700, 130], rows, dtype, seed=22)
    c.call()
    out, lse, q = c.out.clone(), c.lse.clone(), c.q.clone()
    at = (0, rows - 1, G)
    c.q[at][17] = value
    c.call()
    c.ok()
    if value != value:
        assert c.out[at].isnan().all() and c.lse[at].isnan()
    c.out[at], c.lse[at], c.q = out[at], lse[at], q
    c.check()


def test_captured_graphs_share_a_workspace():
    # two graphs over one workspace, replayed one after the other, in both orders
    c = Case(2, 2, 4, 128, 64, 8, [3000, 700], 2, "bf16", seed=11)
    q2 = (c.q.float() * 1.5).to(torch.bfloat16)
    outs = [torch.zeros_like(c.q) for _ in range(2)]
    want = []
    for q, o in zip((c.q, q2), outs):
        s3r.s3r_kvq_attn(c.kvq, q, "bf16", 2, c.scale, o, None, c.ws)
        want.append(o.clone())
    graphs = []
    for q, o in zip((c.q, q2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s3r.s3r_kvq_attn(c.kvq, q, "bf16", 2, c.scale, o, None, c.ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], want[i]), order
    c.ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_past_32_bit_offsets(dtype):
    # 5 GB of pages; the sequences' own lie at its end
    S, H, G, D, P, bits = 2, 2, 2, 128, 64, 4
    nb = s3r.s3r_kvq_page_bytes(D, P, bits)
    total = 5 * 2 ** 30 // (H * nb)
    pages = torch.empty((total, H, nb), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[total - 1, total - 3, total - 5], [total - 2, 0, total - 4]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    kvq = s3r.paged_kvq(pages, table, lens, H * G, D, P, bits)
    ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
    n = 2 * P + 9
    k = torch.randn((S, n, H, D), device="cuda").to(DT[dtype])
    v = torch.randn((S, n, H, D), device="cuda").to(DT[dtype])
    s3r.s3r_kvq_append(kvq, lens, k, v, dtype, n, 0, ws)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    s3r.s3r_kvq_read(kvq, None, n, dtype, ko, vo, ws)
    for x, y in ((k, ko), (v, vo)):
        m, s, z = Q.quantise_rows(x.float().cpu().numpy(), bits)
        ref = (Q.bf16_value(s)[..., None] * m + Q.bf16_value(z)[..., None]).astype(np.float32)
        assert torch.equal(y.cpu(), torch.from_numpy(ref).to(DT[dtype]))
    q = torch.randn((S, 1, H * G, D), device="cuda").to(DT[dtype])
    out, lse = torch.zeros_like(q), torch.zeros((S, 1, H * G), device="cuda")
    wa = torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(kvq, dtype, 1), dtype=torch.uint8, device="cuda")
    s3r.s3r_kvq_attn(kvq, q, dtype, 1, 0.1, out, lse, wa)
    # the same rows in a small cache give the same answer
    small = torch.zeros((6, H, nb), dtype=torch.uint8, device="cuda")
    kvq2 = s3r.paged_kvq(small, torch.arange(6, dtype=torch.int32, device="cuda").reshape(2, 3), lens, H * G, D, P, bits)
    s3r.s3r_kvq_append(kvq2, None, k, v, dtype, n, n, ws)
    out2, lse2 = torch.zeros_like(q), torch.zeros_like(lse)
    s3r.s3r_kvq_attn(kvq2, q, dtype, 1, 0.1, out2, lse2, wa)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert s3r.s3r_device_status(ws) == (0, 0) and s3r.s3r_device_status(wa) == (0, 0)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_run_of_the_calls_together(bits):
    """Rounds of a self-speculating decoder on the quantised cache alone: prompt, drafter's single rows, verification
    rows over the round's positions, rollback; lengths, bytes and outputs as the oracle's."""
    S, H, G, D, P, width, gamma = 3, 2, 4, 128, 64, 4, 3
    rng = np.random.default_rng(12)
    table = rng.permutation(S * width).reshape(S, width).astype(np.int32)
    host = np.zeros((S * width, H, Q.page_bytes(D, P, bits)), dtype=np.uint8)
    pages, dtable = torch.from_numpy(host.copy()).cuda(), torch.from_numpy(table).cuda()
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    kvq = s3r.paged_kvq(pages, dtable, lens, H * G, D, P, bits)
    ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
    wa = {r: torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(kvq, "bf16", r), dtype=torch.uint8, device="cuda")
          for r in (1, gamma + 1)}
    hl = [0] * S

    def store(n, over):
        k, v = (torch.from_numpy(rng.standard_normal((S, n, H, D)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
        s3r.s3r_kvq_append(kvq, lens, k.cuda(), v.cuda(), "bf16", n, over, ws)
        Q.append(host, table, hl, k.float().numpy(), v.float().numpy(), bits, P, over)

    def attend(rows):
        q = torch.from_numpy(rng.standard_normal((S, rows, H * G, D)).astype(np.float32)).to(torch.bfloat16).cuda()
        out, lse = torch.zeros_like(q), torch.zeros((S, rows, H * G), device="cuda")
        s3r.s3r_kvq_attn(kvq, q, "bf16", rows, 0.09, out, lse, wa[rows])
        for b in range(S):
            held = Q.held_rows(host, table[b], hl[b], D, P, bits)
            ref, rl, A, B = Q.attend(q[b].float().cpu().numpy(), held, 0.09, rows)
            # the weights' and the output's roundings as above; scores and float32 sums are far below 2^-10 of A
            few = 15 * hl[b] * 2.0 ** -21 * held["sv"].max()
            tol = 1.01 * (2 ** (bits - 1) * 2.0 ** -12 * B[..., None] + 2.0 ** -8 * np.abs(ref)) + 2.0 ** -10 * A
            if bits == 4:
                tol = tol + 1.01 * 2.0 ** -9 * A + few
            assert (np.abs(out[b].double().cpu().numpy() - ref) <= tol).all()
            assert np.abs(lse[b].double().cpu().numpy() - rl).max() < 1e-3

    store(P + 5, 0)
    for _ in range(4):
        for _ in range(gamma):
            store(1, 0)
            attend(1)
        store(gamma + 1, gamma)
        attend(gamma + 1)
        acc = rng.integers(0, gamma + 1, S)
        s3r.s3r_kvq_rollback(kvq, lens, torch.from_numpy(acc.astype(np.int32)).cuda(), gamma + 1, ws)
        hl = [x - (gamma + 1) + int(a) + 1 for x, a in zip(hl, acc)]
        assert lens.tolist() == hl
    assert np.array_equal(pages.cpu().numpy(), host)
    assert s3r.s3r_device_status(ws) == (0, 0) and all(s3r.s3r_device_status(w) == (0, 0) for w in wa.values())
