"""Attention over the quantised cache where the values' rows differ in kind and scale: rows of equal values (held with
numbers that are all 0) that take much of the weight, rows a thousand times smaller or larger than their neighbours.

The values of a head have a mean of +-1 (times the head's scale) a channel, so that outputs are as large as the values
and the bound below is a small part of them. Bound of an output (u = 2^-24, N = 2^bits - 1, c = N / 2, p normalised
weights, T positions; the sums over rows with numbers, `free` rows without):
- the output's rounding, 2^-8 |out|; a score off by at most e = (32 + D / 4) u scale (s_k (N + 1) + |z_k|) sum |q| and the
  exponential's 2^-21 move a weight by e' = e + 2^-21 + 4 u |score| of itself: sum p e' (|v| + |out|);
- a query's smallest values are met with an error of at most 2^-22 (4 bits, up to 16 packed rows) or 2^-32 of the row's
  largest: D of them times scale s_k N, added to e;
- 4 bits, up to 16 packed rows: a weight w = p s_v is rounded to 9 bits, 2^-9 sum p |v|, and to whole steps of 2^-14
  with the row's largest of at least 2^6: by less than a step, N 2^-20 T max p s_v. Otherwise to float16: 2^-12 of itself and
  2^-25 with the largest at least 2^8, against n - c: (c + 1) (2^-12 sum p s_v + 2^-33 T max p s_v). A row without numbers
  has no s_v of its own; its weight is met as if its step were at most 2^-8 |z|: s_v = 2^-8 |z| in these sums;
- sums in float32 over T positions: (T + 64) u (2 (N + 1) sum p s_v + sum p |v|), and with products that stand for
  p z alone, off by 4 u each."""
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
BIAS = 8.0                                                                     # every query's channel 0


def bounded(q, held, n_v, scale, rows, bits, dtype, n_k=None):
    """One sequence: out, lse and the bound of each output (module docstring). n_v [L, H, D]: the values' numbers; n_k:
    the keys' (a key without numbers has no s_k)."""
    if n_k is not None:
        held = dict(held, sk=np.where((n_k == 0).all(-1), 0.0, held["sk"]))
    R, Hq, D = q.shape
    L, H = held["sk"].shape
    G, N = Hq // H, 2 ** bits - 1
    e4 = dtype == "bf16" and bits == 4 and G * rows <= 16
    out, lse, tol = np.zeros((R, Hq, D)), np.zeros((R, Hq)), np.zeros((R, Hq, D))
    for h in range(H):
        free = (n_v[:, h] == 0).all(-1)
        sv = np.where(free, 2.0 ** -8 * np.abs(held["zv"][:, h]), held["sv"][:, h])
        for r in range(R):
            seen = np.arange(L) <= L - R + r
            k, v, s = held["k"][seen, h], held["v"][seen, h], sv[seen]
            T = len(v)
            for g in range(G):
                x = q[r, h * G + g].astype(np.float64)
                y = k @ x * scale
                p = np.exp(y - y.max())
                lse[r, h * G + g] = y.max() + np.log(p.sum())
                p /= p.sum()
                o = p @ v
                e = (32 + D / 4) * U * scale * (held["sk"][seen, h] * (N + 1) + np.abs(held["zk"][seen, h])) * np.abs(x).sum()
                if dtype == "bf16":
                    e = e + D * 2.0 ** (-22 if e4 else -32) * np.abs(x).max() * scale * N * held["sk"][seen, h]
                e = e + 2.0 ** -21 + 4 * U * np.abs(y)
                A, B, top = p @ np.abs(v), p @ s, (p * s).max()
                t = (p * e) @ np.abs(v) + (p @ e) * np.abs(o) + (T + 64) * U * (2 * (N + 1) * B + A) + 4 * U * A
                if dtype == "bf16":
                    t = t + 2.0 ** -8 * np.abs(o)
                    t = t + (2.0 ** -9 * A + N * 2.0 ** -20 * T * top if e4
                             else (N / 2 + 1) * (2.0 ** -12 * B + 2.0 ** -33 * T * top))
                out[r, h * G + g], tol[r, h * G + g] = o, 1.01 * t
    return out, lse, tol


class Cache:
    """kinds[h](rng, v) turns the values [S, T, D] of head h, made with a mean of +-1 a channel, into what it needs."""

    def __init__(self, lens, kinds, G, rows, D, P, bits, dtype, weight=None, seed=0):
        rng = np.random.default_rng(seed)
        S, H, T = len(lens), len(kinds), max(lens)
        self.lens, self.rows, self.D, self.P, self.bits, self.dtype = lens, rows, D, P, bits, dtype
        self.scale = D ** -0.5
        width = -(-T // P)
        self.table = rng.permutation(S * width).reshape(S, width).astype(np.int32)
        k = rng.standard_normal((S, T, H, D)).astype(np.float32)
        k[..., 0] = 0
        if weight is not None:                              # position 1 takes about this weight of every row
            k[:, 1] *= 0.01
            k[:, 1, :, 0] = np.log(T * 1.13 * weight / (1 - weight)) / (BIAS * self.scale)
        v = np.empty((S, T, H, D), dtype=np.float32)
        mean = rng.choice([-1.0, 1.0], (H, D))
        for h, kind in enumerate(kinds):
            v[:, :, h] = kind(rng, mean[h] + 0.25 * rng.standard_normal((S, T, D)))
        q = 0.5 * rng.standard_normal((S, rows, H * G, D)).astype(np.float32)
        q[..., 0] = BIAS
        self.q = torch.from_numpy(q).to(DT[dtype]).cuda()
        self.pages = torch.zeros((S * width, H, Q.page_bytes(D, P, bits)), dtype=torch.uint8, device="cuda")
        self.dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        full = torch.zeros(S, dtype=torch.int32, device="cuda")
        dtable = torch.from_numpy(self.table).cuda()
        ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
        writer = s3r.paged_kvq(self.pages, dtable, full, H * G, D, P, bits)     # (checked byte for byte elsewhere)
        for a in range(0, T, 1024):
            x, y = (torch.from_numpy(np.ascontiguousarray(z[:, a:a + 1024])).to(DT[dtype]).cuda() for z in (k, v))
            s3r.s3r_kvq_append(writer, full, x, y, dtype, x.shape[1], 0, ws)
        assert s3r.s3r_device_status(ws) == (0, 0)
        self.kvq = s3r.paged_kvq(self.pages, dtable, self.dlens, H * G, D, P, bits)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros((S, rows, H * G), device="cuda")
        self.ws = torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(self.kvq, dtype, rows), dtype=torch.uint8, device="cuda")

    def call(self):
        s3r.s3r_kvq_attn(self.kvq, self.q, self.dtype, self.rows, self.scale, self.out, self.lse, self.ws)

    def numbers(self, b):
        raw, n = self.pages.cpu().numpy(), -(-self.lens[b] // self.P)
        return np.concatenate([np.stack([Q.read_page(raw[i, h], self.D, self.P, self.bits)[3] for h in range(raw.shape[1])], 1)
                               for i in self.table[b, :n]])[:self.lens[b]]

    def check(self, seqs):
        raw = self.pages.cpu().numpy()
        for b in seqs:
            held = Q.held_rows(raw, self.table[b], self.lens[b], self.D, self.P, self.bits)
            ref, lse, tol = bounded(self.q[b].float().cpu().numpy(), held, self.numbers(b), self.scale, self.rows, self.bits,
                                    self.dtype)
            out = self.out[b].double().cpu().numpy()
            worst = np.abs(out - ref) - tol
            G = out.shape[1] // raw.shape[1]
            for h in range(raw.shape[1]):                   # head by head, so that a failure names its kind
                o, r = out[:, h * G:(h + 1) * G], ref[:, h * G:(h + 1) * G]
                l2 = np.linalg.norm(o - r) / (np.linalg.norm(r) + 1e-300)
                assert (worst[:, h * G:(h + 1) * G] <= 1e-18).all(), (b, h, l2, tol[0, h * G, :3], r[0, 0, :3], o[0, 0, :3])
            assert np.abs(self.lse[b].double().cpu().numpy() - lse).max() < 1e-3
        assert s3r.s3r_device_status(self.ws) == (0, 0)


def sink(value, scale):
    """Position 1 holds one value in every channel; the others are `scale` times as large as usual."""
    def kind(rng, v):
        v = scale * v
        v[:, 1] = value
        return v
    return kind


def every_third(value, scale):
    def kind(rng, v):
        v = scale * v
        v[:, ::3] = value
        return v
    return kind


# packed rows of every form of the kernel: 4 and 16 of 4 bits, 20 and 45 of both widths, float32
FORMS = [(4, 4, 1, "bf16"), (4, 4, 4, "bf16"), (4, 4, 5, "bf16"), (4, 5, 9, "bf16"), (8, 4, 1, "bf16"), (8, 5, 9, "bf16"),
         (4, 4, 1, "f32")]
KINDS = [sink(0.0, 1.0), sink(0.0, 0.05), sink(0.0, 1e-3), sink(1.0, 0.05), sink(-3.0, 1.0), sink(2.0 ** -10, 1.0),
         every_third(0.0, 0.05), every_third(0.0, 1e-6), every_third(50.0, 1.0), every_third(0.0, 1e4)]


@pytest.mark.parametrize("weight", [0.5, 0.99])
@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_rows_of_equal_values_that_take_much_of_the_weight(bits, G, rows, dtype, weight):
    c = Cache([3001, 700], KINDS, G, rows, 128, 64, bits, dtype, weight, seed=1)
    c.call()
    c.check([0, 1])


@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (64, 64)])
@pytest.mark.parametrize("bits,G,rows", [(4, 4, 1), (4, 4, 5), (8, 4, 1), (8, 5, 9)])
def test_rows_of_equal_values_in_the_other_layouts(D, P, bits, G, rows):
    c = Cache([901, 333], KINDS, G, rows, D, P, bits, "bf16", 0.95, seed=2)
    c.call()
    c.check([0, 1])


@pytest.mark.parametrize("bits,G,rows", [(4, 4, 1), (4, 4, 5), (8, 4, 1)])
def test_units_of_one_cta(bits, G, rows):
    # 160 (sequence, head) units: a CTA's references span whole sequences
    c = Cache([2048] * 16, KINDS, G, rows, 128, 64, bits, "bf16", 0.99, seed=3)
    c.call()
    c.check([0, 15])


@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_caches_of_equal_values_only(bits, G, rows, dtype):
    c = Cache([200, 65], [every_third(0.0, 0.0), every_third(0.75, 0.0)], G, rows, 128, 64, bits, dtype, seed=4)
    c.call()
    c.check([0, 1])
    assert (c.out[:, :, :G].float().abs() < 1e-15).all()


def test_values_with_a_step_of_one():
    # s = 1 with numbers, beside rows of equal values, which are held with s = 1 too: two values a row, 0 and 15 (255)
    def steps(rng, v):
        v = np.where(rng.random(v.shape) < 0.01, 15.0, 0.0)
        v[:, ::2, 5] = 15.0
        v[:, 3::4] = 0.0
        return v
    for bits in (4, 8):
        for G, rows in ((4, 1), (5, 9)):
            c = Cache([515, 64], [steps, lambda rng, v: 17.0 * steps(rng, v)], G, rows, 128, 64, bits, "bf16", 0.9, seed=5)
            c.call()
            c.check([0, 1])


@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_long_sequences_with_a_bound_close_to_the_outputs(bits, G, rows, dtype):
    # split over many CTAs and merged; a part lost or counted twice is far outside this bound
    c = Cache([9001, 4097], [lambda rng, v: v, lambda rng, v: 0.05 * v], G, rows, 128, 64, bits, dtype, seed=6)
    c.call()
    c.check([0, 1])


@pytest.mark.parametrize("bits,G,rows", [(4, 1, 1), (4, 4, 2), (4, 4, 4), (4, 4, 5), (8, 1, 1)])
def test_many_weights_far_below_the_largest(bits, G, rows):
    """524288 positions, the longest sequence, within one CTA (160 units over the same pages): two positions (one in
    either half of the alternate stages) weigh 5 x 2^20 times as much as each other one, which so lies at a fifth of a
    step of the narrow form's weights; together they have 5% of the weight.

    Bound (norms over a head's outputs): the output's rounding 2^-8 |out|; two large weights rounded, 2^-9 sum p |v|; a weight goes up
    or down to a whole step by thresholds that cover a step evenly over 128 positions (64 of either parity, whose
    numbers are met differently): the mean is off by at most half a step in 64 positions, T 2^-27 N max p s_v, and the
    numbers, drawn without regard to the position, vary by at most N / 2 around theirs, against errors of at most half
    a step in the root mean square: six times sqrt(T) 2^-22 N max p s_v; the accumulator, rounded once for
    32 positions (16 in float16) by at most 2^-23 of partial sums of at most (N + 1) sum p s_v; scores as in the
    module docstring, below 1e-3 here."""
    rng = np.random.default_rng(8)
    S, H, D, P, width, pool = 80, 2, 128, 64, 8192, 256
    T, N, scale = width * P, 2 ** bits - 1, 128 ** -0.5
    k = 0.01 * rng.standard_normal((1, pool * P, H, D)).astype(np.float32)
    k[..., 0] = 0
    k[0, 1, :, 0] = np.log(5 * 2.0 ** 20) / (BIAS * scale)                     # page 0, listed twice
    v = rng.choice([-1.0, 1.0], (H, D)) + 0.25 * rng.standard_normal((1, pool * P, H, D))
    q = 0.01 * rng.standard_normal((S, rows, H * G, D)).astype(np.float32)
    q[:] = q[:1]
    q[..., 0] = BIAS
    k, v, q = (torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda() for x in (k, v, q))
    row = 1 + np.arange(width) % (pool - 1)
    row[0] = row[2] = 0                                                        # positions 1 and 129
    table = torch.from_numpy(np.tile(row, (S, 1)).astype(np.int32)).cuda()
    pages = torch.zeros((pool, H, Q.page_bytes(D, P, bits)), dtype=torch.uint8, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
    plain = torch.arange(pool, dtype=torch.int32, device="cuda")[None].contiguous()
    writer = s3r.paged_kvq(pages, plain, lens, H * G, D, P, bits)
    for a in range(0, pool * P, 1024):
        s3r.s3r_kvq_append(writer, lens, k[:, a:a + 1024].contiguous(), v[:, a:a + 1024].contiguous(), "bf16", 1024, 0, ws)
    full = torch.full((S,), T, dtype=torch.int32, device="cuda")
    kvq = s3r.paged_kvq(pages, table, full, H * G, D, P, bits)
    wa = torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(kvq, "bf16", rows), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((S, rows, H * G), device="cuda")
    s3r.s3r_kvq_attn(kvq, q, "bf16", rows, scale, out, lse, wa)
    assert s3r.s3r_device_status(ws) == (0, 0) and s3r.s3r_device_status(wa) == (0, 0)
    held = Q.held_rows(pages.cpu().numpy(), np.arange(pool), pool * P, D, P, bits)
    times = np.repeat(np.bincount(row, minlength=pool), P).astype(np.float64)
    for b in (0, S - 1):
        for h in range(H):
            for r in range(rows):
                for g in range(G):
                    y = held["k"][:, h] @ q[b, r, h * G + g].double().cpu().numpy() * scale
                    p = np.exp(y - y.max())
                    # the last page, listed 32 times or more, ends the sequence: its last positions are hidden from the first rows
                    n = times.copy()
                    if r < rows - 1:
                        n[row[-1] * P + P - (rows - 1 - r):row[-1] * P + P] -= 1
                    w = n * p / (n * p).sum()
                    one = p / (n * p).sum()
                    ref, A = w @ held["v"][:, h], w @ np.abs(held["v"][:, h])
                    top, B = (one * held["sv"][:, h]).max(), w @ held["sv"][:, h]
                    tol = 2.0 ** -8 * np.abs(ref) + 1e-3 * A
                    if bits == 4 and G * rows <= 16:
                        tol = tol + 2.0 ** -9 * A + N * top * (T * 2.0 ** -27 + 6 * T ** 0.5 * 2.0 ** -22)
                    else:
                        tol = tol + (N / 2 + 1) * (2.0 ** -12 * B + 2.0 ** -33 * T * top)
                    tol = tol + T / (32 if bits == 4 and G * rows <= 16 else 16) * 2.0 ** -23 * (N + 1) * B
                    err = np.linalg.norm(out[b, r, h * G + g].double().cpu().numpy() - ref)
                    assert err <= np.linalg.norm(tol), (b, h, r, g, err / np.linalg.norm(ref), np.linalg.norm(tol) / np.linalg.norm(ref))


@pytest.mark.parametrize("bits,G,rows", [(4, 2, 2), (8, 5, 9)])
def test_unusable_lengths_among_many_sequences(bits, G, rows):
    # the first, the last and some between; more sequences than the kernel has threads
    c = Cache([40] * 700, [lambda rng, v: v], G, rows, 64, 16, bits, "bf16", seed=9)
    c.call()
    ref, lse = c.out.clone(), c.lse.clone()
    assert s3r.s3r_device_status(c.ws) == (0, 0)
    bad = [0, 1, 31, 32, 350, 607, 608, 699]
    c.dlens[bad] = torch.tensor([0, -1, rows - 1, 2 ** 31 - 1, -2 ** 31, 49, rows - 1, 0], dtype=torch.int32, device="cuda")
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.call()
    ref[bad], lse[bad] = 0.0, -float("inf")
    assert torch.equal(c.out, ref) and torch.equal(c.lse, lse)
    assert s3r.s3r_device_status(c.ws)[1] == s3r.S3R_DEV_BAD_CONTEXT_LEN
    c.dlens.zero_()                                                            # no sequence has any page
    c.call()
    assert (c.out == 0).all() and (c.lse == -float("inf")).all()


@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_a_float32_row_below_bf16_is_a_nan_row(bits, G, rows, dtype):
    # its minimum rounds down to -inf: it reads back as NaN, and the rows that see it give NaN
    c = Cache([130, 70], [lambda rng, v: v], G, rows, 128, 64, bits, dtype, seed=10)
    c.call()
    ref = c.out.clone()
    x = torch.ones((2, 1, 1, 128), device="cuda")
    x[1, 0, 0, 3] = -3.4e38
    ws = torch.zeros(s3r.s3r_kv_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    s3r.s3r_kvq_append(c.kvq, None, x, x, "f32", 1, 1, ws)                     # over the last position
    out, val = torch.zeros_like(x), torch.zeros_like(x)
    s3r.s3r_kvq_read(c.kvq, c.dlens - 1, 1, "f32", out, val, ws)
    assert torch.equal(out[0], x[0]) and torch.equal(val[0], x[0]) and out[1].isnan().all() and val[1].isnan().all()
    c.call()
    assert c.out[1, rows - 1].isnan().all() and torch.equal(c.out[1, :rows - 1], ref[1, :rows - 1])
    assert torch.isfinite(c.out[0]).all()
    assert s3r.s3r_device_status(ws) == (0, 0) and s3r.s3r_device_status(c.ws) == (0, 0)


@pytest.mark.parametrize("D,P", [(128, 64), (64, 16)])
@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_keys_of_equal_values_among_small_ones(bits, G, rows, dtype, D, P):
    # every third key is zero or constant; the others a thousandth of usual, queries a thousand times: scores of size 1.
    # A key without numbers scores scale z sum q, whatever step it is held with.
    c = Cache([515, 130], [lambda rng, v: v] * 2, G, rows, D, P, bits, dtype, seed=11)
    rng = np.random.default_rng(12)
    k = 1e-3 * rng.standard_normal((2, 515, 2, D)).astype(np.float32)
    k[:, ::3] = 0.0
    k[:, 1::6] = 2.0 ** -12
    k, v = (torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda() for x in (k, rng.standard_normal((2, 515, 2, D)) + 1.0))
    lens = torch.full((2,), 515, dtype=torch.int32, device="cuda")
    writer = s3r.paged_kvq(c.pages, torch.from_numpy(c.table).cuda(), lens, 2 * G, D, P, bits)
    ws = torch.zeros(s3r.s3r_kv_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    s3r.s3r_kvq_append(writer, None, k, v, dtype, 515, 515, ws)
    c.q = (1e3 * torch.from_numpy(rng.standard_normal(c.q.shape).astype(np.float32)).cuda()).to(DT[dtype])
    c.call()
    assert s3r.s3r_device_status(ws) == (0, 0) and s3r.s3r_device_status(c.ws) == (0, 0)
    raw = c.pages.cpu().numpy()
    for b in range(2):
        held = Q.held_rows(raw, c.table[b], c.lens[b], D, P, bits)
        pages = [[Q.read_page(raw[i, h], D, P, bits) for h in range(2)] for i in c.table[b, :-(-c.lens[b] // P)]]
        n_k, n_v = (np.concatenate([np.stack([x[j] for x in heads], 1) for heads in pages])[:c.lens[b]] for j in (0, 3))
        ref, lse, tol = bounded(c.q[b].float().cpu().numpy(), held, n_v, c.scale, rows, bits, dtype, n_k)
        out = c.out[b].double().cpu().numpy()
        assert (np.abs(out - ref) <= tol).all(), (b, np.abs(out - ref).max(), tol.max())
        assert np.abs(c.lse[b].double().cpu().numpy() - lse).max() < 1e-3      # e' of the docstring: at most 5e-4 here
