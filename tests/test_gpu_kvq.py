"""The quantised cache on the GPU against its float64 oracle: rows stored (new
rows and an existing cache) byte for byte, rows read back exactly, lengths,
and what is left alone; bad lengths and pages; whole runs of the calls."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle.kv_quant as Q                                                     # noqa: E402
from self_sparse_speculative_b200 import s3r                                    # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def cache(S, H, D, P, bits, lens, width, seed, spare=3, fill="random"):
    """A cache with every page of any content: host bytes, table, and the device tensors."""
    rng = np.random.default_rng(seed)
    total = S * width + spare
    pages = (rng.integers(0, 256, (total, H, Q.page_bytes(D, P, bits)), dtype=np.uint8) if fill == "random"
             else np.zeros((total, H, Q.page_bytes(D, P, bits)), dtype=np.uint8))
    table = rng.permutation(total)[:S * width].reshape(S, width).astype(np.int32)
    dev = dict(pages=torch.from_numpy(pages).cuda(), table=torch.from_numpy(table).cuda(),
               lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    dev["kvq"] = s3r.paged_kvq(dev["pages"], dev["table"], dev["lens"], H, D, P, bits)
    dev["ws"] = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
    return pages, table, dev


def rows(shape, dtype, seed):
    """Rows with an offset, outlier channels, equal rows and ties; as device tensor and float32 host copy."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape).astype(np.float32) * np.exp(rng.uniform(-3, 3, shape[:-1] + (1,))).astype(np.float32)
    x += rng.standard_normal(shape[:-1] + (1,)).astype(np.float32)
    x[..., 3] += 8 * rng.standard_normal(shape[:-1]).astype(np.float32)
    x.reshape(-1, shape[-1])[::11] = 0.75                                      # equal values
    x.reshape(-1, shape[-1])[1::11] = rng.integers(0, 31, shape[-1]) / 2.0     # many exact ties at 4 bits
    t = torch.from_numpy(x).to(DT[dtype]).cuda()
    return t, t.float().cpu().numpy()


def ok(dev):
    assert s3r.s3r_device_status(dev["ws"]) == (s3r.S3R_OK, 0)


SHAPES = [(64, 16, 4), (64, 16, 8), (64, 64, 4), (64, 64, 8), (128, 16, 4), (128, 16, 8), (128, 64, 4), (128, 64, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,P,bits", SHAPES)
def test_append_writes_the_oracles_bytes(D, P, bits, dtype):
    # one row; a few across a page; across several pages; overwriting; nothing but a shorter length
    S, H, width = 4, 3, 6
    lens = [0, P - 1, P + 3, 2 * P]
    pages, table, dev = cache(S, H, D, P, bits, lens, width, seed=D + P + bits)
    host = list(lens)
    for i, (n, over) in enumerate([(1, 0), (5, 1), (P + 7, 3), (1, 1), (0, 2), (17, 0), (2 * P, P)]):
        k, kh = rows((S, max(n, 1), H, D), dtype, seed=10 * i)
        v, vh = rows((S, max(n, 1), H, D), dtype, seed=10 * i + 1)
        k, v, kh, vh = k[:, :n].contiguous(), v[:, :n].contiguous(), kh[:, :n], vh[:, :n]
        s3r.s3r_kvq_append(dev["kvq"], dev["lens"], k if n else None, v if n else None, dtype, n, over, dev["ws"])
        Q.append(pages, table, host, kh, vh, bits, P, over)
        assert dev["lens"].tolist() == host, (n, over)
        assert np.array_equal(dev["pages"].cpu().numpy(), pages), (n, over)    # unwritten positions and pages too
    ok(dev)


def test_append_without_lengths_leaves_them():
    D, P, bits, S, H = 128, 64, 4, 3, 2
    lens = [5, 64, 100]
    pages, table, dev = cache(S, H, D, P, bits, lens, 3, seed=5)
    k, kh = rows((S, 4, H, D), "bf16", 1)
    s3r.s3r_kvq_append(dev["kvq"], None, k, k, "bf16", 4, 0, dev["ws"])
    Q.append(pages, table, list(lens), kh, kh, bits, P, 0)
    assert dev["lens"].tolist() == lens and np.array_equal(dev["pages"].cpu().numpy(), pages)
    ok(dev)


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_at_the_edges_of_the_arithmetic(bits):
    # each row alone in the type float32: values next to rounding borders of n and of the bf16 parameters,
    # ranges that overflow float32, tiny and subnormal ranges, -0, NaN and infinities
    D, P, H = 64, 64, 1
    rng = np.random.default_rng(7)
    top = 2 ** bits - 1
    xs = []
    for i in range(200):
        s = Q.bf16_value(Q.bf16_nearest(np.float32(np.exp(rng.uniform(-8, 8)))))
        z = np.float32(rng.standard_normal())
        n = rng.integers(0, top, D)
        x = (z + s * (n + 0.5)).astype(np.float32)                             # borders, then steps around them
        x = np.nextafter(x, np.where(rng.random(D) < 0.5, np.inf, -np.inf).astype(np.float32)) if i % 3 else x
        x[0], x[1] = z, z + s * top
        xs.append(x.astype(np.float32))
    for i in range(100):                                                       # (max - z) / top next to a bf16 midpoint
        m = np.float32(1.0 + (2 * rng.integers(0, 128) + 1) / 256.0) * np.float32(2.0 ** int(rng.integers(-20, 20)))
        hi = np.float32(m * top)
        for _ in range(int(rng.integers(0, 4))):
            hi = np.nextafter(hi, np.float32(np.inf if i % 2 else 0))
        x = rng.uniform(0, 1, D).astype(np.float32) * hi
        x[0], x[1] = 0, hi
        xs.append(x)
    big = np.float32(3.3e38)
    xs += [np.where(np.arange(D) % 2, big, -big).astype(np.float32), np.linspace(-3e38, 3e38, D).astype(np.float32),
           np.linspace(0, 1e-44, D).astype(np.float32), np.linspace(-1e-31, 1e-29, D).astype(np.float32),
           np.linspace(0, 15 * 2.0 ** -100, D).astype(np.float32), np.linspace(0, 14.9 * 2.0 ** -100, D).astype(np.float32),
           np.linspace(0, 255 * 2.0 ** -100, D).astype(np.float32),
           np.full(D, -0.0, dtype=np.float32), np.full(D, 1 + 2.0 ** -20, dtype=np.float32),
           np.where(np.arange(D) == 9, np.nan, 1.0).astype(np.float32),
           np.where(np.arange(D) == 63, np.inf, 1.0).astype(np.float32),
           np.where(np.arange(D) == 0, -np.inf, 1.0).astype(np.float32), np.full(D, np.nan, dtype=np.float32)]
    x = np.stack(xs)
    n = len(x)
    width = -(-n // P)
    pages, table, dev = cache(1, H, D, P, bits, [0], width, seed=9)
    k = torch.from_numpy(x.reshape(1, n, H, D)).cuda()
    s3r.s3r_kvq_append(dev["kvq"], dev["lens"], k, k, "f32", n, 0, dev["ws"])
    Q.append(pages, table, [0], x.reshape(1, n, H, D), x.reshape(1, n, H, D), bits, P, 0)
    got = dev["pages"].cpu().numpy()
    for t in range(n):                                                         # row by row, so that a failure names it
        a = Q.read_page(got[table[0, t // P], 0], D, P, bits)
        b = Q.read_page(pages[table[0, t // P], 0], D, P, bits)
        for i in range(6):
            assert np.array_equal(a[i][t % P], b[i][t % P], equal_nan=True), (t, i, x[t][:4])
    out = torch.zeros((1, n, H, D), device="cuda")
    out2 = torch.zeros_like(out)
    s3r.s3r_kvq_read(dev["kvq"], None, n, "f32", out, out2, dev["ws"])
    held = Q.held_rows(pages, table[0], n, D, P, bits)
    ref = held["k"].astype(np.float32)                                         # one rounding of s n + z
    with np.errstate(over="ignore"):
        assert np.array_equal(out[0].cpu().numpy(), ref, equal_nan=True)
    assert np.array_equal(out2[0].cpu().numpy(), ref, equal_nan=True)
    assert np.isnan(ref[-4:]).all()
    ok(dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,P,bits", SHAPES)
def test_pack_then_read(D, P, bits, dtype):
    S, H, width = 5, 2, 4
    lens = [1, P - 1, P, 2 * P + 5, 4 * P]
    pages, table, dev = cache(S, H, D, P, bits, lens, width, seed=3)
    n_src = S * width + 1
    kc, kh = rows((n_src, H, P, D), dtype, 1)
    vc, vh = rows((n_src, H, P, D), dtype, 2)
    src = np.random.default_rng(4).permutation(n_src)[:S * width].reshape(S, width).astype(np.int32)
    src_t = torch.from_numpy(src).cuda()
    kv = s3r.paged_kv(kc, vc, src_t, dev["lens"], H)
    junk = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    kvq = s3r.paged_kvq(dev["pages"], dev["table"], junk, H, D, P, bits)        # its own lengths are not read
    for last in (0, 3, P + 9, 10 ** 6):
        k2 = kc + 1 if last == 3 else kc
        kv = s3r.paged_kv(k2, vc, src_t, dev["lens"], H)
        s3r.s3r_kvq_pack(kv, kvq, last, dev["ws"])
        kk = k2.float().cpu().numpy()
        for b in range(S):
            for pos in range(max(0, lens[b] - last) if last else 0, lens[b]):
                for h in range(H):
                    Q.write_row(pages[table[b, pos // P], h], D, P, bits, pos % P, kk[src[b, pos // P], h, pos % P],
                                vh[src[b, pos // P], h, pos % P])
        assert np.array_equal(dev["pages"].cpu().numpy(), pages), last
    # read back: windows before, inside and past the sequences; rows of no position stay as they were
    for start, n in ((None, 4 * P), ([0, 3, P, P + 1, 4 * P - 2], 7), ([5, P - 1, 0, 2 * P + 4, 3 * P + 15], P + 3),
                     ([0, 0, 0, 0, 0], 1), ([2 ** 31 - 1, 2 ** 31 - 5, 1, 0, 0], 2 ** 12)):
        st = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
        ko = torch.full((S, n, H, D), -5.0, dtype=DT[dtype], device="cuda")
        vo = torch.full((S, n, H, D), -6.0, dtype=DT[dtype], device="cuda")
        s3r.s3r_kvq_read(dev["kvq"], st, n, dtype, ko, vo, dev["ws"])
        for b in range(S):
            held = Q.held_rows(pages, table[b], lens[b], D, P, bits)
            a = 0 if start is None else start[b]
            m = max(0, min(n, lens[b] - a))
            for out, x, left in ((ko, "k", -5.0), (vo, "v", -6.0)):
                ref = torch.from_numpy(held[x][a:a + m].astype(np.float32)).to(DT[dtype])
                assert torch.equal(out[b, :m].cpu(), ref), (start, b, x)
                assert (out[b, m:] == left).all(), (start, b, x)
    ok(dev)


def test_bad_lengths_and_pages_are_flagged_and_nothing_else_is_touched():
    D, P, bits, S, H = 64, 16, 4, 6, 2
    lens = [20, 30, 0, 48, 2, -3]
    pages, table, dev = cache(S, H, D, P, bits, lens, 3, seed=11)
    table[0, 1], table[1, 1] = -1, 10 ** 6
    dev["table"].copy_(torch.from_numpy(table))
    k, kh = rows((S, 4, H, D), "bf16", 1)
    # 0, 1: the second page is bad; 2: overwrite > L; 3: would pass 3 pages; 4: fine; 5: negative length
    s3r.s3r_kvq_append(dev["kvq"], dev["lens"], k, k, "bf16", 4, 2, dev["ws"])
    for h in range(H):
        for t in range(4):
            Q.write_row(pages[table[4, 0], h], D, P, bits, t, kh[4, t, h], kh[4, t, h])
    assert np.array_equal(dev["pages"].cpu().numpy(), pages)
    assert dev["lens"].tolist() == [22, 32, 0, 48, 4, -3]
    st, bits_ = s3r.s3r_device_status(dev["ws"])
    assert st == s3r.S3R_ERR_DEVICE_CHECK and bits_ == s3r.S3R_DEV_BAD_CONTEXT_LEN | s3r.S3R_DEV_BAD_PAGE_ID
    out = torch.full((S, 40, H, D), 9.0, device="cuda")
    out2 = out.clone()
    start = torch.tensor([0, 0, 0, 0, -1, 0], dtype=torch.int32, device="cuda")
    s3r.s3r_kvq_read(dev["kvq"], start, 40, "f32", out, out2, dev["ws"])
    assert (out[[2, 4, 5]] == 9.0).all() and (out[0, 16:] == 9.0).all() and (out[3] != 9.0).any(-1).all()
    assert s3r.s3r_device_status(dev["ws"])[1] == s3r.S3R_DEV_BAD_CONTEXT_LEN | s3r.S3R_DEV_BAD_PAGE_ID
    ok(dev)                                                                    # read clears the word
    dev["lens"].copy_(torch.tensor([5, 5, 5, 5, 0, 49], dtype=torch.int32))
    acc = torch.tensor([0, 3, 4, -1, 0, 0], dtype=torch.int32, device="cuda")
    s3r.s3r_kvq_rollback(dev["kvq"], dev["lens"], acc, 4, dev["ws"])
    assert dev["lens"].tolist() == [2, 5, 5, 5, 0, 49]
    assert s3r.s3r_device_status(dev["ws"])[1] == s3r.S3R_DEV_BAD_CONTEXT_LEN
    # pack from a cache whose table or lengths are bad
    kc, kh = rows((4, H, P, D), "f32", 2)
    src = torch.tensor([[0, 1, 2], [9, 1, 2], [0, 1, 2], [0, 1, 2], [0, 1, -1], [3, 3, 3]], dtype=torch.int32, device="cuda")
    dev["lens"].copy_(torch.tensor([0, 17, 49, -1, 33, 16], dtype=torch.int32))
    before = pages.copy()
    s3r.s3r_kvq_pack(s3r.paged_kv(kc, kc, src, dev["lens"], H), dev["kvq"], 0, dev["ws"])
    for b, p, i in ((4, 0, 0), (4, 1, 1), (5, 0, 3)):
        for h in range(H):
            for t in range(P):
                Q.write_row(before[table[b, p], h], D, P, bits, t, kh[i, h, t], kh[i, h, t])
    assert np.array_equal(dev["pages"].cpu().numpy(), before)
    assert s3r.s3r_device_status(dev["ws"])[1] == s3r.S3R_DEV_BAD_CONTEXT_LEN | s3r.S3R_DEV_BAD_PAGE_ID


@pytest.mark.parametrize("bits", [4, 8])
def test_bf16_values_far_apart_in_size(bits):
    # bf16 rows whose differences x - z are not exact in float32 (tiny x beside a large minimum, a tiny minimum
    # beside large x), next to and on rounding borders of the large part
    D, P, H = 64, 64, 1
    rng = np.random.default_rng(3)
    xs = []
    for i in range(256):
        top = 2 ** bits - 1
        s = Q.bf16_value(Q.bf16_nearest(np.float32(np.exp(rng.uniform(-3, 3)))))
        x = (s * rng.integers(0, 2 * top + 1, D) / 2).astype(np.float32)       # halves of steps: ties
        x[0], x[1] = 0, s * top
        tiny = (rng.choice([-1, 1], D) * np.exp(rng.uniform(-30, -8, D))).astype(np.float32)
        if i % 3 == 0:
            x = x - np.float32(s * (rng.integers(0, top) + 0.5))               # a border at zero: tiny values beside it
            x[2:12] = tiny[2:12]
        elif i % 3 == 1:
            x[0] = abs(tiny[0]) if i % 2 else -abs(tiny[0])                    # a tiny minimum
        xs.append(x)
    x = Q.bf16_value(Q.bf16_nearest(np.stack(xs))).astype(np.float32)
    n = len(x)
    width = n // P
    pages, table, dev = cache(1, H, D, P, bits, [0], width, seed=2)
    k = torch.from_numpy(x.reshape(1, n, H, D)).to(torch.bfloat16).cuda()
    s3r.s3r_kvq_append(dev["kvq"], dev["lens"], k, k, "bf16", n, 0, dev["ws"])
    Q.append(pages, table, [0], x.reshape(1, n, H, D), x.reshape(1, n, H, D), bits, P, 0)
    assert np.array_equal(dev["pages"].cpu().numpy(), pages)
    ok(dev)


def test_rollback_of_the_lowest_length_is_refused():
    lens = [-2 ** 31, -2 ** 31 + 2, 1, 7]
    _, _, dev = cache(4, 1, 64, 16, 4, lens, 1, seed=3)
    acc = torch.tensor([0, 0, 3, 0], dtype=torch.int32, device="cuda")
    s3r.s3r_kvq_rollback(dev["kvq"], dev["lens"], acc, 4, dev["ws"])
    assert dev["lens"].tolist() == [-2 ** 31, -2 ** 31 + 2, 1, 4]
    assert s3r.s3r_device_status(dev["ws"])[1] == s3r.S3R_DEV_BAD_CONTEXT_LEN
