"""Queries of the quantised attention that are not finite, very large or very small."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from self_sparse_speculative_b200 import s3r                                    # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FORMS = [(4, 4, 1, "bf16"), (4, 4, 4, "bf16"), (4, 4, 5, "bf16"), (4, 5, 9, "bf16"), (8, 4, 1, "bf16"), (8, 5, 9, "bf16"),
         (4, 4, 2, "f32"), (8, 4, 2, "f32")]


def setup(bits, G, rows, dtype, lens=(700, 130), H=2, D=128, P=64, seed=0):
    rng = np.random.default_rng(seed)
    S, width = len(lens), -(-max(lens) // P)
    pages = torch.zeros((S * width, H, s3r.s3r_kvq_page_bytes(D, P, bits)), dtype=torch.uint8, device="cuda")
    table = torch.from_numpy(rng.permutation(S * width).reshape(S, width).astype(np.int32)).cuda()
    dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kvq = s3r.paged_kvq(pages, table, dlens, H * G, D, P, bits)
    ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
    full = torch.full((S,), width * P, dtype=torch.int32, device="cuda")
    k, v = (torch.from_numpy(rng.standard_normal((S * width, H, P, D)).astype(np.float32)).cuda() for _ in range(2))
    k[..., 5] = -k[..., 5].abs() - 0.5                       # channel 5: every key below 0
    s3r.s3r_kvq_pack(s3r.paged_kv(k, v, table, full, H * G), kvq, 0, ws)
    q = torch.from_numpy(rng.standard_normal((S, rows, H * G, D)).astype(np.float32)).to(DT[dtype]).cuda()
    wa = torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(kvq, dtype, rows), dtype=torch.uint8, device="cuda")
    assert s3r.s3r_device_status(ws) == (0, 0)

    def call(q, scale=D ** -0.5):
        out, lse = torch.full_like(q, 7.0), torch.full((S, rows, H * G), 7.0, device="cuda")
        s3r.s3r_kvq_attn(kvq, q, dtype, rows, scale, out, lse, wa)
        assert s3r.s3r_device_status(wa) == (0, 0)
        return out, lse

    return q, call, (pages, table, dlens)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_a_query_that_is_not_finite_gives_nan(bits, G, rows, dtype, value):
    # channel 17: products of both signs; channel 5: every product is -inf (or +inf)
    q, call, _ = setup(bits, G, rows, dtype)
    out, lse = call(q)
    for channel in (17, 5):
        bad = q.clone()
        at = [(0, rows - 1, G), (1, 0, 1)]
        for x in at:
            bad[x][channel] = value
        o, l = call(bad)
        for x in at:
            assert o[x].isnan().all() and l[x].isnan(), (channel, x, o[x][:4], l[x])
            o[x], l[x] = out[x], lse[x]
        assert torch.equal(o, out) and torch.equal(l, lse)   # no other row changes



@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_a_query_that_is_not_finite_and_sees_nothing(bits, G, rows, dtype):
    # a list without pages for one head: its rows are empty whatever their queries hold
    q, _, (pages, table, lens) = setup(bits, G, rows, dtype)
    S, H, D = 2, 2, 128
    kvq = s3r.paged_kvq(pages, table, lens, H * G, D, 64, bits)
    kept = torch.tensor([[[0], [-1]], [[0], [1]]], dtype=torch.int32, device="cuda")
    wa = torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(kvq, dtype, rows, 1), dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((S, rows, H * G), 7.0, device="cuda")
    q[0] = float("inf")
    s3r.s3r_kvq_attn(kvq, q, dtype, rows, 0.1, out, lse, wa, pages=kept, budget_pages=1)
    assert s3r.s3r_device_status(wa) == (0, 0)
    assert out[0, :, :G].isnan().all() and lse[0, :, :G].isnan().all()
    assert (out[0, :, G:] == 0).all() and (lse[0, :, G:] == -float("inf")).all()
    assert torch.isfinite(out[1]).all()


@pytest.mark.parametrize("shift", [-95, -40, 60, 113, 118, 125])
@pytest.mark.parametrize("bits,G,rows,dtype", [f for f in FORMS if f[3] == "bf16"])
def test_powers_of_two_move_between_query_and_scale(bits, G, rows, dtype, shift):
    # q 2^shift with scale 2^-4 2^-shift (a power of two: exact in float32 down to 2^-149): every product moves by a
    # power of two, so that the same bits come out. The largest queries, 3.5 x 2^125, are near the type's largest number.
    q, call, _ = setup(bits, G, rows, dtype)
    q = q.clamp(-3.5, 3.5)
    out, lse = call(q, 0.0625)
    o, l = call((q.float() * 2.0 ** shift).to(torch.bfloat16), 0.0625 * 2.0 ** -shift)
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("size", [1e2, 1e4, 1e6, 1e8])
@pytest.mark.parametrize("bits,G,rows,dtype", FORMS)
def test_scores_that_float32_cannot_tell_apart(bits, G, rows, dtype, size):
    """Scores up to about 1e10, where float32 is off by whole units: which of nearly equal positions win is open, but an
    output is a weighted mean of held values whatever the weights. It lies between the least and the greatest of its
    channel, up to the roundings of the weights (2^-9 of the largest value for the numbers and as much for the sum) and
    of the output (2^-8)."""
    S, H, D, P, lens = 2, 2, 128, 64, (2363, 517)
    rng = np.random.default_rng(3)
    width = -(-max(lens) // P)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    k = new(S * width, H, P, D) * torch.exp(np.log(size) * torch.from_numpy(rng.random((S * width, H, P, 1)).astype(np.float32)).cuda())
    k += 0.1 * size * new(S * width, H, P, 1)
    v = new(S * width, H, P, D)
    pages = torch.zeros((S * width, H, s3r.s3r_kvq_page_bytes(D, P, bits)), dtype=torch.uint8, device="cuda")
    table = torch.arange(S * width, dtype=torch.int32, device="cuda").reshape(S, width)
    full = torch.full((S,), width * P, dtype=torch.int32, device="cuda")
    dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kvq = s3r.paged_kvq(pages, table, dlens, H * G, D, P, bits)
    ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
    s3r.s3r_kvq_pack(s3r.paged_kv(k, v, table, full, H * G), kvq, 0, ws)
    ko, held = torch.zeros((S, max(lens), H, D), device="cuda"), torch.zeros((S, max(lens), H, D), device="cuda")
    s3r.s3r_kvq_read(kvq, None, max(lens), "f32", ko, held, ws)
    wa = torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(kvq, dtype, rows), dtype=torch.uint8, device="cuda")
    assert s3r.s3r_device_status(ws) == (0, 0)
    for seed in range(8):
        q = (8 * new(S, rows, H * G, D)).to(DT[dtype])
        out, lse = torch.zeros_like(q), torch.zeros((S, rows, H * G), device="cuda")
        s3r.s3r_kvq_attn(kvq, q, dtype, rows, 0.1, out, lse, wa)
        assert s3r.s3r_device_status(wa) == (0, 0)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        for b in range(S):
            x = held[b, :lens[b]].repeat_interleave(G, 1)                      # [L, Hq, D]
            tol = 2.0 ** -7 * x.abs().amax(0)
            assert (out[b] <= x.amax(0) + tol).all() and (out[b] >= x.amin(0) - tol).all()
