"""Calls of the quantised cache right behind one another, where each reads what the one before it wrote: rows just
stored, lengths just moved, pages just listed. Without a synchronisation, and captured, they give what they give
one at a time."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from self_sparse_speculative_b200 import s3r                                    # noqa: E402


class Chain:
    """Single rows stored and attended to, rows stored over them, verified, and rolled back."""

    def __init__(self, bits, dtype, G, S=6, H=2, D=128, P=64, steps=24):
        rng = np.random.default_rng(bits)
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dt).cuda()  # noqa: E731
        self.dtype, self.steps, self.S, width = dtype, steps, S, 6
        self.pages = torch.zeros((S * width, H, s3r.s3r_kvq_page_bytes(D, P, bits)), dtype=torch.uint8, device="cuda")
        self.table = torch.from_numpy(rng.permutation(S * width).reshape(S, width).astype(np.int32)).cuda()
        self.start = torch.tensor([1, 62, 63, 64, 127, 200][:S], dtype=torch.int32, device="cuda")
        self.lens = self.start.clone()
        self.kvq = s3r.paged_kvq(self.pages, self.table, self.lens, H * G, D, P, bits)
        self.ws = torch.zeros(s3r.s3r_kv_workspace_bytes(S), dtype=torch.uint8, device="cuda")
        self.wa = [torch.zeros(s3r.s3r_kvq_attn_workspace_bytes(self.kvq, dtype, r), dtype=torch.uint8, device="cuda")
                   for r in (1, 3)]
        self.first = [new(S, 256, H, D) for _ in range(2)]
        self.rows = [[new(S, n, H, D) for _ in range(2)] for _ in range(steps) for n in (1, 3)]
        self.q = [new(S, n, H * G, D) * 4 for _ in range(steps) for n in (1, 3)]
        self.acc = [torch.from_numpy(rng.integers(0, 3, S).astype(np.int32)).cuda() for _ in range(steps)]
        self.outs = [torch.zeros_like(x) for x in self.q]
        self.lse = [torch.zeros(x.shape[:3], device="cuda") for x in self.q]

    def run(self, between):
        self.lens.zero_()
        between()
        s3r.s3r_kvq_append(self.kvq, self.lens, *self.first, self.dtype, 256, 0, self.ws)
        self.lens.copy_(self.start)
        for i in range(self.steps):
            between()
            s3r.s3r_kvq_append(self.kvq, self.lens, *self.rows[2 * i], self.dtype, 1, 0, self.ws)
            between()
            s3r.s3r_kvq_attn(self.kvq, self.q[2 * i], self.dtype, 1, 0.2, self.outs[2 * i], self.lse[2 * i], self.wa[0])
            between()
            s3r.s3r_kvq_append(self.kvq, self.lens, *self.rows[2 * i + 1], self.dtype, 3, 1, self.ws)
            between()
            s3r.s3r_kvq_attn(self.kvq, self.q[2 * i + 1], self.dtype, 3, 0.2, self.outs[2 * i + 1], self.lse[2 * i + 1],
                             self.wa[1])
            between()
            s3r.s3r_kvq_rollback(self.kvq, self.lens, self.acc[i], 3, self.ws)
        between()

    def clear(self):
        for x in self.outs + self.lse:
            x.fill_(9.0)
        self.pages.zero_()
        torch.cuda.synchronize()

    def held(self):
        torch.cuda.synchronize()
        return [x.clone() for x in self.outs + self.lse + [self.pages, self.lens]]


@pytest.mark.parametrize("bits,dtype,G", [(4, "bf16", 4), (4, "bf16", 8), (8, "bf16", 4), (4, "f32", 2)])
def test_calls_behind_one_another(bits, dtype, G):
    c = Chain(bits, dtype, G)
    c.clear()
    c.run(torch.cuda.synchronize)
    want = c.held()
    assert all(torch.isfinite(x.float()).all() for x in want)
    for _ in range(4):
        c.clear()
        c.run(lambda: None)
        assert all(torch.equal(x, y) for x, y in zip(c.held(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(lambda: None)
    for _ in range(4):
        c.clear()
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(c.held(), want))
    assert all(s3r.s3r_device_status(w) == (0, 0) for w in [c.ws] + c.wa)


def test_calls_at_once_on_several_streams():
    # chains over caches and workspaces of their own, on streams of their own at the same time
    forms = [(4, "bf16", 4), (8, "bf16", 4), (4, "bf16", 8), (4, "f32", 2)]
    chains = [Chain(*f) for f in forms]
    want = []
    for c in chains:
        c.clear()
        c.run(lambda: None)
        want.append(c.held())
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(3):
        for c in chains:
            c.clear()
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.run(lambda: None)
        torch.cuda.synchronize()
        for c, w in zip(chains, want):
            assert all(torch.equal(x, y) for x, y in zip(c.held(), w))
    assert all(s3r.s3r_device_status(w) == (0, 0) for c in chains for w in [c.ws] + c.wa)
