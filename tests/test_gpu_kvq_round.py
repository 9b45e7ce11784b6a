"""A round whose drafts attend over the quantised copy of the cache, through
DecodeStep: the copy's bytes, the drafts' outputs, and everything else as in a
round with the cache kept. Also captured and replayed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle.kv_quant as Q                                                     # noqa: E402
from self_sparse_speculative_b200 import s3r                                    # noqa: E402
from self_sparse_speculative_b200.step import DecodeStep                        # noqa: E402
from self_sparse_speculative_b200.workloads import Workload, custom_spec        # noqa: E402

CASES = {
    "bf16-b4": (custom_spec(1, num_seqs=3, num_q_heads=8, num_kv_heads=2, budget_pages=3, vocab=2000), [70, 129, 260], 4),
    "bf16-p16-b8": (custom_spec(1, num_seqs=2, num_q_heads=8, num_kv_heads=2, page_size=16, budget_pages=3, vocab=2000),
                    [33, 100], 8),
    "f32-b4": (custom_spec(0, num_seqs=2, budget_pages=3), [200, 257], 4),
}


@pytest.mark.parametrize("name", list(CASES))
def test_round_with_quantised_drafts(name):
    spec, lens, bits = CASES[name]
    plain = DecodeStep(Workload(spec, seed=4, context_lens=lens))
    plain.context_lens.copy_(plain.lens_committed)
    plain.summaries()
    plain.round_with_kv()
    st = DecodeStep(Workload(spec, seed=4, context_lens=lens), draft_bits=bits)
    st.context_lens.copy_(st.lens_committed)
    st.summaries()
    st.quantise()
    before = st.pages_q.cpu().numpy()
    table, committed = st.block_table.cpu().numpy(), st.lens_committed.tolist()
    st.round_quantised()
    torch.cuda.synchronize()
    for k, (status, flags) in st.device_checks().items():
        assert status == s3r.S3R_OK, (k, flags)
    # verification, sampling, the cache and its lengths do not depend on what drafted
    for x in ("verify_out", "verify_lse", "out_tokens", "num_accepted", "context_lens", "k_cache", "v_cache", "kmin", "kmax"):
        assert torch.equal(getattr(st, x), getattr(plain, x)), x
    # the drafts, step by step, and at the end the verifier's rows, in the copy
    S, Hkv, D, P, g, R = spec.num_seqs, spec.num_kv_heads, spec.head_dim, spec.page_size, spec.gamma, spec.rows
    host, hl = before, list(committed)
    q = st.q_draft.float().cpu().numpy()
    for i in range(g):
        Q.append(host, table, hl, st.k_round_draft[i].float().cpu().numpy(), st.v_round_draft[i].float().cpu().numpy(),
                 bits, P, 0)
        for b in range(S):
            ref, lse, A, B = Q.attend(q[i, b][None], Q.held_rows(host, table[b], hl[b], D, P, bits), float(st.scale), 1)
            out = st.draft_out[i, b].double().cpu().numpy()
            # the weights' and the output's roundings (2^-9 A and half a bf16 step, 2^-8), float32 elsewhere
            tol = (1.01 * (2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -9 * A[0]) + 2.0 ** -10 * A[0] if spec.kv_dtype == "bf16"
                   else 1e-5 * (1 + A[0]))
            assert (np.abs(out - ref[0]) <= tol).all(), (i, b)
            assert np.abs(st.draft_lse[i, b].double().cpu().numpy() - lse[0]).max() < 1e-4
    Q.append(host, table, hl, st.k_round_verify.float().cpu().numpy(), st.v_round_verify.float().cpu().numpy(), bits, P, g)
    assert np.array_equal(st.pages_q.cpu().numpy(), host)
    # the same round captured once and replayed twice
    want = {x: getattr(st, x).clone() for x in ("draft_out", "draft_lse", "verify_out", "out_tokens", "context_lens", "pages_q")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.round_quantised(side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        st.draft_out.zero_()
        st.verify_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in want.items():
            assert torch.equal(getattr(st, x), y), x
