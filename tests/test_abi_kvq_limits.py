"""Further refusals of the quantised cache's calls, on the host before any CUDA call (these run without a GPU)."""
import ctypes

import pytest
import torch

from self_sparse_speculative_b200 import s3r

FAKE = 0x10000   # a 16-byte-aligned non-null address; never dereferenced on these paths
ARG, WS = s3r.S3R_ERR_INVALID_ARG, s3r.S3R_ERR_WORKSPACE


def _kvq(**kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=64, max_pages_per_seq=4,
             num_pages_total=8, bits=4, pages=FAKE, block_table=FAKE, context_lens=FAKE)
    d.update(kw)
    c = s3r.PagedKVQ()
    for k, v in d.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("scale", [2.0 ** 112, -2.0 ** 112, 3e38, float("nan"), float("inf")])
def test_scales_that_leave_float32_are_refused(scale):
    st = s3r.lib().s3r_kvq_attn(ctypes.byref(_kvq()), FAKE, s3r.S3R_BF16, 1, None, 0, scale, FAKE, None, FAKE, 1 << 40, None)
    assert st == ARG


def test_packing_refuses_a_source_of_another_device():
    k = torch.zeros((8, 2, 64, 128), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    kv = s3r.paged_kv(k, k, table, lens, 8)
    assert kv.devices == {-1}
    kvq, ws = _kvq(), FAKE
    for at, name in (({0, 5}, "cuda:5"), ({0, -1}, "the host")):
        kv.devices = at
        current = s3r._kvq_env
        s3r._kvq_env = lambda dtype: (0, None, None)                           # a process whose current device is cuda:0
        try:
            with pytest.raises(ValueError, match=f"source cache lives on {name}"):
                s3r.s3r_kvq_pack(kv, kvq, 0, ws, workspace_bytes=4096, stream=0)
        finally:
            s3r._kvq_env = current


def test_workspaces_off_their_alignment_are_refused():
    lib, c, big, bf = s3r.lib(), _kvq(), 1 << 40, s3r.S3R_BF16
    r, kv = ctypes.byref(c), s3r.PagedKV(2, 8, 2, 128, 64, 4, 8, bf, FAKE, FAKE, FAKE, FAKE)
    for off in (1, 4, 8):                                                      # partial outputs are read 16 bytes at a time
        assert lib.s3r_kvq_attn(r, FAKE, bf, 1, None, 0, 0.1, FAKE, None, FAKE + off, big, None) == WS
    for off in (1, 2, 3):                                                      # counters of 4 bytes
        assert lib.s3r_kvq_append(r, FAKE, FAKE, FAKE, bf, 1, 0, FAKE + off, big, None) == WS
        assert lib.s3r_kvq_pack(ctypes.byref(kv), r, 0, FAKE + off, big, None) == WS
        assert lib.s3r_kvq_read(r, None, 1, bf, FAKE, FAKE, FAKE + off, big, None) == WS
        assert lib.s3r_kvq_rollback(r, FAKE, FAKE, 3, FAKE + off, big, None) == WS


def test_a_first_value_below_bf16_reads_as_nan():
    # the definition's own rows: z rounds down to -inf, s = inf
    import numpy as np
    import oracle.kv_quant as Q
    x = np.array([-3.4e38] + [0.0] * 63, dtype=np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        n, s, z = Q.quantise_rows(x, 4)
        assert Q.bf16_value(z) == -np.inf and Q.bf16_value(s) == np.inf
        assert np.isnan(Q.bf16_value(s) * 0.0 + Q.bf16_value(z))
