"""Refusals of the quantised cache's calls, on the host before any CUDA call
(so these run without a GPU)."""
import ctypes

import pytest
import torch

from self_sparse_speculative_b200 import s3r

FAKE = 0x10000   # a 16-byte-aligned non-null address; never dereferenced on these paths
ARG, UNS, WS = s3r.S3R_ERR_INVALID_ARG, s3r.S3R_ERR_UNSUPPORTED, s3r.S3R_ERR_WORKSPACE


def _kvq(**kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=64, max_pages_per_seq=4,
             num_pages_total=8, bits=4, pages=FAKE, block_table=FAKE, context_lens=FAKE)
    d.update(kw)
    c = s3r.PagedKVQ()
    for k, v in d.items():
        setattr(c, k, v)
    return c


def _kv(**kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=64, max_pages_per_seq=4,
             num_pages_total=8, dtype=s3r.S3R_BF16, k_cache=FAKE, v_cache=FAKE, block_table=FAKE, context_lens=FAKE)
    d.update(kw)
    kv = s3r.PagedKV()
    for k, v in d.items():
        setattr(kv, k, v)
    return kv


def _calls(c):
    """Status of every call on the cache description c, all other arguments in order."""
    lib, r, big = s3r.lib(), ctypes.byref(c), 1 << 40
    return [lib.s3r_kvq_append(r, c.context_lens, FAKE, FAKE, s3r.S3R_BF16, 1, 0, FAKE, big, None),
            lib.s3r_kvq_pack(ctypes.byref(_kv()), r, 0, FAKE, big, None),
            lib.s3r_kvq_read(r, None, 1, s3r.S3R_BF16, FAKE, FAKE, FAKE, big, None),
            lib.s3r_kvq_rollback(r, c.context_lens, FAKE, 3, FAKE, big, None),
            lib.s3r_kvq_attn(r, FAKE, s3r.S3R_BF16, 1, None, 0, 0.1, FAKE, None, FAKE, big, None)]


@pytest.mark.parametrize("field,value,status", [
    ("num_seqs", 0, ARG), ("num_q_heads", 7, ARG), ("num_kv_heads", 0, ARG), ("max_pages_per_seq", 0, ARG),
    ("num_pages_total", 0, ARG), ("pages", 0, ARG), ("pages", FAKE + 8, ARG), ("block_table", 0, ARG),
    ("context_lens", 0, ARG), ("bits", 5, UNS), ("bits", 0, UNS), ("head_dim", 96, UNS), ("page_size", 32, UNS),
    ("num_q_heads", 32, UNS), ("max_pages_per_seq", 9000, UNS), ("num_pages_total", 1 << 30, UNS),
    ("num_seqs", 70000, UNS),
])
def test_bad_descriptions_are_refused(field, value, status):
    c = _kvq(**{field: value})
    assert _calls(c) == [status] * 5
    assert s3r.lib().s3r_kvq_attn_workspace_bytes(ctypes.byref(c), s3r.S3R_BF16, 1, 0) == 0


def test_page_bytes():
    assert s3r.s3r_kvq_page_bytes(128, 64, 4) == 2 * 4096 + 512
    assert s3r.s3r_kvq_page_bytes(64, 16, 8) == 2 * 1024 + 128
    for bad in ((96, 64, 4), (128, 32, 4), (128, 64, 6)):
        assert s3r.s3r_kvq_page_bytes(*bad) == 0


def test_argument_checks():
    lib, c = s3r.lib(), _kvq()
    r, big, bf = ctypes.byref(c), 1 << 40, s3r.S3R_BF16
    ws = s3r.s3r_kv_workspace_bytes(2)
    app = lambda *a: lib.s3r_kvq_append(r, *a, None)  # noqa: E731
    assert app(FAKE + 64, FAKE, FAKE, bf, 1, 0, FAKE, big) == ARG           # lengths of another cache
    assert app(FAKE, None, FAKE, bf, 1, 0, FAKE, big) == ARG
    assert app(FAKE, FAKE, FAKE + 2, bf, 1, 0, FAKE, big) == ARG
    assert app(FAKE, FAKE, FAKE, 2, 1, 0, FAKE, big) == ARG                 # type
    assert app(FAKE, FAKE, FAKE, bf, -1, 0, FAKE, big) == ARG
    assert app(FAKE, FAKE, FAKE, bf, 1025, 0, FAKE, big) == ARG
    assert app(FAKE, FAKE, FAKE, bf, 1, 1025, FAKE, big) == ARG
    assert app(FAKE, FAKE, FAKE, bf, 1, 0, None, big) == WS
    assert app(FAKE, FAKE, FAKE, bf, 1, 0, FAKE, ws - 1) == WS
    assert app(FAKE, None, None, bf, 0, 0, FAKE, ws) == s3r.S3R_OK          # nothing to do, nothing enqueued
    assert app(None, None, None, bf, 0, 3, FAKE, ws) == s3r.S3R_OK
    for kw in (dict(num_seqs=3), dict(num_kv_heads=1), dict(head_dim=64), dict(page_size=16)):
        assert lib.s3r_kvq_pack(ctypes.byref(_kv(**kw)), r, 0, FAKE, big, None) == ARG, kw
    assert lib.s3r_kvq_pack(ctypes.byref(_kv()), r, -1, FAKE, big, None) == ARG
    assert lib.s3r_kvq_pack(None, r, 0, FAKE, big, None) == ARG
    rd = lambda *a: lib.s3r_kvq_read(r, None, *a, None)  # noqa: E731
    assert rd(-1, bf, FAKE, FAKE, FAKE, big) == ARG
    assert rd(1, bf, None, FAKE, FAKE, big) == ARG
    assert rd(1, bf, FAKE, FAKE + 8, FAKE, big) == ARG
    assert rd(1, 5, FAKE, FAKE, FAKE, big) == ARG
    assert rd(0, bf, None, None, FAKE, big) == s3r.S3R_OK
    assert lib.s3r_kvq_rollback(r, None, FAKE, 3, FAKE, big, None) == ARG
    assert lib.s3r_kvq_rollback(r, FAKE, None, 3, FAKE, big, None) == ARG
    assert lib.s3r_kvq_rollback(r, FAKE, FAKE, 18, FAKE, big, None) == ARG
    assert lib.s3r_kvq_rollback(r, FAKE, FAKE, 0, FAKE, big, None) == ARG
    need = lib.s3r_kvq_attn_workspace_bytes(r, bf, 5, 0)
    assert need > 0
    at = lambda q, dt, rows, lst, B, sc, out, w, wb: lib.s3r_kvq_attn(r, q, dt, rows, lst, B, sc, out, None, w, wb, None)  # noqa: E731
    assert at(None, bf, 5, None, 0, 0.1, FAKE, FAKE, big) == ARG
    assert at(FAKE, bf, 5, None, 0, 0.1, FAKE + 4, FAKE, big) == ARG
    assert at(FAKE, bf, 5, None, 0, float("inf"), FAKE, FAKE, big) == ARG
    assert at(FAKE, 9, 5, None, 0, 0.1, FAKE, FAKE, big) == ARG
    assert at(FAKE, bf, 0, None, 0, 0.1, FAKE, FAKE, big) == ARG
    assert at(FAKE, bf, 18, None, 0, 0.1, FAKE, FAKE, big) == UNS
    assert at(FAKE, bf, 5, FAKE, 0, 0.1, FAKE, FAKE, big) == ARG            # a list without its length
    assert at(FAKE, bf, 5, None, 3, 0.1, FAKE, FAKE, big) == ARG            # a length without its list
    assert at(FAKE, bf, 5, FAKE, 8193, 0.1, FAKE, FAKE, big) == UNS
    assert at(FAKE, bf, 5, FAKE, -1, 0.1, FAKE, FAKE, big) == ARG
    assert at(FAKE, bf, 5, None, 0, 0.1, FAKE, FAKE, need - 1) == WS
    assert at(FAKE, bf, 5, None, 0, 0.1, FAKE, None, need) == WS
    wide = _kvq(num_q_heads=16)                                             # G = 8: 17 rows are 136 packed ones
    assert lib.s3r_kvq_attn_workspace_bytes(ctypes.byref(wide), bf, 16, 0) > 0
    assert lib.s3r_kvq_attn_workspace_bytes(ctypes.byref(wide), bf, 17, 0) == 0
    assert lib.s3r_kvq_attn_workspace_bytes(ctypes.byref(_kvq(num_seqs=1025)), bf, 1, 0) == 0


def test_binding_refuses_tensors_of_other_shapes_and_places():
    pages = torch.zeros((8, 2, s3r.s3r_kvq_page_bytes(128, 64, 4)), dtype=torch.uint8)
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="bytes per head"):
        s3r.paged_kvq(pages, table, lens, 8, 128, 64, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        s3r.paged_kvq(pages, table, lens, 8, 128, 64, 4)
    with pytest.raises(ValueError, match="contiguous"):
        s3r.paged_kvq(pages.transpose(0, 1).contiguous().transpose(0, 1), table, lens, 8, 128, 64, 4)
    c, ws = _kvq(), torch.zeros(4096, dtype=torch.uint8)
    row = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_new"):
        s3r.s3r_kvq_append(c, FAKE, row[:1], row, "bf16", 1, 0, ws, stream=0)
    with pytest.raises(ValueError, match="k_new"):
        s3r.s3r_kvq_append(c, FAKE, row.float(), row, "bf16", 1, 0, ws, stream=0)
    with pytest.raises(ValueError, match="v_out"):
        s3r.s3r_kvq_read(c, None, 1, "bf16", FAKE, row.transpose(1, 2), ws, stream=0)
    with pytest.raises(ValueError, match="pages"):
        s3r.s3r_kvq_attn(c, FAKE, "bf16", 1, 0.1, FAKE, None, ws, pages=torch.zeros((2, 2, 3), dtype=torch.int32),
                         budget_pages=4, stream=0)


class _Elsewhere:
    """A workspace of another device."""
    device = "cuda:5"
    numel = lambda self: 1 << 20           # noqa: E731
    element_size = lambda self: 1          # noqa: E731
    get_device = lambda self: 5            # noqa: E731
    data_ptr = lambda self: FAKE           # noqa: E731


@pytest.mark.parametrize("what", ["cache", "workspace"])
def test_binding_refuses_a_cache_or_workspace_of_another_device(what):
    c, ws, match = _kvq(), torch.zeros(4096, dtype=torch.uint8), "quantised cache lives on cuda:5"
    if what == "cache":
        c.device = 5
    else:
        ws, match = _Elsewhere(), "workspace lives on cuda:5"
    calls = [lambda: s3r.s3r_kvq_append(c, FAKE, FAKE, FAKE, "bf16", 1, 0, ws, stream=0),
             lambda: s3r.s3r_kvq_pack(_kv(), c, 0, ws, stream=0),
             lambda: s3r.s3r_kvq_read(c, None, 1, "bf16", FAKE, FAKE, ws, stream=0),
             lambda: s3r.s3r_kvq_rollback(c, FAKE, FAKE, 1, ws, stream=0),
             lambda: s3r.s3r_kvq_attn(c, FAKE, "bf16", 1, 0.1, FAKE, None, ws, stream=0)]
    for call in calls:
        with pytest.raises(ValueError, match=match):
            call()
