"""Pins of the quantised cache's oracle: hand-worked rows, the distance a held
row may have, the byte layout, and attention against PyTorch's float64
attention on the held rows."""
import numpy as np
import pytest
import torch

import oracle.kv_quant as Q


def test_hand_worked_rows():
    # z = -1, s = (2 - -1) / 15 = 0.2 -> bf16 0.2001953125; (x - z) / s
    n, s, z = Q.quantise_rows(np.array([-1.0, 2.0, 0.0, -0.9]), 4)
    assert Q.bf16_value(z) == -1.0 and Q.bf16_value(s) == 0.2001953125
    assert n.tolist() == [0, 15, 5, 0]                       # 0, 14.985, 4.995, 0.4995
    # ties go to the even number: s = 1 exactly
    n, s, z = Q.quantise_rows(np.array([0.0, 15.0, 0.5, 1.5, 2.5, 7.5]), 4)
    assert Q.bf16_value(s) == 1.0 and n.tolist() == [0, 15, 0, 2, 2, 8]
    n, s, z = Q.quantise_rows(np.array([0.0, 255.0, 0.5, 254.5, 253.5]), 8)
    assert Q.bf16_value(s) == 1.0 and n.tolist() == [0, 255, 0, 254, 254]
    # equal values, and rows that are not finite
    n, s, z = Q.quantise_rows(np.full(4, 3.25), 4)
    assert (Q.bf16_value(s), Q.bf16_value(z)) == (1.0, 3.25) and not n.any()
    for bad in (np.nan, np.inf, -np.inf):
        n, s, z = Q.quantise_rows(np.array([0.0, bad]), 8)
        assert np.isnan(Q.bf16_value(z)) and not n.any()
    # the minimum is rounded down to bf16: 1 + 2^-9 -> 1, -(1 + 2^-9) -> -(1 + 2^-7)
    assert Q.bf16_value(Q.bf16_down(np.float32(1 + 2 ** -9))) == 1.0
    assert Q.bf16_value(Q.bf16_down(np.float32(-1 - 2 ** -9))) == -(1 + 2 ** -7)


@pytest.mark.parametrize("bits", [4, 8])
def test_held_rows_are_within_half_a_step(bits):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)).astype(np.float32) * rng.choice([1e-20, 1e-3, 1, 1e10], (200, 1)).astype(np.float32)
    n, s, z = Q.quantise_rows(x, bits)
    s, z = Q.bf16_value(s)[:, None], Q.bf16_value(z)[:, None]
    # half a step; the largest value may lie up to 2^-8 of the range (s rounded down) past the last step
    top = 2 ** bits - 1
    assert (np.abs(s * n + z - x) <= 0.5 * s + top * s * 2.0 ** -8).all()
    assert (z <= x).all() and n.max() == top


@pytest.mark.parametrize("D,P,bits", [(64, 16, 4), (64, 16, 8), (128, 64, 4), (128, 64, 8), (64, 64, 4), (128, 16, 8)])
def test_layout_holds_every_number_once(D, P, bits):
    t, d = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    used = []
    for at in (Q._k_at, Q._v_at):
        byte, shift = at(D, P, bits, t, d)
        used.append((byte * 8 + shift).reshape(-1))
    used = np.concatenate(used)
    assert len(np.unique(used)) == 2 * P * D and used.max() < 8 * Q.page_bytes(D, P, bits)
    rng = np.random.default_rng(1)
    page = rng.integers(0, 256, Q.page_bytes(D, P, bits), dtype=np.uint8)
    k, v = rng.standard_normal((2, P, D)).astype(np.float32)
    for i in rng.permutation(P):
        Q.write_row(page, D, P, bits, i, k[i], v[i])
    nk, sk, zk, nv, sv, zv = Q.read_page(page, D, P, bits)
    for x, (n, s, z) in ((k, (nk, sk, zk)), (v, (nv, sv, zv))):
        m, a, b = Q.quantise_rows(x, bits)
        assert (n == m).all() and (s == Q.bf16_value(a)).all() and (z == Q.bf16_value(b)).all()


def test_attention_is_torch_attention_on_the_held_rows():
    rng = np.random.default_rng(2)
    D, P, bits, H, G, R, L = 64, 16, 4, 2, 3, 4, 41
    pages = np.zeros((3, H, Q.page_bytes(D, P, bits)), dtype=np.uint8)
    table = np.array([[2, 0, 1]])
    lens = np.zeros(1, dtype=np.int64)
    k, v = rng.standard_normal((2, 1, L, H, D)).astype(np.float32)
    Q.append(pages, table, lens, k, v, bits, P, 0)
    assert lens[0] == L
    held = Q.held_rows(pages, table[0], L, D, P, bits)
    q = rng.standard_normal((R, H * G, D))
    out, lse, _, _ = Q.attend(q, held, 0.125, R)
    tk = torch.from_numpy(held["k"]).permute(1, 0, 2).repeat_interleave(G, 0)
    tv = torch.from_numpy(held["v"]).permute(1, 0, 2).repeat_interleave(G, 0)
    mask = torch.arange(L)[None] <= L - R + torch.arange(R)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).permute(1, 0, 2), tk, tv, attn_mask=mask,
                                                           scale=0.125)
    assert np.allclose(out, ref.permute(1, 0, 2).numpy(), atol=1e-12)
    # a list of all pages, each once, is the same attention
    out2, lse2, _, _ = Q.attend(q, held, 0.125, R, [list(range(32, 41)) + list(range(32))] * H)
    assert np.allclose(out, out2, atol=1e-12) and np.allclose(lse, lse2, atol=1e-12)
