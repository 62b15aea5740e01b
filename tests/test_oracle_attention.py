"""Pins of the attention oracle: closed forms, brute force and torch's own double-precision operations."""
import numpy as np
import pytest
import torch

from oracle import attention as oa


def test_slots_worked_example():
    # page 4: request 0 holds 5 tokens (pages 7, 2) and brings 4; request 1 holds none and brings 1; 2 brings none
    table, slots, pos, cu, counts = oa.kv_slots([5, 0, 8], [4, 1, 0], [9, 3, 6], [[7, 2, -1], [-1, -1, -1], [1, 4, -1]], 4,
                                                8, position_base=10)
    assert table.tolist() == [[7, 2, 9], [3, -1, -1], [1, 4, -1]]
    assert slots.tolist() == [9, 10, 11, 36, 12, -1, -1, -1]
    assert pos.tolist() == [15, 16, 17, 18, 10, 0, 0, 0]
    assert cu.tolist() == [0, 4, 5, 5] and counts.tolist() == [2, 2, 0]


def test_slots_short_list_and_full_table():
    table, slots, _, _, counts = oa.kv_slots([3, 0], [2, 5], [8], [[5, -1], [-1, -1]], 4, 16)
    assert table.tolist() == [[5, 8], [-1, -1]]                    # request 1 finds the list empty
    assert slots[:7].tolist() == [23, 32, -1, -1, -1, -1, -1] and counts.tolist() == [1, 3, 5]
    _, slots, _, _, counts = oa.kv_slots([7], [3], [2], [[0, 1]], 4, 3)
    assert slots.tolist() == [7, -1, -1] and counts.tolist() == [0, 0, 2]


def test_norm_and_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    w = rng.standard_normal(64)
    y = oa.norm_rope(x, w, 0.0, None, None, False)
    np.testing.assert_allclose((y / w) @ np.ones(64) * 0 + ((y / w) ** 2).mean(-1), 1.0, rtol=1e-12)
    # a rotation: keeps each pair's length, adds angles, and is the identity at angle 0
    ang = rng.uniform(0, 6, (5, 16))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        r = oa.norm_rope(x, None, 0.0, cs, [4, 0, 9], inter)        # position 9 counts as 4, the last
        a, b = (r[..., 0:32:2], r[..., 1:32:2]) if inter else (r[..., :16], r[..., 16:32])
        xa, xb = (x[..., 0:32:2], x[..., 1:32:2]) if inter else (x[..., :16], x[..., 16:32])
        z = (xa + 1j * xb) * np.exp(1j * ang[[4, 0, 4]])[:, None]
        np.testing.assert_allclose(a + 1j * b, z, rtol=1e-12, atol=1e-12)
        np.testing.assert_array_equal(r[..., 32:], x[..., 32:])


@pytest.mark.parametrize("lq,lk", [(5, 5), (3, 9), (6, 2)])
def test_prompt_against_torch_double(lq, lk):
    rng = np.random.default_rng(lq * 10 + lk)
    q, k, v = (torch.from_numpy(rng.standard_normal((n, h, 8))) for n, h in ((lq, 4), (lk, 2), (lk, 2)))
    out, lse = oa.attn_prompt(q.numpy(), k.numpy(), v.numpy(), [0, lq], [0, lk], 0.3)
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(2, 1)) * 0.3
    s = s.masked_fill(torch.arange(lk)[None] > torch.arange(lq)[:, None] + lk - lq, -torch.inf)
    p = torch.nan_to_num(torch.softmax(s, -1))                      # rows without a key: 0
    np.testing.assert_allclose(out, torch.einsum("hij,jhd->ihd", p, v.repeat_interleave(2, 1)).numpy(), atol=1e-13)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).t().numpy(), atol=1e-13)


def test_decode_is_the_last_row_of_a_prompt():
    """A request behind a prefix: its query against prefix + own keys laid out one after the other."""
    rng = np.random.default_rng(3)
    page, prefix, own = 4, 6, 5
    kc, vc = rng.standard_normal((8, page, 2, 8)), rng.standard_normal((8, page, 2, 8))
    q = rng.standard_normal((1, 4, 8))
    out, lse = oa.attn_decode(q, kc, vc, [[3, 1]], [own], [6, 0], prefix, 0.5)
    rows = [(6, 0), (6, 1), (6, 2), (6, 3), (0, 0), (0, 1), (3, 0), (3, 1), (3, 2), (3, 3), (1, 0)]
    k = np.stack([kc[r] for r in rows])
    v = np.stack([vc[r] for r in rows])
    ref, lref = oa.attn_prompt(q, k, v, [0, 1], [0, 11], 0.5)
    np.testing.assert_allclose(out, ref, atol=1e-14)
    np.testing.assert_allclose(lse, lref, atol=1e-14)


def test_equal_keys_average_the_values():
    k = np.ones((7, 1, 8))
    v = np.arange(7.0)[:, None, None] * np.ones(8)
    out, lse = oa.attn_prompt(np.ones((7, 1, 8)), k, v, [0, 7], [0, 7], 1.0)
    np.testing.assert_allclose(out[:, 0, 0], np.arange(7) / 2)
    np.testing.assert_allclose(lse[:, 0], 8 + np.log(np.arange(1, 8)))
