"""Pins of the oracle of the 4-bit cache, the pages and the residual stream's norms: worked examples and identities."""
import numpy as np
import torch

import oracle
import synth
from oracle import cache as oc


def test_rows_are_the_activation_quantiser():
    for g in (1.0, 0.25, 8.0):
        bits = synth.random_bf16(1, (7, 64), 3.0)
        c, s = oracle.quantize_nvfp4(bits, g)
        c2, s2 = oc.nvfp4_rows(oracle.bf16_value(bits), g)
        assert np.array_equal(c, c2) and np.array_equal(s, s2)
        assert np.array_equal(oc.nvfp4_values(c2, s2, g), oracle.dequant_nvfp4_act(c, s, g))


def test_rows_worked_example():
    x = np.zeros(16)
    x[:6] = [6.0, -0.25, 0.75, 2.5, -5.0, 0.26]                     # scale 1: ties to 0, 1, 2, 4; 0.26 to 0.5
    c, s = oc.nvfp4_rows(x, 1.0)
    assert s.tolist() == [0x38] and c[:3].tolist() == [7 | 8 << 4, 2 | 4 << 4, (8 | 6) | 1 << 4]
    assert oc.nvfp4_values(c, s, 2.0)[:6].tolist() == [12.0, 0.0, 2.0, 4.0, -8.0, 1.0]


def test_cache_values_layout():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 16, 2, 32))                          # pages, page, heads, dim
    c, s = oc.nvfp4_rows(np.swapaxes(x, 1, 2), 1.0)
    k, v = oc.cache_values(c, s, c, np.swapaxes(s, 2, 3), 1.0, 1.0)
    assert np.array_equal(k, v) and k.shape == x.shape and np.abs(k - x).max() < 0.6


def test_gather_worked_example():
    rows = np.arange(12).reshape(3, 4)                               # 3 pages of 4 rows
    out = oc.gather(rows, [[2, -1], [0]], [1, 7, 10], 11, [1], 2, np.full(11, -7))
    assert out.tolist() == [-7, 4, 5, 8, 9, 10, 11, 4, 5, 0, -7]
    assert oc.gather(rows, [[2, -1]], [0, 6], 6, [], 0, np.zeros(6)).tolist() == [8, 9, 10, 11, 0, 0]


def test_fork_worked_example():
    buf = np.arange(6)[:, None] * 10
    table, lens, (b,), counts = oc.fork([[4, 1, -1], [9, 9, 9], [9, 9, 9], [9, 9, 9]], [6, 0, 0, 3], [0, 0, 7], [1, 2, 3], [5, 0], 4,
                                        [buf])
    assert table.tolist() == [[4, 1, -1], [4, 5, 9], [4, 0, 9], [9, 9, 9]] and lens.tolist() == [6, 6, 6, 3]
    assert b[:, 0].tolist() == [10, 10, 20, 30, 40, 10] and counts.tolist() == [2, 2]
    table, lens, _, counts = oc.fork([[4, 1], [9, 9]], [6, 0], [0], [1], [], 4, [buf])
    assert table.tolist() == [[4, 1], [4, -1]] and lens.tolist() == [6, 4] and counts.tolist() == [0, 1]
    table, lens, (b,), counts = oc.fork([[4, 1], [9, 9]], [8, 0], [0], [1], [], 4, [buf])
    assert table.tolist() == [[4, 1], [4, 1]] and lens.tolist() == [8, 8] and counts.tolist() == [0, 0] and np.array_equal(b, buf)


def test_free_and_compact_worked_example():
    table, lens = [[5, 2, 7], [5, 6, 1], [3, 3, 3]], [9, 8, 0]       # page 4: 3 pages, 2 pages, none; page 5 shared
    free, counts = oc.free_pages(table, lens, 4, 8)
    assert free.tolist() == [0, 1, 3, 4, -1, -1, -1, -1] and counts.tolist() == [4, 4]
    out, (b,), counts = oc.compact(table, lens, 4, [np.arange(8) * 10])
    assert out.tolist() == [[0, 2, 3], [0, 1, -1], [-1, -1, -1]] and counts.tolist() == [4, 3]
    assert b.tolist() == [50, 60, 20, 70, 40, 50, 60, 70]
    free, _ = oc.free_pages(out, lens, 4, 8)
    assert free[:4].tolist() == [4, 5, 6, 7]


def test_block_norm_against_torch():
    rng = np.random.default_rng(2)
    x, r, w, p, g = rng.standard_normal((5, 40)), rng.standard_normal((5, 40)), *rng.standard_normal((3, 40))
    norm = lambda a, b: torch.nn.functional.rms_norm(torch.tensor(a), (40,), torch.tensor(b), 1e-5).numpy()  # noqa: E731
    h, y = oc.block_norm(x, w, r, p, g, 0.5, 1e-5)
    np.testing.assert_allclose(h, r + 0.5 * g * norm(x, p), rtol=1e-12)
    np.testing.assert_allclose(y, norm(h, w), rtol=1e-12)
    h, y = oc.block_norm(x, w, eps=1e-5)
    assert np.array_equal(h, x)
    np.testing.assert_allclose(y, norm(x, w), rtol=1e-12)
