"""Pins of the 4-bit cache's oracle: formats, rounding, layout and the page model (CPU)."""
import numpy as np
import pytest
import torch

from oracle import kv4


def test_format_tables_match_their_definitions():
    assert list(kv4.E2M1) == [0, .5, 1, 1.5, 2, 3, 4, 6]
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv4.E4M3, e4m3)


def test_rounding_is_to_nearest_with_ties_to_the_even_code():
    x = np.array([0.0, .24, .25, .26, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.0, 100.0])
    assert list(kv4.nearest(x, kv4.E2M1)) == [0, 0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 7]
    y = np.random.default_rng(0).random(2000) * 448
    ref = torch.tensor(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv4.nearest(y, kv4.E4M3), ref)


def test_quantise_worked_example():
    x = np.zeros((1, 1, 64))
    x[0, 0, :4] = [6.0, -3.0, 1.25, 0.2]  # scale 1: codes of 6, -3, 1 (tie to even), 0
    x[0, 0, 16] = np.inf
    x[0, 0, 32] = 6 * 2.0 ** -11            # its scale, half of the smallest e4m3 number, ties to 0
    codes, s = kv4.quantise(x, np.ones(1))
    assert list(codes[0, 0, :4]) == [7, 13, 2, 0]
    assert list(s[0, 0]) == [0x38, 0x7f, 0, 0]
    assert not codes[0, 0, 16:].any()


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_append_then_rows_gives_code_times_scale_and_leaves_the_rest(D, P):
    rng = np.random.default_rng(D)
    H, table, lens = 2, [[3, 1, -1], [0, 2, -1]], [P + 5, 7]
    pool = rng.integers(0, 256, (4, H, P // 16, 18 * D), dtype=np.uint8)
    before = pool.copy()
    counts = [8, 3]
    k, v = rng.standard_normal((2, 11, H, D))
    ks, vs = np.array([.5, 2.0]), np.array([1.0, 4.0])
    kv4.append(pool, table, lens, [0, 1], counts, k, v, ks, vs)
    kc, sk = kv4.quantise(k, ks)
    want = np.concatenate([kv4.E2M1, -kv4.E2M1])[kc] * np.repeat(kv4.E4M3[sk], 16, -1) * ks[None, :, None]
    for slot, a, b in ((0, 0, 8), (1, 8, 11)):
        got, _ = kv4.rows(pool, table, slot, lens[slot], ks, vs)
        assert np.array_equal(got[:, -(b - a):], want[a:b].transpose(1, 0, 2))
        # the error of a value is at most half the gap 2 between the codes 4 and 6, times the scale
        assert np.abs(got[:, -(b - a):] - k[a:b].transpose(1, 0, 2)).max() <= 1.3 * np.repeat(
            kv4.E4M3[sk], 16, -1).max() * ks.max()
    assert np.array_equal(pool[2], before[2])  # no position of this call
    k0, v0 = kv4.unit_rows(before[3, 0, 0], D)
    k1, v1 = kv4.unit_rows(pool[3, 0, 0], D)
    n = P + 5 - 8
    keep = min(n, 16)
    assert np.array_equal(k0[:keep], k1[:keep], equal_nan=True) and np.array_equal(v0[:keep], v1[:keep], equal_nan=True)


def test_page_model_shares_full_pages_and_compacts():
    m = kv4.Pages(8, 4, 4, 16)
    assert m.reserve([0, 1], [40, 16]) == (4, 0)
    assert m.table[0] == [0, 1, 2, -1] and m.table[1][0] == 3
    assert m.fork([0, 0], [2, 3]) == (2, 0)
    assert m.refs == [3, 3, 1, 1, 1, 1, 0, 0] and m.table[3] == [0, 1, 5, -1]
    m.release([0, 0])
    assert m.refs == [2, 2, 0, 1, 1, 1, 0, 0] and m.lens[0] == 0
    assert m.compact() == (3, 0)
    assert m.refs == [2, 2, 1, 1, 1, 0, 0, 0] and m.table[3] == [0, 1, 2, -1]
    assert m.reserve([0], [64]) == (3, 1)
    assert m.reserve([0, 0], [1, 1]) == (3, -1)
    assert m.fork([2], [1]) == (3, -1)


def test_attention_ignores_masked_keys_whatever_they_hold():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 3, 8)), rng.standard_normal((1, 5, 8)), rng.standard_normal((1, 5, 8))
    o, lse = kv4.attention(q, k, v, 0.3, True)
    k[:, -1], v[:, -1] = np.nan, np.nan
    o2, lse2 = kv4.attention(q, k, v, 0.3, True)
    assert np.array_equal(o[:, :2], o2[:, :2]) and np.array_equal(lse[:, :2], lse2[:, :2])
    assert np.isnan(o2[:, 2]).all()
    o, lse = kv4.attention(q, k[:, :1], v[:, :1], 0.3, True)
    assert (lse[:, :2] == -np.inf).all() and not o[:, :2].any()
