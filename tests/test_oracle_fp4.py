"""Pins for the oracle of the 4-bit cache, of reading a cache back and of joining partial
attentions: closed forms, invariants, and planted mistakes that must show."""
import numpy as np
import pytest

import oracle


def test_e2m1_values_round_trip_and_ties_go_to_even():
    v = np.array(oracle.E2M1_VALUES)
    assert np.array_equal(oracle.e2m1_encode(v), np.arange(8)) and np.array_equal(oracle.e2m1_encode(-v), np.arange(8, 16))
    ties = (v[1:] + v[:-1]) / 2
    assert oracle.e2m1_encode(ties).tolist() == [0, 2, 2, 4, 4, 6, 6]
    for k, t in enumerate(ties):
        assert oracle.e2m1_encode(np.nextafter(t, 0)) == k and oracle.e2m1_encode(np.nextafter(t, 9)) == k + 1
    assert oracle.e2m1_encode(1e9) == 7
    b = np.arange(256, dtype=np.uint8)
    got = oracle.e2m1_decode(b[:, None])
    assert np.array_equal(oracle.e2m1_encode(got[:, 0]), b & 15) and np.array_equal(oracle.e2m1_encode(got[:, 1]), b >> 4)


def test_row_descales():
    a = np.float32([6.0, 3.0, 6.01, 0.0, 1e-37, np.inf, np.nan, 3.3e38])
    s = oracle.row_descale(a)
    assert s[0] == 1.0 and s[1] == 0.5 and s[3] == 0.0 and s[4] == 2.0 ** -100 and np.isnan(s[5:7]).all()
    assert s[2] == 1.0 + 2.0 ** -7
    fine = s[[0, 1, 2, 4, 7]]
    assert np.all(fine.view(np.uint32) & 0xFFFF == 0) and np.all(a[[0, 1, 2, 4, 7]] / fine <= 6.0)
    # no smaller bfloat16 would do
    down = (s[[0, 1, 2, 7]].view(np.uint32) - 0x10000).view(np.float32)
    assert np.all(a[[0, 1, 2, 7]].astype(np.float64) / down > 6.0)


def test_rows_are_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 64)).astype(np.float32)
    x[3] = 0
    b, s = oracle.quantize_rows(x)
    got = oracle.e2m1_decode(b) * s[:, None]
    assert np.all(np.abs(got - x) <= np.maximum(np.abs(x), s[:, None]) * 0.25 * (1 + 1e-6))
    assert np.all(got[3] == 0) and s[3] == 0
    # of values that are codes already, nothing is lost
    again = oracle.quantize_rows((oracle.e2m1_decode(b)).astype(np.float32))
    assert np.array_equal(oracle.e2m1_decode(again[0]) * again[1][:, None], oracle.e2m1_decode(b))


@pytest.mark.parametrize("interleaved", [False, True])
def test_float32_key_rows_are_the_float64_ones_rounded(interleaved):
    rng = np.random.default_rng(2)
    k = rng.standard_normal((5, 2, 64))
    c, s = oracle.rope_table(9, 48)
    signs = np.where(rng.random(64) < 0.5, -1.0, 1.0)
    pos = np.array([0, 8, 3, 3, 7])
    got = oracle.key_rows_f32(k, pos, c, s, interleaved, signs)
    ref = oracle.key_rows(k, pos, c, s, interleaved, signs)
    assert got.dtype == np.float32 and np.allclose(got, ref, atol=2.0 ** -19)
    assert not np.allclose(oracle.key_rows_f32(k, pos, c, s, not interleaved, signs), ref, atol=0.1)


def test_append_writes_its_slots_only():
    rng = np.random.default_rng(3)
    codes, descale = rng.integers(0, 256, (3, 2, 16, 32)).astype(np.uint8), np.ones((3, 2, 16), np.float32)
    x = rng.standard_normal((3, 2, 64)).astype(np.float32)
    c, s = oracle.append_fp4(x, codes, descale, [20, -1, 47])
    changed = np.argwhere((c != codes).any(-1).any(1))
    assert changed.tolist() == [[1, 4], [2, 15]]
    v = oracle.dequantize_cache_fp4(c, s)
    assert v.shape == (3, 16, 2, 64) and np.abs(v[1, 4] - x[0]).max() < 1.0
    assert np.array_equal(v[1, 4, 1], oracle.e2m1_decode(c[1, 1, 4]) * s[1, 1, 4])


def test_read_back_of_ranges():
    v = np.arange(4 * 2 * 1 * 1, dtype=np.float64).reshape(4, 2, 1, 1)      # slot s holds s
    got = oracle.read_cache(v, [[3, 0], [1, 2]], [3, 4], [1, 0], [4, 2])
    assert got[0].ravel().tolist() == [7, 0, 0, 0] and got[1].ravel().tolist() == [2, 3]


def test_merge_is_attention_over_the_union():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((1, 2, 3, 8)), rng.standard_normal((1, 2, 9, 8)), rng.standard_normal((1, 2, 9, 8))
    parts = [oracle.attention_cross_forward(q, k[:, :, s], v[:, :, s], 0.4) for s in (slice(0, 4), slice(4, 9))]
    o, lse = oracle.merge_attention(*parts[0], *parts[1])
    ref = oracle.attention_cross_forward(q, k, v, 0.4)
    assert np.allclose(o, ref[0]) and np.allclose(lse, ref[1])
    none = np.full_like(lse, -np.inf)
    o, lse = oracle.merge_attention(*ref, np.full_like(ref[0], np.nan), none)
    assert np.array_equal(o, ref[0]) and np.array_equal(lse, ref[1])
    o, lse = oracle.merge_attention(ref[0], none, ref[0], none)
    assert np.all(o == 0) and np.all(lse == -np.inf)
