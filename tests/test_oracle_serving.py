"""Pins for the oracle of cross attention, rotary positions, block tables and the
e4m3 cache append: closed forms, invariants, finite differences, and planted
mistakes that must show."""
import numpy as np
import pytest

import oracle


def _normal(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_cross_of_equal_lengths_is_attention():
    q, k, v, do = (_normal(i, 2, 4, 9, 8) for i in range(4))
    o, lse = oracle.attention_cross_forward(q, k, v, 0.3)
    ref_o, ref_l = oracle.attention_forward(q, k, v, 0.3)
    assert np.array_equal(o, ref_o) and np.array_equal(lse, ref_l)
    for a, b in zip(oracle.attention_cross_backward(q, k, v, do, 0.3), oracle.attention_backward(q, k, v, do, 0.3)):
        assert np.array_equal(a, b)


def test_cross_one_key_copies_its_value_and_no_key_gives_nothing():
    q, k, v, do = _normal(1, 2, 4, 5, 8), _normal(2, 2, 2, 7, 8), _normal(3, 2, 2, 7, 8), _normal(4, 2, 4, 5, 8)
    o, lse = oracle.attention_cross_forward(q, k, v, 0.5, [1, 0])
    assert np.allclose(o[0], np.repeat(v[0, :, :1], 2, 0)) and np.all(o[1] == 0)
    assert np.allclose(lse[0], 0.5 * np.einsum("hnd,hd->hn", q[0], np.repeat(k[0, :, 0], 2, 0)))
    assert np.all(lse[1] == -np.inf)
    dq, dk, dv = oracle.attention_cross_backward(q, k, v, do, 0.5, [1, 0])
    assert np.allclose(dq, 0) and np.allclose(dk, 0)          # softmax over one key is constant
    assert np.allclose(dv[0, :, 0], do[0].reshape(2, 2, 5, 8).sum((1, 2))) and np.all(dv[0, :, 1:] == 0)
    assert np.all(dv[1] == 0)


def test_cross_ignores_what_stands_behind_the_lengths():
    q, k, v = _normal(1, 2, 2, 5, 8), _normal(2, 2, 2, 7, 8), _normal(3, 2, 2, 7, 8)
    a = oracle.attention_cross_forward(q, k, v, 0.5, [4, 6])
    k[0, :, 4:], v[1, :, 6:] = np.nan, np.inf
    b = oracle.attention_cross_forward(q, k, v, 0.5, [4, 6])
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_cross_gradient_by_differences():
    q, k, v, do = _normal(1, 1, 2, 3, 4), _normal(2, 1, 1, 5, 4), _normal(3, 1, 1, 5, 4), _normal(4, 1, 2, 3, 4)
    lens, eps = [4], 1e-6
    grads = oracle.attention_cross_backward(q, k, v, do, 0.7, lens)
    for x, g in zip((q, k, v), grads):
        for at in np.ndindex(x.shape):
            keep = x[at]
            x[at] = keep + eps
            up = (oracle.attention_cross_forward(q, k, v, 0.7, lens)[0] * do).sum()
            x[at] = keep - eps
            down = (oracle.attention_cross_forward(q, k, v, 0.7, lens)[0] * do).sum()
            x[at] = keep
            assert abs((up - down) / (2 * eps) - g[at]) < 1e-7


def test_rope_table_closed_forms():
    c, s = oracle.rope_table(5, 16, first=3)
    assert np.allclose(c ** 2 + s ** 2, 1)
    assert np.allclose(np.arctan2(s[:, 0], c[:, 0]), (np.arange(3, 8) + np.pi) % (2 * np.pi) - np.pi)
    # interpolation of every frequency: position 2 p at factor 2 is position p
    c2, s2 = oracle.rope_table(10, 16, factor=2.0)
    c1, s1 = oracle.rope_table(5, 16)
    assert np.allclose(c2[::2], c1) and np.allclose(s2[::2], s1)
    # by parts: fast columns as without a factor, slow ones as interpolated
    cp, _ = oracle.rope_table(64, 64, factor=4.0, orig_len=512, low=1.0, high=32.0)
    plain, whole = oracle.rope_table(64, 64)[0], oracle.rope_table(64, 64, factor=4.0)[0]
    turns = 512 * 10000.0 ** (-2 * np.arange(32) / 64) / (2 * np.pi)
    assert np.allclose(cp[:, turns >= 32], plain[:, turns >= 32])
    assert np.allclose(cp[:, turns <= 1], whole[:, turns <= 1])
    between = (turns > 1) & (turns < 32)
    assert between.any() and not np.allclose(cp[:, between], plain[:, between])
    assert np.allclose(oracle.rope_table(4, 16, attn_factor=1.5)[0], 1.5 * oracle.rope_table(4, 16)[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_rotation_invariants(interleaved):
    c, s = oracle.rope_table(9, 8)
    x, y = _normal(1, 9, 12), _normal(2, 9, 12)
    r = oracle.rope_rotate(x, c, s, interleaved)
    assert np.array_equal(r[:, 8:], x[:, 8:]) and np.array_equal(r[0], x[0])
    assert np.allclose(np.linalg.norm(r, axis=1), np.linalg.norm(x, axis=1))
    assert np.allclose(oracle.rope_rotate(r, c, s, interleaved, inverse=True), x)
    # the inverse is the transpose: <R x, y> = <x, R' y>
    back = oracle.rope_rotate(y, c, s, interleaved, inverse=True)
    assert np.allclose((r * y).sum(1), (x * back).sum(1))
    # scores depend on the distance of the positions alone
    q = oracle.rope_rotate(np.repeat(x[:1], 9, 0), c, s, interleaved)
    k = oracle.rope_rotate(np.repeat(y[:1], 9, 0), c, s, interleaved)
    assert np.allclose((q[4] * k[1]).sum(), (q[8] * k[5]).sum())
    assert not np.allclose((q[4] * k[1]).sum(), (q[8] * k[4]).sum())


def test_rope_halves_is_the_prepass_rotation_and_layouts_are_permutations():
    c, s = oracle.rope_table(6, 16)
    x = _normal(3, 6, 16)
    r = oracle.rope_rotate(x, c, s)
    assert np.allclose(r, oracle.rotary_embed(x, c, s))
    order = np.arange(16).reshape(2, 8).T.ravel()            # halves -> neighbours
    assert np.allclose(oracle.rope_rotate(x[:, order], c, s, True), r[:, order])


def test_block_tables_by_hand():
    table = [[7, -1, -1], [-1, -1, -1], [2, 5, -1]]
    got = oracle.block_tables(table, [3, 0, 8], [2, 0, 1], [9, 4, 6], 4, 5)
    assert got[0].tolist() == [[7, 9, -1], [-1, -1, -1], [2, 5, 4]]
    assert got[1].tolist() == [5, 0, 9] and got[2].tolist() == [0, 2, 2, 3]
    assert got[3].tolist() == [7 * 4 + 3, 9 * 4, 4 * 4, -1, -1] and got[4].tolist() == [3, 4, 8, -1, -1]
    assert got[5] == 2


def test_append_fp8_of_whole_pages_is_the_block_quantiser():
    x = _normal(5, 2 * 16, 2, 8).astype(np.float32)
    codes, desc = oracle.append_fp8(x, np.full((3, 16, 2, 8), 0x55, np.uint8), np.ones((3, 2), np.float32),
                                    np.r_[32:48, 0:16])
    cache = np.zeros((3, 16, 2, 8), np.float32)
    cache[2], cache[0] = x[:16], x[16:]
    ref_c, ref_d = oracle.quantize_paged_cache(cache)
    assert np.array_equal(codes[[0, 2]], ref_c[[0, 2]]) and np.array_equal(desc[[0, 2]], ref_d[[0, 2]])
    assert np.all(codes[1] == 0x55) and np.all(desc[1] == 1)


def test_append_fp8_growing_descale():
    """Rows one by one: the descale is the running maximum's, earlier values stay
    within their roundings (half a step each time the descale grew), and a row that
    does not raise the maximum changes no code of the others."""
    x = _normal(6, 16, 1, 8).astype(np.float32)
    codes, desc = np.zeros((1, 16, 1, 8), np.uint8), np.ones((1, 1), np.float32)
    grew = 0
    for t in range(16):
        before, was = codes.copy(), desc.copy()
        codes, desc = oracle.append_fp8(x[t:t + 1], codes, desc, np.array([t]))
        top = np.abs(x[:t + 1]).max() / np.float32(448)
        assert desc[0, 0] == np.float32(top)
        if t and desc[0, 0] == was[0, 0]:
            assert np.array_equal(codes[0, :t], before[0, :t])
        else:
            grew += 1
        value = oracle.e4m3_decode(codes[0, :t + 1, 0]) * desc[0, 0]
        bound = grew * np.maximum(np.abs(x[:t + 1, 0]) * 2.0 ** -4, 2.0 ** -10 * desc[0, 0]) * 1.1
        assert np.all(np.abs(value - x[:t + 1, 0]) <= bound)
    assert grew >= 2


@pytest.mark.parametrize("size", [1e-20, 1e-25, 1e-30, 1e-37, 1e-40])
def test_append_fp8_of_tiny_values(size):
    """A descale of 2^-90 at least: values within half a step of it, zeros exact."""
    x = (_normal(7, 16, 2, 8) * size).astype(np.float32)
    x[3], x[:, 1, 2] = 0, 0
    codes, desc = oracle.append_fp8(x, np.full((1, 16, 2, 8), 0x7F, np.uint8), np.full((1, 2), np.nan, np.float32),
                                    np.arange(16))
    assert np.all(desc >= 2.0 ** -90) and np.all(desc <= max(2.0 ** -90, np.abs(x).max()))
    value = oracle.e4m3_decode(codes[0]) * desc[0][:, None]
    assert np.all(np.abs(value - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * desc[0][:, None]))
    assert not value[3].any() and not value[:, 1, 2].any()
