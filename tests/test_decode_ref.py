"""The plain forms of the decode-step operators, pinned against closed forms and independent computations."""
import math

import numpy as np
import pytest

from oracle import decode_ref as R


def cache(rng, pages, heads, size, D):
    return rng.standard_normal((pages, heads, size, D)), rng.standard_normal((pages, heads, size, D))


def test_attention_of_equal_keys_is_the_mean():
    rng = np.random.default_rng(1)
    k, v = cache(rng, 4, 2, 3, 8)
    k[:] = k[0, 0, 0]
    table = np.array([[2, 0, 3]])
    q = rng.standard_normal((1, 1, 4, 8))
    o, w, _, _ = R.attn_decode(k, v, table, [7], q, 1, 0.5, weights=np.ones((1, 2, 9)), decay=0.5)
    for h in range(4):
        rows = [v[table[0, j // 3], h // 2, j % 3] for j in range(7)]
        np.testing.assert_allclose(o[0, 0, h], np.mean(rows, 0), rtol=1e-12)
    np.testing.assert_allclose(w[:, :, :7], 0.5 + 2 / 7, rtol=1e-12)
    assert (w[:, :, 7:] == 1).all()


def test_attention_ranges():
    """With one-hot values the output is the softmax itself: its support is the row's range."""
    rng = np.random.default_rng(2)
    k, v = cache(rng, 1, 1, 8, 8)
    v[0, 0] = np.eye(8)
    q = rng.standard_normal((1, 3, 1, 8))
    table = np.zeros((1, 1), int)
    for window, want in ((0, [range(0, 4), range(0, 5), range(0, 6)]), (2, [range(2, 4), range(3, 5), range(4, 6)])):
        o = R.attn_decode(k, v, table, [6], q, 3, 1.0, window=window)[0]
        for i in range(3):
            assert set(np.flatnonzero(o[0, i, 0])) == set(want[i])
            np.testing.assert_allclose(o[0, i, 0].sum(), 1)
    assert (R.attn_decode(k, v, table, [2], q, 3, 1.0)[0][0, 0] == 0).all()  # fewer slots than new tokens
    assert (R.attn_decode(k, v, table, [0], q, 3, 1.0)[0] == 0).all()


def test_attention_softcap_and_scales():
    rng = np.random.default_rng(3)
    k, v = cache(rng, 1, 1, 5, 8)
    q = rng.standard_normal((1, 1, 1, 8))
    table = np.zeros((1, 1), int)
    s = 3 * np.tanh(k[0, 0] @ q[0, 0, 0] * 0.7 * 2.0 / 3)
    p = np.exp(s) / np.exp(s).sum()
    o = R.attn_decode(k, v, table, [5], q, 1, 0.7, softcap=3.0, k_scale=2.0, v_scale=0.25)[0]
    np.testing.assert_allclose(o[0, 0, 0], 0.25 * p @ v[0, 0], rtol=1e-12)


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_is_a_rotation(pairs):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 2, 8)).astype(np.float32)
    a = rng.uniform(-3, 3, (3, 3))
    y = R.rope(x, np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32), 6, pairs)
    for t in range(3):
        for h in range(2):
            for i in range(3):
                at = (2 * i, 2 * i + 1) if pairs else (i, i + 3)
                z = complex(x[t, h, at[0]], x[t, h, at[1]]) * np.exp(1j * a[t, i])
                np.testing.assert_allclose([y[t, h, at[0]], y[t, h, at[1]]], [z.real, z.imag], atol=1e-6)
    assert (y[..., 6:] == x[..., 6:]).all()
    assert (R.rope(x, np.zeros((3, 0), np.float32), 0, pairs) == x).all()


def test_evict_by_hand():
    w = np.array([[[5, 1, 1, 0, 9, 2, float("nan"), 3.0]]])
    p = np.arange(8)[None, None]
    new, take = R.kv_evict([7], w, p, 4, 0, 0)      # slot 7 is not there
    assert new[0] == 4 and take[0][0] == [0, 4, 5, 6]
    new, take = R.kv_evict([7], w, p, 4, 2, 1)      # 0, 1 and 6 are protected
    assert take[0][0] == [0, 1, 4, 6]
    new, take = R.kv_evict([7], w, p, 2, 1, 1)      # only protected ones fit
    assert take[0][0] == [0, 6]
    new, take = R.kv_evict([3], w, p, 4, 0, 0)
    assert new[0] == 3 and take[0][0] == [0, 1, 2]
    w = np.zeros((1, 1, 6))                          # equal weights: the lowest slots go
    assert R.kv_evict([6], w, p, 4, 0, 0)[1][0][0] == [4, 5, 2, 3]
    # every slot protected: still cut to the budget
    assert R.kv_evict([6], w, np.full((1, 1, 6), 7), 4, 0, 1)[1][0][0] == [4, 5, 2, 3]


def test_norm_closed_forms():
    y = np.array([[3.0, -3.0, 3.0, -3.0]])
    r = np.ones((1, 4))
    h, x = R.norm_residual(y, 1, None, None, 0.0, None, 2.0, r, 0, None, None, 0.0)
    np.testing.assert_allclose(h, [[3, -1, 3, -1]])
    np.testing.assert_allclose(x, h)
    h, x = R.norm_residual(None, 1, None, None, 0.0, None, 2.0, y + 5, 2, [2, 2, 2, 2], [1, 0, 0, 0], 0.0)
    np.testing.assert_allclose(h, y + 5)
    np.testing.assert_allclose(x, [[3, -2, 2, -2]])


def test_sample_weight_is_a_power_of_two():
    """Against 2^-d: the series of degree 7 about the middle errs by (ln 2 / 2)^8 / 8! < 6e-9 of the value, each of 14
    roundings by 2^-25 of at most the value, the last truncation by 2^-40."""
    for d in np.linspace(0, 40.99, 2001, dtype=np.float32):
        want = 2.0 ** (40 - float(d))
        assert abs(int(R.sample_weight(d)) - want) <= want * 15 * 2 ** -25 + 1, d
    assert R.sample_weight(np.float32(41)) == 0 and R.sample_weight(np.float32("nan")) == 0
    assert R.sample_weight(np.float32("inf")) == 0


def test_sample_by_hand():
    z = np.log(np.array([0.1, 0.4, 0.1, 0.3, 0.1], np.float32))
    draw = lambda **a: R.sample(z, **{**dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.0), **a})  # noqa: E731
    assert [draw(u=x)[0] for x in (0.05, 0.15, 0.45, 0.55, 0.65, 0.85, 0.95)] == [0, 1, 1, 2, 3, 3, 4]
    assert draw(u=0.99)[1] == pytest.approx(0.1, abs=1e-6)
    assert draw(top_k=2, u=0.58)[0] == 3 and draw(top_k=2, u=0.56)[0] == 1
    assert draw(top_k=3, u=0.0)[0] == 0           # equal logits: the lowest index stays
    assert draw(top_p=0.69, u=0.99)[0] == 3 and draw(top_p=0.39, u=0.99)[0] == 1 and draw(top_p=0.0, u=0.9)[0] == 1
    assert draw(min_p=0.5, u=0.0)[0] == 1 and draw(min_p=0.2, u=0.0)[0] == 0
    assert draw(temperature=0.0, u=0.9) == (1, 1.0)
    assert R.sample(np.full(3, -np.inf), 1.0, 0, 1.0, 0.0, 0.5) == (-1, 0.0)
    assert R.sample(np.array([0, np.inf, np.nan]), 1.0, 0, 1.0, 0.0, 0.9) == (1, 1.0)


def test_sample_frequencies():
    rng = np.random.default_rng(5)
    z = rng.standard_normal(12).astype(np.float32)
    p = np.exp(z / 0.8) / np.exp(z / 0.8).sum()
    u = (np.arange(4000) + 0.5) / 4000            # a stratified stream: counts are the probabilities to one part
    got = np.bincount([R.sample(z, 0.8, 0, 1.0, 0.0, x)[0] for x in u], minlength=12) / 4000
    assert np.abs(got - p).max() <= 1 / 4000 + 1e-6
    assert math.isclose(sum(got), 1)


def test_sample_weight_stays_in_its_octave():
    """The series ends in [1/2, 1] for every fraction near 0 and near 1, so 24 bits hold it exactly."""
    grid = np.arange(2 ** 22, dtype=np.float64)
    for d in (grid * 2.0 ** -25, 0.75 + grid * 2.0 ** -24):
        w = R.sample_weight(d.astype(np.float32))
        assert w.min() >= 2 ** 39 and w.max() <= 2 ** 40
    assert R.sample_weight(0.0) == 2 ** 40
