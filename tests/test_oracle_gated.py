"""The float64 oracle of gated attention and of the norm with rotation: the
recurrence against the matrix of token pairs, gradients against central
differences, steps against the sequence."""
import numpy as np
import pytest

from oracle import gated as og


def draw(seed, B=2, T=7, H=4, Hk=2, d=3):
    r = np.random.default_rng(seed)
    q, k, v = r.normal(size=(B, T, H, d)), r.normal(size=(B, T, Hk, d)), r.normal(size=(B, T, Hk, d))
    g = -np.abs(r.normal(size=(B, T, Hk)))
    return r, q, k, v, g


def test_recurrence_equals_pairs():
    r, q, k, v, g = draw(0)
    g[0, 3] = -np.inf
    out, _ = og.gated_forward(q, k, v, g, 0.7)
    with np.errstate(invalid="ignore"):
        for b in range(2):
            for h in range(4):
                ref = og.gated_pairs(q[b, :, h], k[b, :, h // 2], v[b, :, h // 2], g[b, :, h // 2], 0.7)
                np.testing.assert_allclose(out[b, :, h], ref, rtol=1e-12, atol=1e-13)


def test_lengths_cut_the_sequence():
    r, q, k, v, g = draw(1)
    s0 = r.normal(size=(2, 2, 3, 3))
    out, S = og.gated_forward(q, k, v, g, 1.0, s0, lens=[3, 0])
    ref, Sr = og.gated_forward(q[:1, :3], k[:1, :3], v[:1, :3], g[:1, :3], 1.0, s0[:1])
    np.testing.assert_allclose(out[0, :3], ref[0])
    assert not out[0, 3:].any() and not out[1].any()
    np.testing.assert_allclose(S[0], Sr[0])
    np.testing.assert_allclose(S[1], s0[1])


def test_gradients_against_differences():
    r, q, k, v, g = draw(2, T=5)
    s0, w, ws = r.normal(size=(2, 2, 3, 3)), r.normal(size=q.shape), r.normal(size=(2, 2, 3, 3))
    lens = [5, 3]

    def loss():
        o, S = og.gated_forward(q, k, v, g, 0.7, s0, lens)
        return np.sum(o * w) + np.sum(S * ws)
    grads = og.gated_backward(q, k, v, g, w, 0.7, s0, ws, lens)
    for x, gr in zip((q, k, v, g, s0), grads):
        for _ in range(25):
            i = tuple(r.integers(n) for n in x.shape)
            old, h = x[i], 1e-5
            x[i] = old + h
            up = loss()
            x[i] = old - h
            num = (up - loss()) / (2 * h)
            x[i] = old
            assert abs(num - gr[i]) <= 1e-8 * (1 + abs(num))


def test_steps_equal_the_sequence():
    r, q, k, v, g = draw(3)
    out, S = og.gated_forward(q, k, v, g, 0.5)
    pool = np.zeros((2, 2, 3, 3))
    for t in range(7):
        o, pool = og.gated_step(q[:, t], k[:, t], v[:, t], g[:, t], pool, 0.5)
        np.testing.assert_allclose(o, out[:, t], rtol=1e-12)
    np.testing.assert_allclose(pool, S, rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_properties(interleaved):
    r = np.random.default_rng(4)
    d, sections = 8, (2, 1)
    freq, w = r.random(3), r.normal(size=d)
    x, y = r.normal(size=(1, 1, 1, d)), r.normal(size=(1, 1, 1, d))
    dots = [np.sum(og.norm_rope(x, w, np.array([[[a + 5, b + 9]]]), freq, sections, interleaved, 1e-6)
                   * og.norm_rope(y, w, np.array([[[a, b]]]), freq, sections, interleaved, 1e-6))
            for a, b in ((0, 0), (100, -7), (12345, 3))]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)     # only the difference of positions counts
    n = og.norm_rope(x, np.ones(d), np.zeros((1, 1, 2)), freq, sections, interleaved, 0.0)
    np.testing.assert_allclose(np.mean(n * n), 1.0)
    dy = r.normal(size=x.shape)
    pos = np.array([[[3, 4]]])
    dx, dw = og.norm_rope_backward(x, w, pos, freq, sections, interleaved, 1e-3, dy)
    loss = lambda: np.sum(dy * og.norm_rope(x, w, pos, freq, sections, interleaved, 1e-3))  # noqa: E731
    for a, gr in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + 1e-6
            up = loss()
            a[i] = old - 1e-6
            num = (up - loss()) / 2e-6
            a[i] = old
            assert abs(num - gr[i]) <= 1e-7
