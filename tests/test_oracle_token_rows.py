"""The token rows' float64 oracle, pinned without restating it: closed forms,
central differences for every gradient, and identities."""
import numpy as np
import pytest

from oracle import token_rows as T


def _difference(f, x, at, step):
    hi, lo = x.copy(), x.copy()
    hi[at] += step
    lo[at] -= step
    return (f(hi) - f(lo)) / (2 * step)


def test_embed_is_indexing():
    rng = np.random.default_rng(1)
    table = rng.standard_normal((7, 8)).astype(np.float32)
    ids = np.array([3, -1, 6, 0, 3, 7])
    y = T.embed_rows(table, ids, 2.0)
    assert np.array_equal(y[0], 2 * table[3]) and np.array_equal(y[4], y[0])
    assert not y[1].any() and not y[5].any()


def test_embed_gradient_is_the_transpose():
    rng = np.random.default_rng(2)
    ids = np.array([3, -1, 6, 0, 3, 7, 3])
    dy, table = rng.standard_normal((7, 8)), rng.standard_normal((7, 8)).astype(np.float32)
    d, mag, count = T.embed_rows_backward(dy, ids, 7, 0.5)
    # <dy, E W> = <E^T dy, W>
    assert np.isclose((T.embed_rows(table, ids, 0.5) * dy).sum(), (d * table).sum(), rtol=1e-6)
    assert count.tolist() == [1, 0, 0, 3, 0, 0, 1] and (mag >= np.abs(d)).all()


@pytest.mark.parametrize("hd", [16, 48, 64])
def test_qk_keeps_the_rms_and_reduces_to_it_at_position_zero(hd):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 2 * hd))
    inv = (10000.0 ** (-np.arange(0, hd, 2) / hd)).astype(np.float32)
    y, _ = T.qk_rows_rms(x, np.array([0, 5, 10 ** 6]), inv, None, hd, 0.0)
    heads = y.reshape(3, 2, hd)
    assert np.allclose((heads ** 2).mean(-1), 1)
    v = x.reshape(3, 2, hd)
    assert np.allclose(heads[0], v[0] / np.sqrt((v[0] ** 2).mean(-1, keepdims=True)))


def test_qk_quarter_turn():
    """A pair turned by pi/2 (to the fp32 value of pi/2): (a, b) -> (-b, a)."""
    inv = np.zeros(8, np.float32)
    inv[2] = np.float32(np.pi / 2)
    x = np.arange(1, 17, dtype=np.float64)[None]
    y, _ = T.qk_rows_rms(x, np.array([1]), inv, None, 16, 0.0)
    D = np.sqrt((x ** 2).mean())
    want = x[0].copy()
    want[2], want[10] = -x[0, 10], x[0, 2]
    assert np.allclose(y[0] * D, want, atol=1e-6)


def test_qk_gradient_against_differences():
    rng = np.random.default_rng(4)
    hd, rows, heads = 16, 3, 2
    x, dy = rng.standard_normal((2, rows, heads * hd))
    w = rng.uniform(0.5, 1.5, hd)
    pos = np.array([0, 7, 300])
    inv = (100.0 ** (-np.arange(0, hd, 2) / hd)).astype(np.float32)
    f = lambda v, u: (T.qk_rows_rms(v, pos, inv, u, hd, 1e-3)[0] * dy).sum()  # noqa: E731
    dx, dw, mag, dw_mag = T.qk_rows_rms_backward(x, pos, inv, w, dy, hd, 1e-3)
    for at in [(0, 0), (1, 9), (2, 31), (2, 17)]:
        assert np.isclose(dx[at], _difference(lambda v: f(v, w), x, at, 1e-5), rtol=1e-6, atol=1e-8)
    for j in (0, 5, 15):
        assert np.isclose(dw[j], _difference(lambda u: f(x, u), w, j, 1e-5), rtol=1e-6, atol=1e-8)
    assert (mag >= np.abs(dx)).all() and (dw_mag >= np.abs(dw)).all()


def test_logprob_closed_forms():
    z = np.full((1, 10), 3.0, np.float32)                     # uniform over 10
    logp, ent, lse, ids, top = T.logprob_rows(z, [4], 3)
    assert np.isclose(logp[0], -np.log(10)) and np.isclose(ent[0], np.log(10))
    assert np.isclose(lse[0], 3 + np.log(10)) and ids[0].tolist() == [0, 1, 2]
    z[0, 5:] = -np.inf                                        # uniform over 5
    logp, ent, lse, ids, _ = T.logprob_rows(z, [7], 6)
    assert logp[0] == -np.inf and np.isclose(ent[0], np.log(5))
    assert ids[0].tolist() == [0, 1, 2, 3, 4, -1]
    z[:] = -np.inf
    logp, ent, lse, ids, top = T.logprob_rows(z, [7], 2)
    assert (logp[0], ent[0], lse[0]) == (-np.inf, 0.0, -np.inf) and ids[0].tolist() == [-1, -1]
    logp, *_ = T.logprob_rows(z, [-100])
    assert logp[0] == 0


def test_logprob_of_two_tokens_is_the_logistic():
    z = np.array([[1.5, -0.25]], np.float32)
    logp, ent, *_ = T.logprob_rows(z, [1])
    p = 1 / (1 + np.exp(1.75))
    assert np.isclose(logp[0], np.log(p)) and np.isclose(ent[0], -p * np.log(p) - (1 - p) * np.log(1 - p))


def test_logprob_gradient_against_differences():
    """Differences of the float64 forward; lse and entropy enter the gradient
    as fp32, so it is good to about 1e-6."""
    rng = np.random.default_rng(5)
    rows, vocab, tau = 3, 11, 0.75
    x = rng.standard_normal((rows, vocab))
    scale = rng.uniform(0.5, 2, vocab).astype(np.float32)
    labels = np.array([2, -1, 10])
    g, gh = rng.standard_normal((2, rows))

    def f(v, s):
        total = 0.0
        for i in range(rows):
            z = v[i] * s * tau
            lse = np.log(np.exp(z).sum())
            p = np.exp(z - lse)
            total += gh[i] * -(p * (z - lse)).sum()
            if labels[i] >= 0:
                total += g[i] * (z[labels[i]] - lse)
        return total

    z = x * scale * tau
    lse = np.log(np.exp(z).sum(-1))
    ent = -(np.exp(z - lse[:, None]) * (z - lse[:, None])).sum(-1)
    dx, ds, unit, ds_unit, ds_mag = T.logprob_rows_backward(x, z, labels, lse, ent, g, gh, scale, tau)
    s64 = scale.astype(np.float64)
    for at in [(0, 2), (0, 5), (1, 0), (2, 10)]:
        assert np.isclose(dx[at], _difference(lambda v: f(v, s64), x, at, 1e-5), rtol=1e-5, atol=1e-7)
    for j in (0, 2, 10):
        assert np.isclose(ds[j], _difference(lambda u: f(x, u), s64, j, 1e-5), rtol=1e-5, atol=1e-7)
    assert np.allclose((dx / s64).sum(-1), 0, atol=1e-9)      # dz sums to zero over a row
