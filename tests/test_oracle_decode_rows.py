"""The decoding step's float64 oracle, pinned without restating it: closed
forms, central differences for the gradient, and identities."""
import math

import numpy as np
import pytest

from oracle import decode_rows as D


def test_e4m3_values():
    import torch
    v = D.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    assert np.nanmax(v) == D.E4M3_MAX and v[1] == 2.0 ** -9


def test_frequencies():
    assert np.allclose(D.frequencies(8), [1, 0.1, 0.01, 0.001])
    f, g = D.frequencies(64), D.frequencies(64, factor=8, original=4096, low=1, high=32)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 8)
    assert (np.diff(g) < 0).all() and (g <= f).all() and (g >= f / 8 * (1 - 1e-15)).all()
    assert np.allclose(D.frequencies(16, factor=4), D.frequencies(16) / 4)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [2, 6, 16, 48])
def test_rope_turns_pairs(rotary, interleaved):
    rng = np.random.default_rng(rotary)
    x = rng.standard_normal((3, 2 * 48))
    inv = D.frequencies(rotary).astype(np.float32)
    y, mag = D.rope_heads(x, np.array([0, 5, 10 ** 6]), inv, 48, interleaved)
    assert np.array_equal(y[0], x[0])                       # position 0
    h, g = x.reshape(3, 2, 48), y.reshape(3, 2, 48)
    assert np.array_equal(h[:, :, rotary:], g[:, :, rotary:])
    assert np.allclose((h ** 2).sum(-1), (g ** 2).sum(-1))  # a rotation
    assert (np.abs(y - x) <= 2 * mag + 1e-12).all()
    # relative positions: <turn_a q, turn_b k> goes by b - a
    q, k = rng.standard_normal((2, 1, 48))
    dots = [(D.rope_heads(q, np.array([a]), inv, 48, interleaved)[0]
             * D.rope_heads(k, np.array([a + 7]), inv, 48, interleaved)[0]).sum() for a in (0, 3, 1000)]
    assert np.allclose(dots, dots[0])


def test_rope_quarter_turn():
    inv = np.zeros(4, np.float32)
    inv[1] = np.float32(np.pi / 2)
    x = np.arange(1, 17, dtype=np.float64)[None]
    y, _ = D.rope_heads(x, np.array([1]), inv, 16, amplitude=2.0)
    want = x[0].copy()
    want[:8] *= 2
    want[1], want[5] = -2 * x[0, 5], 2 * x[0, 1]
    assert np.allclose(y[0], want, atol=1e-5)
    y, _ = D.rope_heads(x, np.array([1]), inv, 16, True, 2.0)
    want = x[0].copy()
    want[:8] *= 2
    want[2], want[3] = -2 * x[0, 3], 2 * x[0, 2]
    assert np.allclose(y[0], want, atol=1e-5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient_against_differences(interleaved):
    rng = np.random.default_rng(4)
    x, dy = rng.standard_normal((2, 2, 32))
    pos, inv = np.array([3, 70]), D.frequencies(10).astype(np.float32)
    f = lambda v: (D.rope_heads(v, pos, inv, 16, interleaved, 1.3)[0] * dy).sum()  # noqa: E731
    dx, _ = D.rope_heads(dy, pos, inv, 16, interleaved, 1.3, back=True)
    for at in [(0, 0), (1, 4), (0, 9), (1, 17), (1, 31)]:
        hi, lo = x.copy(), x.copy()
        hi[at] += 1e-5
        lo[at] -= 1e-5
        assert np.isclose((f(hi) - f(lo)) / 2e-5, dx[at], rtol=1e-7, atol=1e-8)


def test_places_and_what_is_visible():
    table = np.array([[4, -1], [0, 9]], np.int32)
    assert D.token_place(table, 5, 8, 0, 7) == (4, 7) and D.token_place(table, 5, 8, 1, 3) == (0, 3)
    for seq, token in ((0, 8), (1, 8), (0, 16), (0, -1), (2, 0), (-1, 0)):
        assert D.token_place(table, 5, 8, seq, token) is None
    assert list(D.visible(5, 2, 0, 0, 16)) == [0, 1, 2, 3] and list(D.visible(5, 2, 1, 0, 16)) == [0, 1, 2, 3, 4]
    assert list(D.visible(5, 2, 1, 2, 16)) == [3, 4] and list(D.visible(1, 3, 0, 0, 16)) == []
    assert list(D.visible(99, 1, 0, 0, 16)) == list(range(16)) and list(D.visible(-3, 1, 0, 0, 16)) == []


def test_attention_of_one_and_of_equal_keys():
    rng = np.random.default_rng(5)
    k, v = rng.standard_normal((2, 3, 4, 2, 16))
    table = np.array([[2, 0, 1]], np.int32)
    q = rng.standard_normal((1, 4 * 16))
    out, lse, mag, big, seen = D.attention(q, k, v, table, np.array([1]), 1, 4, 0, 0.25)
    assert seen[0] == 1
    for g in range(4):                                      # one key: its value, and its z
        assert np.allclose(out.reshape(4, 16)[g], v[2, 0, g // 2])
        assert np.isclose(lse[0, g], 0.25 * k[2, 0, g // 2] @ q.reshape(4, 16)[g])
    out, lse, *_ = D.attention(0 * q, k, v, table, np.array([7]), 1, 4, 0, 0.25)
    want = np.concatenate([v[2], v[0, :3]])                 # equal keys: the mean
    assert np.allclose(out.reshape(4, 16)[3], want[:, 1].mean(0)) and np.allclose(lse, math.log(7))
    out, lse, *_ = D.attention(q, k, v, table, np.array([0]), 1, 4, 0, 0.25)
    assert not out.any() and (lse == -np.inf).all()


def test_attention_against_a_softmax_of_everything():
    import torch
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((2, 6, 4, 1, 16))
    table = np.array([[3, 5, -1, 0]], np.int32)
    q = rng.standard_normal((3, 16))
    out, lse, mag, _, seen = D.attention(q, k, v, table, np.array([15]), 3, 1, 9, 1.0)
    flat_k, flat_v = (np.concatenate([x[3], x[5], np.full((4, 1, 16), np.nan), x[0]])[:, 0] for x in (k, v))
    for j in range(3):
        keys = [t for t in range(12 + j + 1) if t > 12 + j - 9 and not 8 <= t < 12]
        z = torch.from_numpy(flat_k[keys] @ q[j])
        assert np.isclose(lse[j, 0], torch.logsumexp(z, 0).item()) and seen[j] == len(keys)
        assert np.allclose(out[j], torch.softmax(z, 0).numpy() @ flat_v[keys])
        assert (mag[j] >= np.abs(out[j]) - 1e-12).all()


@pytest.mark.parametrize("certain", [False, True])
def test_verified_tokens_have_the_target_distribution(certain):
    """Over all random numbers, drafts drawn from q give tokens drawn from p:
    the chance of token j is sum_d q(d) [accept_d 1(j = d) + refuse_d w_j / sum w]."""
    rng = np.random.default_rng(7)
    zt, zd = rng.standard_normal((2, 6)).astype(np.float32) * 2
    zt[3] = -np.inf
    p, _ = D.probabilities(zt)
    q = np.eye(6)[4] if certain else D.probabilities(zd)[0]
    steps = 400
    us = (np.arange(steps) + 0.5) / steps
    got = np.zeros(6)
    for d in range(6):
        if q[d] == 0:
            continue
        first = np.array([D.verify_sequence(np.stack([zt, zt]), None if certain else zd[None], [d], [u], 0.5)[0]
                          for u in us], dtype=object)
        accept = np.mean([len(t) == 2 for t in first])
        assert abs(accept - min(1, p[d] / q[d])) <= 1 / steps
        refused = [u for u, t in zip(us, first) if len(t) == 1]
        got[d] += q[d] * accept
        if refused:
            picks = [D.verify_sequence(np.stack([zt, zt]), None if certain else zd[None], [d], [refused[0]], u)[0][0]
                     for u in us]
            got += q[d] * (1 - accept) * np.bincount(picks, minlength=6) / steps
    assert np.abs(got - p).max() < 3 / steps and got[3] == 0


def test_verify_ends():
    z = np.zeros((3, 4), np.float32)
    assert D.verify_sequence(z, None, [1, 2], [0.0, 0.0], 0.6)[0] == [1, 2, 2]
    assert D.verify_sequence(z, None, [1, -1], [0.0, 0.0], 0.0)[0] == [1, 0]
    assert D.verify_sequence(z, None, [1, 2], [0.3, 0.0], 0.0)[0] == [0]           # 0.3 >= 1/4
    assert D.verify_sequence(z, None, [0, 2], [0.3, 0.0], 0.0)[0] == [1]           # the refused one is off
    assert D.verify_sequence(z, None, [0, 2], [0.3, 0.0], 2.0)[0] == [3]
    assert D.verify_sequence(z, None, [0, 2], [0.3, 0.0], math.nan)[0] == [3]
    bad = z.copy()
    bad[0, 1] = np.nan
    assert D.verify_sequence(bad, None, [0, 2], [0.0, 0.0], 0.0)[:2] == ([-1], [0.0])
    assert D.verify_sequence(z, bad[:2], [0, 2], [0.0, 0.0], 0.0)[0] == [0]        # no q: from p
    t, lp, _ = D.verify_sequence(z, z[:2], [3, 2], [0.99, 0.99], 0.5)
    assert t == [3, 2, 2] and np.allclose(lp, -math.log(4))
