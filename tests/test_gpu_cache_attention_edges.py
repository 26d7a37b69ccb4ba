"""ds_cache_attention_rows on the GPU where its numerics and its cuts have edges,
against the float64 oracle, beside the cases of test_gpu_cache_attention.py.

Bounds as there, without the 2^-16 that weights of 16 bits would leave: z off by
E = 2^-24 (2 hd + 12) S, a weight by 2 E + 2^-24 (n + 96), out by sum p |v| times
(2 E + 2^-24 (2 n + 96)).
"""
import numpy as np
import pytest

from gpu_util import announce
from oracle import decode_rows as D
from test_gpu_cache_attention import Case
from token_util import U, bf16_round, close, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


def near(got, want, rel):
    """Each bf16 value is one that a value within rel of `want` rounds to."""
    lo, hi = bf16_round(want * (1 - rel)), bf16_round(want * (1 + rel))
    bad = (got < np.minimum(lo, hi)) | (got > np.maximum(lo, hi))
    assert not bad.any(), f"{bad.sum()} of {bad.size} beyond {rel:.3g}"


@pytest.mark.parametrize("kind,group", [("bf16", 4), ("bf16", 20), ("e4m3", 4), ("e4m3", 20)])
def test_weights_keep_the_bits_of_fp32(B, kind, group):
    """Two tokens a sequence, the first of score 0 and value 0, the second's score
    z one exact product in [-4, 0): out = v w / (1 + w), w = exp z, rounded once.
    In units of 2^-24 of it: z log2 e (2 |z|: the constant, the product), exp (2),
    w times v in the matrix instruction (4), 1 + w, its reciprocal, the product, v's
    scale (1 each), and 1 for `near`: at most 8 + 2 + 4 + 4 + 1 = 19.  Weights of 16
    bits would be up to 128 off, which moves about one of 2,000 outputs."""
    rng = np.random.default_rng(30 + group)
    heads, hd, seqs = 4, 64, 60
    c = Case([2] * seqs, heads, group, hd, 16, 31, kind=kind)
    c.scale = 1.0
    if kind == "e4m3":
        c.scales = np.ones((2, heads), np.float32)
    c.k[:], c.v[:] = 0, 0
    for s in range(seqs):
        page, off = D.token_place(c.table, c.n_pages, 16, s, 1)
        c.k[page, off, :, 0] = 0.125 * rng.integers(1, 9, heads)  # exact in either type
        c.v[page, off] = (8 + rng.integers(0, 8, (heads, hd))) * 0.125
    q = np.zeros((seqs, heads * group, hd))
    q[:, :, 0] = -rng.uniform(0.25, 4, (seqs, heads * group))
    c.q = bf16_round(q.reshape(seqs, -1))
    announce("attention of two tokens", kind, group)
    got = c.run(B)
    out, _ = c.check(got)
    near(host(got[0]), out, 19 * U)


def test_a_tiny_scale_of_values_costs_no_bits(B):
    """Two tokens a sequence as above, w v times a scale of 1e-40: in units of 2^-24
    at most 19, and 1 for one product more.  The scale over 1 + w has 16 bits."""
    rng = np.random.default_rng(32)
    heads, group, hd, seqs = 4, 4, 64, 60
    c = Case([2] * seqs, heads, group, hd, 16, 33, kind="e4m3")
    c.scale = 1.0
    c.scales = np.ones(heads, np.float32), np.full(heads, 1e-40, np.float32)
    c.k[:], c.v[:] = 0, 0
    for s in range(seqs):
        page, off = D.token_place(c.table, c.n_pages, 16, s, 1)
        c.k[page, off, :, 0] = 0.125 * rng.integers(1, 9, heads)
        c.v[page, off] = (8 + rng.integers(0, 7, (heads, hd))) * 32.0  # 256 to 448
    q = np.zeros((seqs, heads * group, hd))
    q[:, :, 0] = -rng.uniform(0.0, 0.5, (seqs, heads * group))
    c.q = bf16_round(q.reshape(seqs, -1))
    announce("attention of values of a tiny scale")
    out = D.attention(c.q, c.k, c.v, c.table, c.lens, 1, c.nq, 0, c.scale, *c.scales)[0]
    fine = out > 2.0 ** -126                                      # (bf16 has fewer bits below)
    assert fine.mean() > 0.5
    got = host(c.run(B)[0])
    near(got[fine], out[fine], 20 * U)


@pytest.mark.parametrize("scale", [np.inf, np.nan])
def test_rows_that_see_nothing_are_zeros_under_any_scale(B, scale):
    """Of one chunk, of several, and of a length without pages."""
    c = Case([0, 40, 700, 300], 2, 4, 64, 16, 34, kind="e4m3")
    c.table[1:3] = -1
    c.scales = tuple(np.full(2, scale, np.float32) for _ in "kv")
    announce("attention of nothing under a scale of", scale)
    out, lse = (host(x) for x in c.run(B))
    assert not out[:3].any() and (lse[:3] == -np.inf).all() and np.isnan(out[3]).all()


def check(c, got):
    out, lse, mag, big, seen = D.attention(c.q, c.k, c.v, c.table, c.lens, c.new, c.nq, c.window, c.scale, *c.scales)
    E, n = U * (2 * c.hd + 12) * big, seen[:, None]
    close(host(got[1]), lse, E + U * (n + 96 + 4 * np.abs(np.where(np.isfinite(lse), lse, 0))), "lse")
    rel = np.repeat(2 * E + U * (2 * n + 96), c.hd, axis=1)
    with np.errstate(invalid="ignore"):
        fine = np.isfinite(out)
        close(np.where(fine, host(got[0]), 0), np.where(fine, out, 0), np.where(fine, rel * mag, 0), "out", bf16=True)
    return out


# kv heads, lengths: keys times heads about 65,536, where a least chunk goes from
# 128 keys to 256, and about 128 chunks of either, past which chunks hold more
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,window", [(1, 0), (3, 0), (2, 8192), (5, 8189)])
@pytest.mark.parametrize("heads,lens", [(8, [8191, 8192, 8193, 5]), (8, [33000, 8190, 32767, 32769]),
                                        (4, [16383, 16384, 16385, 16400]), (3, [21845, 21846, 300])])
def test_where_the_cut_changes(B, heads, lens, new, window, kind):
    c = Case(lens, heads, 2, 32, 64, 35 + heads, new, window, kind)
    announce("attention where the cut changes", heads, lens, new, window, kind)
    got = c.run(B)
    check(c, got)
    for s in (0, len(lens) - 1):                                  # alone, under its own table: the same bits
        one = Case([lens[s]], heads, 2, 32, 64, 1, new, window, kind)
        per = one.table.shape[1]
        one.k, one.v, one.scales, one.q = c.k, c.v, c.scales, c.q[s * new:(s + 1) * new]
        one.table, one.n_pages = c.table[s:s + 1, :per], c.n_pages
        for x, y in zip(one.run(B), got):
            assert np.array_equal(host(x), host(y)[s * new:(s + 1) * new])


@pytest.mark.parametrize("lens", [[300, 90], [1700, 1100]])
def test_rows_beside_infinite_values_are_as_exact_as_others(B, lens):
    """They are summed again by themselves, one key at a time, in fp32."""
    c = Case(lens, 1, 4, 64, 16, 36, 2)
    at = lambda s, t: D.token_place(c.table, c.n_pages, 16, s, t)  # noqa: E731
    c.v[at(0, 7)][..., 3] = np.inf
    c.v[at(0, lens[0] - 20)][..., 5] = -np.inf
    c.v[at(0, lens[0] - 1)][..., 9] = np.inf                      # the newest: its own row alone
    c.v[at(0, 20)][..., 11], c.v[at(0, 21)][..., 11] = np.inf, -np.inf
    announce("attention beside infinite values", lens)
    got = c.run(B)
    out = check(c, got)
    assert np.array_equal(np.isfinite(host(got[0])), np.isfinite(out)) and not np.isfinite(out[:2]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group,new", [(7, 5), (3, 11), (16, 3), (5, 16), (40, 1)])
def test_rows_of_several_groups(B, group, new, kind):
    """33 to 80 rows a kv head: two or three groups of two row tiles, the last of
    them not full."""
    c = Case([1500, 40, 0, 300], 2, group, 64, 16, 37 + group, new, kind=kind)
    announce("attention of rows of several groups", group, new, kind)
    check(c, c.run(B))


@pytest.mark.parametrize("kind,group,new,window", [("bf16", 4, 5, 0), ("e4m3", 4, 5, 0), ("bf16", 7, 5, 0), ("bf16", 3, 16, 0),
                                                   ("e4m3", 40, 2, 0)])
def test_a_newest_token_alone_has_the_same_bits(B, kind, group, new, window):
    """In one row tile, among several tokens in two, and in several groups."""
    lens = [700, 90, 33]
    c = Case(lens, 2, group, 96, 16, 38, new, window, kind)
    announce("attention of a newest token alone", kind, group, new)
    whole = [host(x) for x in c.run(B)]
    c.q, c.new = c.q.reshape(3, new, -1)[:, -1].copy(), 1
    for x, y in zip(c.run(B), whole):
        assert np.array_equal(host(x), y.reshape(3, new, -1)[:, -1])


def test_values_below_the_normal_range(B):
    """bf16 values under 2^-126 count as what they are, in one chunk and several."""
    c = Case([40, 600], 1, 4, 64, 16, 39)
    c.v = np.float32(2.0 ** -130) * np.clip(np.round(c.v * 2), -8, 8)
    announce("attention of values below the normal range")
    out, lse, mag, big, seen = D.attention(c.q, c.k, c.v, c.table, c.lens, 1, 4, 0, c.scale)
    got = host(c.run(B)[0]).astype(np.float64)
    bound = np.repeat(2 * U * (2 * 64 + 12) * big + U * (2 * seen[:, None] + 96), 64, axis=1) * mag
    # fp32's step below its normal range is 2^-149, bf16's 2^-133: half of that one, and
    # half of the other for each of a key's three products, with room for their join
    assert (np.abs(got - out) <= bound + 2.0 ** -134 + 2 * 600 * 2.0 ** -149).all()
