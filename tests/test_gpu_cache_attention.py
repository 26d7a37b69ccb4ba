"""ds_cache_attention_rows on the GPU against the float64 oracle.

Bounds.  With S the largest sum |scale q k| of a row's head and n the tokens it
sees, z is off by at most E = 2^-24 ((2 hd + 12) S): the dot product's hd
products and sums (twice, for the instruction's own order), the two scales, log2
e, the difference from the running maximum.  A weight exp(z) / sum is then off
by 2 E + 2^-24 (n + 96) relative to itself, for its own error and its sum's:
exp, the sums over n weights, the factors of at most 8 + log n joins.  The two
bf16 parts of a weight leave 2^-16 of it.  So out is off by sum p |v| times
(2 E + 2^-16 + 2^-24 (2 n + 96)), lse by E + 2^-24 (n + 96 + 4 |lse|); out adds
half a bf16 step.
"""
import math

import numpy as np
import pytest

from decode_util import Paged, random_pages
from gpu_util import announce
from oracle import decode_rows as D
from token_util import U, bf16_round, bits, close, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


class Case:
    def __init__(self, lens, heads, group, hd, page, seed, new=1, window=0, kind="bf16", order="token", extra=0, sd=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.window = np.array(lens, np.int32), new, window
        self.heads, self.nq, self.hd, self.page, self.kind, self.order = heads, heads * group, hd, page, kind, order
        per = max(1, -(-max(max(lens), 1) // page)) + extra
        self.n_pages = len(lens) * per + 2
        self.table = rng.permutation(self.n_pages)[:len(lens) * per].reshape(len(lens), per).astype(np.int32)
        self.k, self.v = random_pages(rng, (self.n_pages, page, heads, hd), kind)
        self.q = bf16_round(rng.standard_normal((len(lens) * new, self.nq * hd)) * sd)
        self.scales = rng.uniform(0.5, 2.0, (2, heads)).astype(np.float32) if kind == "e4m3" else (None, None)
        self.scale = hd ** -0.5

    def paged(self, B):
        return Paged(B, self.k, self.v, self.table, self.kind, self.order, *self.scales)

    def run(self, B, paged=None, **kw):
        import torch
        paged = paged or self.paged(B)
        got = B.ds_cache_attention_rows(paged.cache, dev(self.q, torch.bfloat16), dev(self.lens), scale=self.scale,
                                        window=self.window, want_lse=True, **kw)
        torch.cuda.synchronize()
        return got

    def check(self, got):
        out, lse, mag, big, seen = D.attention(self.q, self.k, self.v, self.table, self.lens, self.new, self.nq,
                                               self.window, self.scale, *self.scales)
        E = U * (2 * self.hd + 12) * big
        n = seen[:, None]
        close(host(got[1]), lse, E + U * (n + 96 + 4 * np.abs(np.where(np.isfinite(lse), lse, 0))), "lse")
        rel = np.repeat(2 * E + 2.0 ** -16 + U * (2 * n + 96), self.hd, axis=1)
        with np.errstate(invalid="ignore"):
            close(host(got[0]), out, rel * np.where(np.isfinite(mag), mag, 0), "out", bf16=True)
        return out, lse


# lens, kv heads, group, head_dim, page, new
CASES = [([1], 1, 1, 16, 1, 1), ([1, 0, 2], 2, 1, 32, 16, 1), ([37], 12, 1, 64, 16, 1), ([255, 256, 257], 2, 4, 128, 16, 1),
         ([700, 3, 31, 33], 4, 4, 256, 64, 1), ([100, 40], 1, 7, 80, 8, 1), ([513], 2, 16, 96, 32, 1),
         ([64, 900], 1, 17, 112, 128, 1), ([300], 1, 48, 48, 4, 1), ([90, 5, 1, 2, 0], 2, 4, 64, 16, 5),
         ([300, 16, 17], 3, 2, 160, 16, 16), ([50], 1, 1, 192, 2, 2), ([65, 1000], 2, 8, 240, 16, 3),
         ([129], 1, 5, 208, 1, 7), ([2000], 1, 1, 64, 4096, 2), ([40], 2, 3, 224, 16, 2), ([77], 1, 2, 144, 8, 4),
         ([60], 2, 6, 176, 16, 1)]


@pytest.mark.parametrize("kind,order", [("bf16", "token"), ("bf16", "head"), ("bf16", "both"), ("e4m3", "token"),
                                        ("e4m3", "head"), ("e4m3", "wide")])
@pytest.mark.parametrize("lens,heads,group,hd,page,new", CASES)
def test_attention(B, lens, heads, group, hd, page, new, kind, order):
    c = Case(lens, heads, group, hd, page, hd + page, new, kind=kind, order=order, extra=len(lens) % 2)
    announce("attention", lens, heads, group, hd, page, new, kind, order)
    c.check(c.run(B))


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 300, 10 ** 6])
@pytest.mark.parametrize("new,group,kind", [(1, 4, "bf16"), (5, 2, "e4m3"), (16, 3, "bf16")])
def test_window(B, window, new, group, kind):
    c = Case([700, 64, 1, 0, 33, 310], 2, group, 64, 16, window % 97 + new, new, window, kind)
    announce("attention in a window", window, new, group, kind)
    c.check(c.run(B))


@pytest.mark.parametrize("sd,kind", [(8.0, "bf16"), (40.0, "e4m3"), (0.01, "bf16")])
def test_peaked_and_flat_rows(B, sd, kind):
    c = Case([1500, 290], 2, 4, 128, 16, 3, 2, kind=kind, sd=sd)
    announce("attention of peaked rows", sd, kind)
    c.check(c.run(B))


def test_a_long_sequence_and_short_ones(B):
    """Past 128 chunks of 256 a chunk holds more blocks."""
    for kind in ("bf16", "e4m3"):
        c = Case([33500, 1, 4100], 1, 2, 32, 16, 4, 1, kind=kind)
        announce("attention over 33,500 tokens", kind)
        c.check(c.run(B))


def test_pages_that_are_none(B):
    c = Case([200, 64, 128, 40], 2, 4, 64, 16, 5, 3)
    c.table[0, 1], c.table[0, 5], c.table[0, 12] = -1, c.n_pages, 2 ** 31 - 1
    c.table[1, :] = -1
    c.table[2, 7] = -2 ** 31                                      # the newest page
    c.table[3, 0] = c.n_pages + 5
    announce("attention with pages that are none")
    out, lse = c.check(c.run(B))
    assert not out[3:6].any() and (lse[3:6] == -np.inf).all()
    c.window = 20
    c.check(c.run(B))


def test_lengths_outside_the_table(B):
    c = Case([64, 64, 64, 64], 1, 4, 32, 16, 6, 2)
    c.lens = np.array([-1, 65, 2 ** 31 - 1, -2 ** 31], np.int32)  # below 0 counts as 0, past the table as all of it
    announce("attention with lengths outside the table")
    c.check(c.run(B))
    c = Case([5, 9], 1, 1, 32, 16, 6, 1)
    c.table = c.table[:, :0]                                      # no pages a sequence
    out, lse = c.check(c.run(B))
    assert not out.any() and (lse == -np.inf).all()
    c = Case([5, 9], 1, 1, 32, 16, 6, 1)
    none = Paged(B, c.k[:0], c.v[:0], c.table)
    out, lse = c.run(B, none)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("kind,new,window", [("bf16", 1, 0), ("bf16", 5, 0), ("e4m3", 3, 40), ("bf16", 16, 7)])
def test_what_a_row_does_not_see_does_not_reach_it(B, bad, kind, new, window):
    """NaN or infinity in every token that no row sees, then in one that only
    the later new tokens see."""
    if kind == "e4m3":
        bad = np.nan                                              # the type has no infinities
    lens = [100, 33, 2, 300]
    c = Case(lens, 2, 3, 64, 16, 7, new, window, kind)
    clean = c.run(B)
    c.check(clean)
    k, v = c.k.copy(), c.v.copy()
    c.k[:], c.v[:] = bad, bad
    for s, n in enumerate(lens):
        for t in range(max(0, n - new - window + 1) if window else 0, n):
            p, o = D.token_place(c.table, c.n_pages, 16, s, t)
            c.k[p, o], c.v[p, o] = k[p, o], v[p, o]
    announce("attention beside", bad, kind, new, window)
    got = c.run(B)
    for x, y in zip(got, clean):
        assert np.array_equal(host(x), host(y))
    if new == 1:
        return
    last = D.token_place(c.table, c.n_pages, 16, 0, lens[0] - 1)
    c.k[last], c.v[last] = bad, bad
    got = c.run(B)
    for x, y in zip(got, clean):
        x, y = host(x), host(y)
        assert np.array_equal(x[:new - 1], y[:new - 1]) and np.array_equal(x[new:], y[new:])
        assert np.isnan(x[new - 1]).all()


@pytest.mark.parametrize("group,new,window", [(40, 2, 0), (17, 4, 50), (2, 9, 0)])
def test_a_new_token_does_not_reach_earlier_ones(B, group, new, window):
    """Heads of one token that fill tiles of their own, and tiles of several."""
    c = Case([200, 31], 1, group, 64, 16, 17, new, window)
    clean = [host(x) for x in c.run(B)]
    c.check(c.run(B))
    last = D.token_place(c.table, c.n_pages, 16, 0, 199)
    c.k[last], c.v[last] = np.nan, np.inf
    announce("attention of earlier tokens", group, new, window)
    got = [host(x) for x in c.run(B)]
    for x, y in zip(got, clean):
        assert np.array_equal(x[:new - 1], y[:new - 1]) and np.array_equal(x[new:], y[new:])
        assert np.isnan(x[new - 1]).all()


@pytest.mark.parametrize("lens", [[90, 33], [1700, 200]])
def test_values_whose_sums_overflow(B, lens):
    """V up to bf16's largest: their mean is finite, their sum is not."""
    c = Case(lens, 1, 4, 64, 16, 18, 2)
    clean = [host(x) for x in c.run(B)]
    c.v = bf16_round(np.sign(c.v) * np.minimum(np.abs(c.v), 1.0) * np.float32(3.38e38))
    c.v[..., :7] = np.float32(3.38e38)
    c.v = bf16_round(c.v)
    announce("attention over large values", lens)
    got = c.run(B)
    c.check(got)
    assert np.isfinite(host(got[0])).all() and np.array_equal(host(got[1]), clean[1])


def test_infinite_values_that_are_seen(B):
    """An infinity in V makes its dimension infinite, of its sign, for the rows
    that see it; infinities of both signs make NaN; others keep their bits."""
    c = Case([300, 90], 1, 4, 64, 16, 8, 2)
    clean = [host(x) for x in c.run(B)]
    at = lambda s, t: D.token_place(c.table, c.n_pages, 16, s, t)  # noqa: E731
    c.v[at(0, 7)][..., 3] = np.inf
    c.v[at(0, 280)][..., 5] = -np.inf
    c.v[at(0, 299)][..., 9] = np.inf                              # the newest: its own row alone
    c.v[at(0, 20)][..., 11], c.v[at(0, 21)][..., 11] = np.inf, -np.inf
    announce("attention over infinite values")
    got = [host(x) for x in c.run(B)]
    out = got[0].reshape(4, 4, 64)
    assert (out[:2, :, 3] == np.inf).all() and (out[:2, :, 5] == -np.inf).all() and np.isnan(out[:2, :, 11]).all()
    assert (out[1, :, 9] == np.inf).all() and np.isfinite(out[0, :, 9]).all()
    assert np.array_equal(got[1], clean[1]) and np.array_equal(got[0][2:], clean[0][2:])
    want, lse, mag, big, seen = D.attention(c.q, c.k, c.v, c.table, c.lens, 2, 4, 0, c.scale)
    fine = np.isfinite(want)
    rel = np.repeat(4 * U * (2 * 64 + 12) * big + 2.0 ** -8, 64, axis=1)   # P in one part beside an infinity
    assert (np.abs(got[0] - want)[fine] <= (rel * mag + 2.0 ** -8 * np.abs(want))[fine]).all()


@pytest.mark.parametrize("kind,new,group,window", [("e4m3", 1, 3, 0), ("e4m3", 5, 6, 200), ("bf16", 2, 9, 333)])
def test_a_nan_in_a_seen_value_is_its_dimensions(B, kind, new, group, window):
    """... for the rows that see it, over several chunks and tiles."""
    c = Case([700, 150], 2, group, 80, 16, 19, new, window, kind)
    for t in (600, 690, 699):
        c.v[D.token_place(c.table, c.n_pages, 16, 0, t)][..., t % 80] = np.nan
    announce("attention over a NaN in V", kind, new, group, window)
    got = c.run(B)
    with np.errstate(invalid="ignore"):
        want = D.attention(c.q, c.k, c.v, c.table, c.lens, new, c.nq, window, c.scale, *c.scales)[0]
    assert np.array_equal(np.isnan(host(got[0])), np.isnan(want)) and np.isnan(want).any() and not np.isnan(want).all()
    out, lse = c.check(got)
    assert np.isfinite(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_lse_of_one_score_is_rounded_twice(B, kind):
    """One product a score and one token a row: z is off by the rounding of z
    log2 e (1 unit of 2^-24 of it), the result by its own (1)."""
    c = Case([1] * 60, 2, 4, 64, 16, 21, kind=kind)
    rng = np.random.default_rng(22)
    q = np.zeros((60, 8, 64), np.float32)
    at = rng.integers(0, 64, (60, 8))
    np.put_along_axis(q, at[..., None], bf16_round(rng.standard_normal((60, 8, 1)) * 9), 2)
    c.q, c.scale = q.reshape(60, 512), 0.1171875 * 1.1
    announce("lse of single scores", kind)
    got = host(c.run(B)[1])
    c.check(c.run(B))
    lse = D.attention(c.q, c.k, c.v, c.table, c.lens, 1, 8, 0, c.scale, *c.scales)[1]
    assert (np.abs(got - lse) <= 2.001 * U * np.abs(lse) + 1e-30).all()


def test_many_empty_sequences(B):
    c = Case([0] * 1500 + [70] + [0] * 37, 1, 2, 32, 16, 20, 1)
    announce("attention of 1,537 sequences and hardly a token")
    out, lse = c.check(c.run(B))
    assert not out[:1500].any() and out[1500].any() and (lse[1501:] == -np.inf).all()


def test_scores_that_are_all_minus_infinity(B):
    """Keys of -infinity (a mask written into the cache) leave nothing; some do
    not matter beside others; a scale of 0 gives the mean."""
    c = Case([40, 40, 40], 1, 2, 32, 16, 9)
    c.q = np.abs(c.q) + np.float32(0.5)
    c.q = bf16_round(c.q)
    for s, ts in ((0, range(40)), (1, range(0, 40, 2))):
        for t in ts:
            c.k[D.token_place(c.table, c.n_pages, 16, s, t)] = -np.inf
    announce("attention over keys of -infinity")
    out, lse = c.check(c.run(B))
    assert not out[0].any() and (lse[0] == -np.inf).all() and np.isfinite(lse[1:]).all()
    c = Case([40], 1, 2, 32, 16, 9)
    c.scale = 0.0
    c.check(c.run(B))
    c.scale = -0.3
    c.check(c.run(B))


def test_a_nan_in_q_is_its_own_rows(B):
    c = Case([300, 300], 2, 4, 64, 16, 10, 2)
    clean = [host(x) for x in c.run(B)]
    c.q[1, 64 * 3 + 5] = np.nan                                   # sequence 0, new token 1, head 3
    announce("attention of a NaN in q")
    got = [host(x) for x in c.run(B)]
    out, was = got[0].reshape(4, 8, 64), clean[0].reshape(4, 8, 64)
    assert np.isnan(out[1, 3]).all() and np.isnan(got[1][1, 3])
    keep = np.ones((4, 8), bool)
    keep[1, 3] = False
    assert np.array_equal(out[keep], was[keep]) and np.array_equal(got[1][keep], clean[1][keep])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_do_not_depend_on_the_batch(B, kind):
    """A sequence alone, in other pages, under a wider table, its tokens one by
    one and several at once: the same bits."""
    lens = [700, 40, 300, 1]
    c = Case(lens, 2, 4, 128, 16, 11, 3, kind=kind)
    whole = c.run(B)
    announce("attention row by row", kind)
    for s in (0, 1, 3):
        one = Case([lens[s]], 2, 4, 128, 16, 12, 3, kind=kind, extra=5)
        one.scales = c.scales
        for t in range(lens[s]):
            a, b = D.token_place(c.table, c.n_pages, 16, s, t), D.token_place(one.table, one.n_pages, 16, 0, t)
            one.k[b], one.v[b] = c.k[a], c.v[a]
        one.q = c.q[s * 3:s * 3 + 3]
        got = one.run(B)
        for x, y in zip(got, whole):
            assert np.array_equal(host(x), host(y)[s * 3:s * 3 + 3])
        one.new, one.q = 1, one.q[2:]                             # the newest token alone
        for x, y in zip(one.run(B), whole):
            assert np.array_equal(host(x), host(y)[s * 3 + 2:s * 3 + 3])


def test_strided_rows_and_no_lse(B):
    import torch
    c = Case([90, 300], 2, 3, 64, 16, 13, 2)
    want = c.run(B)
    paged = c.paged(B)
    wide = torch.full((4, 6 * 64 + 40), 3.0, dtype=torch.bfloat16, device="cuda:0")
    wide[:, :384] = dev(c.q, torch.bfloat16)
    to = torch.full((4, 6 * 64 + 8), 3.0, dtype=torch.bfloat16, device="cuda:0")
    announce("attention of strided rows")
    got = B.ds_cache_attention_rows(paged.cache, wide[:, :384], dev(c.lens), out=to[:, :384])
    torch.cuda.synchronize()
    assert got.data_ptr() == to.data_ptr() and torch.equal(bits(to[:, :384].contiguous()), bits(want[0]))
    assert bool((to[:, 384:] == 3.0).all())
    narrow = B.KvCache(paged.k, paged.v, dev(np.pad(c.table, ((0, 0), (0, 9)), constant_values=-1))[:, :c.table.shape[1]])
    got = B.ds_cache_attention_rows(narrow, wide[:, :384], dev(c.lens))
    torch.cuda.synchronize()
    assert torch.equal(bits(got), bits(want[0]))


def test_offsets_past_32_bits(B):
    import torch
    stride = (3 << 29) // 2                                       # elements: pages 1.5 GiB apart
    half = 3 * stride + 4096
    buf = torch.empty(2 * half, dtype=torch.bfloat16, device="cuda:0")
    c = Case([60], 2, 2, 32, 16, 14)
    c.table[0] = [3, 0, 2, 1]
    c.k, c.v = c.k[:4], c.v[:4]
    k, v = (buf[i * half:].as_strided((4, 16, 2, 32), (stride, 64, 32, 1)) for i in (0, 1))
    k.copy_(dev(c.k, torch.bfloat16))
    v.copy_(dev(c.v, torch.bfloat16))
    c.n_pages = 4
    announce("attention past 4 GiB")
    got = B.ds_cache_attention_rows(B.KvCache(k, v, dev(c.table)), dev(c.q, torch.bfloat16), dev(c.lens), want_lse=True)
    torch.cuda.synchronize()
    c.check(got)


def test_many_sequences(B):
    """More (row, head) pairs than workgroups at once, lengths of all kinds."""
    rng = np.random.default_rng(15)
    c = Case(rng.integers(0, 40, 700).tolist(), 2, 2, 32, 8, 15, 1)
    announce("attention of 700 sequences")
    c.check(c.run(B))


def test_no_sequences(B):
    import torch
    c = Case([3], 1, 2, 32, 4, 16)
    cache = B.KvCache(dev(c.k, torch.bfloat16), dev(c.v, torch.bfloat16), torch.empty(0, 4, dtype=torch.int32, device="cuda:0"))
    out, lse = B.ds_cache_attention_rows(cache, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda:0"),
                                         torch.empty(0, dtype=torch.int32, device="cuda:0"), want_lse=True)
    assert out.shape == (0, 64) and lse.shape == (0, 2)
