"""ds_cache_append_rows on the GPU against the float64 oracle.

Bounds as of ds_qk_rows_rms' forward (48 units of 2^-24 of an element's two
terms: the norm, the weight, the turn), with the amplitude (1) and, in e4m3,
the division by the scale (2): under 52.  Stored values add half a step of
their type.  Everything else that the cache's buffers hold must stay bit for
bit.
"""
import numpy as np
import pytest

from decode_util import HALF_E4M3, LEAST_E4M3, Paged, random_pages, values_of
from gpu_util import announce
from oracle import decode_rows as D
from token_util import HALF_BF16, U, bf16_round, bits, close, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


class Case:
    """`new` tokens of each sequence, from what each holds already."""

    def __init__(self, new, heads, nq, hd, rotary, page, seed, kind="bf16", interleaved=False, rms=True, amplitude=1.0):
        rng = np.random.default_rng(seed)
        self.kind, self.interleaved, self.rms, self.amplitude = kind, interleaved, rms, amplitude
        self.heads, self.nq, self.hd, self.page, self.n_seqs = heads, nq, hd, page, len(new)
        before = rng.integers(0, 3 * page + 40, len(new))
        self.seqs = np.repeat(np.arange(len(new)), new).astype(np.int32)
        self.pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)]).astype(np.int32) \
            if sum(new) else np.zeros(0, np.int32)
        order = rng.permutation(len(self.pos))                    # rows of a batch in no order
        self.seqs, self.pos = self.seqs[order], self.pos[order]
        per = int(-(-(before + np.array(new)).max() // page)) + 1
        self.n_pages = len(new) * per + 2
        self.table = rng.permutation(self.n_pages)[:len(new) * per].reshape(len(new), per).astype(np.int32)
        rows = len(self.pos)
        r = lambda n: bf16_round(rng.standard_normal((rows, n * hd)))  # noqa: E731
        self.q, self.k, self.v = r(nq), r(heads), r(heads)
        self.inv = D.frequencies(rotary).astype(np.float32) if rotary else None
        self.qw, self.kw = (rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32) if rms else (None, None))
        self.scales = rng.uniform(0.02, 2.0, (2, heads)).astype(np.float32) if kind == "e4m3" else (None, None)
        self.was = random_pages(rng, (self.n_pages, page, heads, hd), kind)

    def paged(self, B, order="token"):
        return Paged(B, *self.was, self.table, self.kind, order, *self.scales)

    def run(self, B, paged, **over):
        import torch
        b = torch.bfloat16
        opt = lambda a: None if a is None else dev(a)  # noqa: E731
        kw = dict(seqs=dev(self.seqs), inv_freq=opt(self.inv), interleaved=self.interleaved, amplitude=self.amplitude,
                  q=dev(self.q, b) if self.nq else None, rms_eps=1e-6 if self.rms else None,
                  q_weight=opt(self.qw) if self.nq else None, k_weight=opt(self.kw))
        kw.update(over)
        q = B.ds_cache_append_rows(paged.cache, dev(self.k, b), dev(self.v, b), dev(self.pos), **kw)
        torch.cuda.synchronize()
        return q

    def heads_of(self, x, w):
        n = D.normed_heads(x, w, self.hd, 1e-6) if self.rms else x.astype(np.float64)
        if self.inv is None:
            return n, np.abs(n)
        y, mag = D.rope_heads(n, self.pos, self.inv, self.hd, self.interleaved, self.amplitude)
        return y, np.maximum(mag, np.abs(y)) if self.rms else mag

    def check(self, paged, q_out):
        if q_out is not None:
            want, mag = self.heads_of(self.q, self.qw)
            close(host(q_out), want, 52 * U * mag, "q", bf16=True)
        stored = {}
        for row, (s, p) in enumerate(zip(self.seqs, self.pos)):
            at = D.token_place(self.table, self.n_pages, self.page, int(s), int(p))
            if at is not None:
                assert at not in stored, "the case writes a token twice"
                stored[at] = row
        k, kmag = self.heads_of(self.k, self.kw)
        for t, was, new, mag, scale, name in ((paged.k, self.was[0], k, kmag, self.scales[0], "k"),
                                              (paged.v, self.was[1], self.v.astype(np.float64), 0 * kmag,
                                               self.scales[1], "v")):
            got = values_of(t)
            rest = np.ones(got.shape[:2], bool)
            for (page, off), row in stored.items():
                rest[page, off] = False
                x, m = new[row].reshape(-1, self.hd), mag[row].reshape(-1, self.hd)
                if self.kind == "e4m3":
                    x, m = np.clip(x / scale[:, None], -D.E4M3_MAX, D.E4M3_MAX), m / scale[:, None]
                    bound = 52 * U * m * (1 + HALF_E4M3) + 3 * U * np.abs(x) + np.maximum(HALF_E4M3 * np.abs(x), LEAST_E4M3)
                else:
                    bound = 52 * U * m * (1 + HALF_BF16) + HALF_BF16 * np.abs(x)
                close(got[page, off], x, bound, f"{name} of row {row}")
            assert np.array_equal(got[rest], was.astype(np.float64)[rest]), f"{name}: other tokens changed"


# new tokens, kv heads, q heads, head_dim, rotary, page
CASES = [([1], 1, 1, 16, 16, 1), ([1] * 9, 4, 16, 256, 256, 16), ([5, 0, 33, 1], 2, 6, 80, 20, 8),
         ([17, 40], 8, 8, 128, 64, 16), ([3, 3, 3], 3, 0, 64, 64, 4), ([100], 1, 7, 96, 96, 64),
         ([2, 9], 12, 12, 64, 0, 32), ([6], 5, 5, 48, 34, 128), ([2, 2], 2, 8, 240, 126, 2)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("order,interleaved,rms", [("token", False, True), ("head", True, True), ("both", False, False),
                                                   ("wide", True, False)])
@pytest.mark.parametrize("new,heads,nq,hd,rotary,page", CASES)
def test_append(B, new, heads, nq, hd, rotary, page, order, interleaved, rms, kind):
    c = Case(new, heads, nq, hd, rotary, page, hd + page, kind, interleaved, rms, amplitude=1.0 if rms else 1.125)
    announce("append", new, heads, nq, hd, rotary, page, order, kind, interleaved, rms)
    paged = c.paged(B, order)
    gaps = None if paged.store is None else paged.bits()[0].copy()
    c.check(paged, c.run(B, paged))
    if order == "wide":
        after = paged.bits()[0]
        inside = np.zeros(gaps.shape, bool)
        inside[:, :, :-1, :-1, :-16] = True
        assert np.array_equal(after[~inside], gaps[~inside]), "between the tokens"


def test_rows_outside_the_cache_store_nothing(B):
    import torch
    c = Case([20, 20, 20], 2, 4, 64, 64, 8, 3)
    c.pos[:4] = -1, -2 ** 31, 2 ** 31 - 1, c.table.shape[1] * c.page
    c.seqs[4:8] = -1, 3, 2 ** 31 - 1, -2 ** 31
    c.table[1, :2] = -1
    c.table[2, 1] = c.n_pages
    c.table[2, 2] = 2 ** 31 - 1
    c.table[0, 0] = -2 ** 31
    for order in ("token", "head"):
        announce("append outside the cache", order)
        paged = c.paged(B, order)
        c.check(paged, c.run(B, paged))
    # no pages at all
    none = Paged(B, *(w[:0] for w in c.was), c.table)
    q = c.run(B, none)
    want, mag = c.heads_of(c.q, c.qw)
    close(host(q), want, 52 * U * mag, "q", bf16=True)
    assert none.k.numel() == 0 and torch.isfinite(q.float()).all()


def test_equal_shares_of_the_sequences(B):
    c = Case([4, 4, 4], 2, 4, 64, 32, 16, 5)
    order = np.argsort(c.seqs, kind="stable")                     # rows of a sequence together
    c.seqs, c.pos, c.q, c.k, c.v = (x[order] for x in (c.seqs, c.pos, c.q, c.k, c.v))
    announce("append with no sequence numbers")
    paged = c.paged(B)
    c.check(paged, c.run(B, paged, seqs=None))


def test_many_rows_are_several_launches(B, monkeypatch):
    c = Case([150, 150], 2, 2, 32, 32, 16, 6)
    order = np.argsort(c.seqs, kind="stable")
    c.seqs, c.pos, c.q, c.k, c.v = (x[order] for x in (c.seqs, c.pos, c.q, c.k, c.v))
    monkeypatch.setenv("DS_ROWS_TEST_MAX_GROUPS", "3")
    announce("append in pieces")
    paged = c.paged(B)
    c.check(paged, c.run(B, paged, seqs=None))


def test_in_place_and_strided(B):
    import torch
    c = Case([30], 2, 6, 64, 64, 16, 7)
    qkv = dev(np.concatenate([c.q, c.k, c.v], 1), torch.bfloat16)
    q, k, v = qkv[:, :384], qkv[:, 384:512], qkv[:, 512:]
    announce("append from a fused projection, q in place")
    paged = c.paged(B)
    got = B.ds_cache_append_rows(paged.cache, k, v, dev(c.pos), seqs=dev(c.seqs), inv_freq=dev(c.inv), q=q,
                                 rms_eps=1e-6, q_weight=dev(c.qw), k_weight=dev(c.kw), q_out=q)
    torch.cuda.synchronize()
    assert got is q
    c.check(paged, q)
    assert torch.equal(bits(k.contiguous()), bits(dev(c.k, torch.bfloat16)))


def test_e4m3_rounds_to_nearest_and_saturates(B):
    """Every border between two e4m3 values goes to the even one, beyond it to
    the nearer; past the range to the largest; NaN stays NaN."""
    import torch
    vals = np.sort(D.e4m3_values()[:127])
    mids = (vals[1:] + vals[:-1]) / 2                             # exact in bf16
    xs = np.concatenate([vals, mids, -mids, [500, 464, 1e30, np.inf, -np.inf, np.nan, -1e4, 2.0 ** -20]])
    xs = np.concatenate([xs, np.zeros(-len(xs) % 64)]).astype(np.float32)
    xs = bf16_round(xs)
    rows = len(xs) // 64
    big = Paged(B, np.zeros((rows, 1, 1, 64)), np.zeros((rows, 1, 1, 64)), np.arange(rows)[None], "e4m3")
    announce("e4m3 rounding")
    x = dev(xs.reshape(rows, 64), torch.bfloat16)
    B.ds_cache_append_rows(big.cache, x, x, dev(np.arange(rows, dtype=np.int32)), seqs=dev(np.zeros(rows, np.int32)))
    torch.cuda.synchronize()
    want = torch.from_numpy(xs).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    for t in (big.k, big.v):
        assert np.array_equal(values_of(t).reshape(-1), want.astype(np.float64), equal_nan=True)


def test_offsets_past_32_bits(B):
    """Pages 1.5 GiB apart: the last lies past 4 GiB of its buffer."""
    import torch
    stride = (3 << 29) // 2                                       # elements
    buf = torch.empty(2 * (3 * stride + 4096), dtype=torch.bfloat16, device="cuda:0")
    half = 3 * stride + 4096
    view = lambda i: buf[i * half:].as_strided((4, 4, 2, 32), (stride, 64, 32, 1))  # noqa: E731
    k, v = view(0), view(1)
    k.zero_()
    v.zero_()
    cache = B.KvCache(k, v, dev(np.array([[3, 0, 2]], np.int32)))
    rng = np.random.default_rng(8)
    x = dev(bf16_round(rng.standard_normal((12, 64))), torch.bfloat16)
    announce("append past 4 GiB")
    B.ds_cache_append_rows(cache, x, -x, dev(np.arange(12, dtype=np.int32)))
    torch.cuda.synchronize()
    got = torch.cat([k[3], k[0], k[2]]).reshape(12, 64)
    assert torch.equal(got, x) and torch.equal(torch.cat([v[3], v[0], v[2]]).reshape(12, 64), -x)
    assert not k[1].any() and not v[1].any()


def test_heads_that_overflow_or_vanish(B):
    """Sums of squares past fp32's range, and heads of tiny values with eps 0."""
    c = Case([6], 2, 2, 64, 64, 16, 9)
    for x in (c.q, c.k):
        h = x.reshape(-1, 64)
        h[0] *= np.float32(2.0 ** 100)
        h[1] *= np.float32(2.0 ** -100)
        h[3] = 0
    c.q, c.k = bf16_round(c.q), bf16_round(c.k)
    announce("append heads of extreme size")
    paged = c.paged(B)
    c.check(paged, c.run(B, paged))


def test_no_rows(B):
    import torch
    c = Case([3], 2, 2, 32, 32, 4, 10)
    paged = c.paged(B)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda:0")
    i = torch.empty(0, dtype=torch.int32, device="cuda:0")
    assert B.ds_cache_append_rows(paged.cache, e, e, i, q=e).shape == (0, 64)
    assert B.ds_cache_append_rows(paged.cache, e, e, i) is None


@pytest.mark.parametrize("heads,nq,hd,kind", [(10, 70, 64, "bf16"), (70, 3, 32, "e4m3"), (5, 5, 256, "bf16")])
def test_many_rows_are_as_a_few(B, heads, nq, hd, kind):
    """More heads than a pass of one to four waves, however many rows there are."""
    import torch
    c = Case([1700, 1, 1501, 3], heads, nq, hd, hd, 16, 11, kind)
    announce("append of many rows", heads, nq, hd, kind)
    whole, parts = c.paged(B), c.paged(B)
    q = c.run(B, whole)
    b, pieces, a = torch.bfloat16, [], 0
    for n in (7, 600, 1700, len(c.pos) - 2307):            # four, two or one wave a row, by the device's size
        i, a = slice(a, a + n), a + n
        pieces.append(B.ds_cache_append_rows(
            parts.cache, dev(c.k[i], b), dev(c.v[i], b), dev(c.pos[i]), seqs=dev(c.seqs[i]), inv_freq=dev(c.inv),
            q=dev(c.q[i], b), rms_eps=1e-6, q_weight=dev(c.qw), k_weight=dev(c.kw)))
    torch.cuda.synchronize()
    assert torch.equal(bits(q), bits(torch.cat(pieces)))
    for x, y in zip(whole.bits(), parts.bits()):
        assert np.array_equal(x, y)
    want, mag = c.heads_of(c.q, c.qw)
    close(host(q), want, 52 * U * mag, "q", bf16=True)
