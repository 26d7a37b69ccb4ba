"""ds_draft_verify_rows on the GPU against the float64 oracle.

Accepted counts and tokens must be equal: probabilities are in fp64 on both
sides, and every case's random numbers keep at least 1e-9 (relative) from the
border of each decision, which the oracle reports.  Log probabilities are
rounded to fp32 once: 2^-24 relative, with 1e-12 for the fp64 sums.
"""
import numpy as np
import pytest

from gpu_util import announce
from oracle import decode_rows as D
from token_util import U, bf16_round, close, dev, host

pytestmark = pytest.mark.gpu
MARGIN = 1e-9


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


class Case:
    def __init__(self, seqs, drafts, vocab, seed, kinds=("fp32", "fp32"), certain=False, scaled=False, inv_temp=1.0,
                 noise=0.7):
        rng = np.random.default_rng(seed)
        self.seqs, self.drafts, self.vocab, self.kinds, self.inv_temp = seqs, drafts, vocab, kinds, inv_temp
        t = rng.standard_normal((seqs, drafts + 1, vocab)).astype(np.float32) * 2
        d = t[:, :drafts] + rng.standard_normal((seqs, drafts, vocab)).astype(np.float32) * np.float32(noise)
        fit = lambda a, k: bf16_round(a) if k == "bf16" else a.astype(np.float32)  # noqa: E731
        self.target, self.draft = fit(t, kinds[0]), None if certain else fit(d, kinds[1])
        self.scale = rng.uniform(0.8, 1.25, vocab).astype(np.float32) if scaled else None
        self.draft_scale = rng.uniform(0.8, 1.25, vocab).astype(np.float32) if scaled and not certain else None
        g = -np.log(-np.log(rng.uniform(1e-30, 1, d.shape)))
        self.drafted = (d * inv_temp + (0.3 * g if certain else g)).argmax(-1).reshape(seqs, drafts).astype(np.int64)
        self.ua = rng.random((seqs, drafts)).astype(np.float32)
        self.us = rng.random(seqs).astype(np.float32)

    def args(self, ids=np.int64):
        import torch
        types = {"fp32": torch.float32, "bf16": torch.bfloat16}
        opt = lambda a: None if a is None else dev(a)  # noqa: E731
        draft = None if self.draft is None else dev(self.draft.reshape(-1, self.vocab), types[self.kinds[1]])
        return (dev(self.target.reshape(-1, self.vocab), types[self.kinds[0]]), dev(self.drafted.astype(ids)), dev(self.ua),
                dev(self.us)), dict(draft=draft, scale=opt(self.scale), inv_temp=self.inv_temp,
                                    draft_scale=opt(self.draft_scale), draft_inv_temp=self.inv_temp)

    def run(self, B, ids=np.int64):
        import torch
        a, kw = self.args(ids)
        got = B.ds_draft_verify_rows(*a, **kw)
        torch.cuda.synchronize()
        return got

    def check(self, got):
        counts = []
        acc, tok, logp = host(got.accepted), host(got.tokens), host(got.logp)
        for s in range(self.seqs):
            t = D.scaled_logits(self.target[s], self.scale, self.inv_temp)
            d = None if self.draft is None else D.scaled_logits(self.draft[s], self.draft_scale, self.inv_temp)
            want, lp, margin = D.verify_sequence(t, d, self.drafted[s], self.ua[s], self.us[s])
            assert margin > MARGIN, f"sequence {s}: too near a border to tell"
            n = len(want)
            assert acc[s] == n - 1 and tok[s].tolist() == want + [-1] * (self.drafts + 1 - n), f"sequence {s}"
            close(logp[s], lp + [0.0] * (self.drafts + 1 - n), U * np.abs(lp + [0.0] * (self.drafts + 1 - n)) + 1e-12, "logp")
            counts.append(n - 1)
        return counts


CASES = [(1, 0, 1), (5, 0, 7), (3, 1, 2), (40, 3, 50), (9, 4, 2048), (4, 2, 2049), (6, 5, 32003), (2, 32, 300),
         (3, 2, 131072), (150, 2, 33)]


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("kinds,scaled,inv_temp", [(("fp32", "fp32"), False, 1.0), (("bf16", "bf16"), True, 0.8),
                                                   (("bf16", "fp32"), False, 1.5), (("fp32", "bf16"), True, 1.0)])
@pytest.mark.parametrize("seqs,drafts,vocab", CASES)
def test_verify(B, seqs, drafts, vocab, kinds, scaled, inv_temp, certain):
    c = Case(seqs, drafts, vocab, vocab + drafts, kinds, certain, scaled, inv_temp)
    announce("verify", seqs, drafts, vocab, kinds, certain, scaled)
    c.check(c.run(B))
    c.check(c.run(B, np.int32))


def test_one_draft_logits_of_a_vocabulary_of_a_million(B):
    c = Case(2, 1, 1 << 20, 3)
    announce("verify a vocabulary of 2^20")
    c.check(c.run(B))


def test_close_drafts_are_mostly_accepted(B):
    c = Case(64, 4, 500, 4, noise=0.05)
    announce("verify close drafts")
    n = c.check(c.run(B))
    assert np.mean(n) > 3 and 4 in n
    c = Case(64, 4, 500, 5, noise=4.0)
    n = c.check(c.run(B))
    assert np.mean(n) < 1 and 0 in n


def test_drafts_that_end_and_masked_tokens(B):
    for certain in (False, True):
        c = Case(12, 3, 700, 6, certain=certain)
        c.drafted[0] = -1
        c.drafted[1, 1:] = [700, 5]
        c.drafted[2, 2] = -100
        c.drafted[3, 0] = 2 ** 31 - 1
        c.target[4:8, :, ::2] = -np.inf                           # a grammar: every other token
        c.drafted[4, 0], c.drafted[5, 0] = 2, 3                   # one it forbids, one it allows
        c.target[8, :, 1:] = -np.inf                              # all but one
        if not certain:
            c.draft[9, :, 1:] = -np.inf
        announce("verify drafts that end", certain)
        c.check(c.run(B))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_rows_that_say_nothing(B, bad):
    """A target row with a NaN or +infinity, or masked whole, gives -1; a draft
    row of that kind refuses its token and leaves the target's distribution.
    Other sequences keep their results."""
    c = Case(8, 2, 5000, 7, noise=0.05)
    was = c.run(B)
    fill = slice(None) if bad == -np.inf else slice(4321, 4322)
    c.target[1, 0, fill] = bad
    c.target[2, 1, fill] = bad
    c.target[3, 2, fill] = bad
    c.draft[4, 0, fill] = bad
    c.draft[5, 1, fill] = bad
    c.ua[1:6] = 0.01                                              # reach the second rows where the first says something
    announce("verify rows of", bad)
    got = c.run(B)
    c.check(got)
    assert host(got.tokens)[1].tolist() == [-1, -1, -1]
    for s in (0, 6, 7):
        assert np.array_equal(host(got.tokens)[s], host(was.tokens)[s])


def test_equal_rows_and_random_numbers_at_the_ends(B):
    c = Case(6, 2, 300, 8)
    c.draft[:] = c.target[:, :2]                                  # p = q: u < 1 accepts everything
    c.ua[:] = np.float32(1 - 2.0 ** -24)
    c.us[:] = [0.0, 1 - 2.0 ** -24, 0.5, -1.0, 1.5, np.nan]
    announce("verify equal rows")
    got = c.run(B)
    assert host(got.accepted).tolist() == [2] * 6
    tok = host(got.tokens)
    assert tok[0, 2] == 0 and tok[1, 2] == 299 and tok[3, 2] == 0 and tok[4, 2] == 299 and tok[5, 2] == 299
    c.ua[0, 0], c.ua[1, 1], c.ua[2, 0] = 1.0, np.nan, 2.0         # not below p / q: refused, and nothing is left over
    c.us[:] = 0.25
    got = c.run(B)
    assert host(got.accepted).tolist() == [0, 1, 0, 2, 2, 2]
    for s, i in ((0, 0), (1, 1), (2, 0)):                         # the token comes from p itself
        p, _ = D.probabilities(D.scaled_logits(c.target[s, i], None, 1.0))
        assert host(got.tokens)[s, i] == np.flatnonzero(np.cumsum(p) > 0.25)[0]


def test_far_logits_and_peaked_rows(B):
    """Rows thousands from zero, and rows whose top stands 1e4 above."""
    c = Case(10, 2, 3001, 9)
    c.target[:4] += 5000
    c.draft[:4] -= 3000
    c.target[5, :, 17] = 1e4
    c.target[6, 0, 17], c.drafted[6, 0] = 1e30, 17
    c.draft[7, 0, 9] = 1e4
    c.drafted[7, 0] = 9
    announce("verify far logits")
    c.check(c.run(B))


def test_strided_rows(B):
    import torch
    c = Case(5, 3, 1000, 10, kinds=("bf16", "bf16"))
    (t, ids, ua, us), kw = c.args()
    wide = torch.full((20, 1003), 50.0, dtype=torch.bfloat16, device="cuda:0")
    wide[:, :1000] = t
    dw = torch.full((15, 1001), 50.0, dtype=torch.bfloat16, device="cuda:0")
    dw[:, 1:] = kw["draft"]
    announce("verify strided rows")
    got = B.ds_draft_verify_rows(wide[:, :1000], ids, ua, us, **{**kw, "draft": dw[:, 1:]})
    torch.cuda.synchronize()
    c.check(got)


def test_many_samples_have_the_target_distribution(B):
    """4,096 sequences over one small vocabulary: tokens by frequency."""
    import torch
    rng = np.random.default_rng(11)
    n, vocab = 4096, 6
    zt, zd = rng.standard_normal((2, vocab)).astype(np.float32)
    p, _ = D.probabilities(zt)
    q, _ = D.probabilities(zd)
    drafted = rng.choice(vocab, (n, 1), p=q)
    t, d = dev(np.tile(zt, (2 * n, 1))), dev(np.tile(zd, (n, 1)))
    announce("verify many sequences")
    got = B.ds_draft_verify_rows(t, dev(drafted), dev(rng.random((n, 1)).astype(np.float32)),
                                 dev(rng.random(n).astype(np.float32)), draft=d)
    torch.cuda.synchronize()
    f = np.bincount(host(got.tokens)[:, 0], minlength=vocab) / n
    assert (np.abs(f - p) < 5 * np.sqrt(p * (1 - p) / n)).all()   # 5 standard deviations, from fixed numbers


def test_no_sequences(B):
    import torch
    z = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    r = B.ds_draft_verify_rows(z(0, 9), z(0, 2, dtype=torch.int64), z(0, 2), z(0))
    assert r.accepted.shape == (0,) and r.tokens.shape == (0, 3) and r.logp.shape == (0, 3)
