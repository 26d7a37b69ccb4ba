"""ds_draft_verify_rows where a launch of its own decides: batches whose last
launch has more workgroups (a sequence's parts of 4,096 tokens) than twice the
device's compute units, token by token against the float64 oracle, and bit for
bit against the same sequences a few at a time, which decide by themselves.
"""
import numpy as np
import pytest

from gpu_util import announce
from oracle import decode_rows as D
from test_gpu_draft_verify import MARGIN, Case
from token_util import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


def clear_of_borders(c):
    """The case with new random numbers for sequences that a border is too near to."""
    rng = np.random.default_rng(99)
    for s in range(c.seqs):
        for _ in range(20):
            t = D.scaled_logits(c.target[s], c.scale, c.inv_temp)
            d = None if c.draft is None else D.scaled_logits(c.draft[s], c.draft_scale, c.inv_temp)
            if D.verify_sequence(t, d, c.drafted[s], c.ua[s], c.us[s])[2] > MARGIN:
                break
            c.ua[s], c.us[s] = rng.random(c.drafts), rng.random()
    return c


def decides_apart(c):
    import torch
    return c.seqs * -(-c.vocab // 4096) > 2 * torch.cuda.get_device_properties(0).multi_processor_count


def few_at_a_time(B, c, got, step):
    """Each few sequences alone: the same bits."""
    import torch
    (t, ids, ua, us), kw = c.args()
    for a in range(0, c.seqs, step):
        b = min(c.seqs, a + step)
        few = {**kw, "draft": None if kw["draft"] is None else kw["draft"][a * c.drafts:b * c.drafts]}
        one = B.ds_draft_verify_rows(t[a * (c.drafts + 1):b * (c.drafts + 1)], ids[a:b].contiguous(), ua[a:b].contiguous(),
                                     us[a:b].contiguous(), **few)
        torch.cuda.synchronize()
        assert torch.equal(one.accepted, got.accepted[a:b]) and torch.equal(one.tokens, got.tokens[a:b])
        assert torch.equal(bits(one.logp), bits(got.logp[a:b]))


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("kinds,scaled,inv_temp", [(("fp32", "fp32"), False, 1.0), (("bf16", "bf16"), True, 0.8)])
@pytest.mark.parametrize("seqs,drafts,vocab", [(600, 2, 33), (530, 0, 4096), (300, 1, 4097), (200, 4, 10001), (40, 3, 65536)])
def test_batches(B, seqs, drafts, vocab, kinds, scaled, inv_temp, certain):
    c = clear_of_borders(Case(seqs, drafts, vocab, seqs + vocab, kinds, certain, scaled, inv_temp))
    announce("verify a batch", seqs, drafts, vocab, kinds, certain)
    assert decides_apart(c)
    got = c.run(B)
    counts = c.check(got)
    c.check(c.run(B, np.int32))
    assert drafts == 0 or certain or len(set(counts)) > 1         # (certain drafts are hardly ever accepted of 65,536)
    few_at_a_time(B, c, got, 25 if vocab < 60000 else 7)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("certain", [False, True])
def test_ended_masked_and_empty_rows_in_batches(B, certain, bad):
    """Drafts that end, grammars, rows that say nothing, of parts and slices that
    the vocabulary ends in, among hundreds of sequences."""
    c = Case(240, 3, 9001, 60, certain=certain, noise=0.3)
    fill = slice(None) if bad == -np.inf else slice(8999, 9000)
    for s in range(0, 240, 12):
        c.drafted[s] = -1
        c.drafted[s + 1, 1:] = [9001, 5]
        c.drafted[s + 2, 2] = -100
        c.drafted[s + 3, 0] = 2 ** 31 - 1
        c.target[s + 4:s + 6, :, ::2] = -np.inf
        c.drafted[s + 4, 0], c.drafted[s + 5, 0] = 2, 3
        c.target[s + 6, :, :9000] = -np.inf                       # all but the last
        c.target[s + 7, 0, fill] = bad
        c.target[s + 8, 1, fill] = bad
        c.target[s + 9, 3, fill] = bad
        if not certain:
            c.draft[s + 10, 0, fill] = bad
            c.draft[s + 11, 1, fill] = bad
        c.ua[s + 7:s + 12] = 0.01
    clear_of_borders(c)
    announce("verify a batch of ended, masked and empty rows", certain, bad)
    assert decides_apart(c)
    got = c.run(B)
    c.check(got)
    few_at_a_time(B, c, got, 12)


def test_random_numbers_at_the_ends_in_batches(B):
    import torch
    c = Case(300, 2, 9001, 61, certain=True)
    c.ua[:] = 0.0                                                 # below any probability: all accepted
    c.us[0::4], c.us[1::4], c.us[2::4], c.us[3::4] = 0.0, 1.0, np.nan, -1.0
    c.target[:, :, 4000:] -= 60
    announce("verify a batch of random numbers at the ends")
    got = c.run(B)
    tokens = got.tokens.cpu().numpy()
    assert (got.accepted == 2).all() and decides_apart(c)
    assert (tokens[0::4, 2] == 0).all() and (tokens[3::4, 2] == 0).all()
    assert (tokens[1::4, 2] == 9000).all() and (tokens[2::4, 2] == 9000).all()
    assert torch.isfinite(got.logp).all()
