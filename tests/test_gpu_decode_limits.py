"""The decoding step's calls on the GPU at the ends of their ranges: the most
sequences and rows, the widest vocabulary in a batch, strides past 32 bits."""
import numpy as np
import pytest

from gpu_util import announce
from oracle import decode_rows as D
from test_gpu_draft_verify import Case as Drafts
from test_gpu_draft_verify_batches import clear_of_borders, few_at_a_time
from token_util import U, bf16_round, bits, close, dev, host

pytestmark = pytest.mark.gpu
FAR = (1 << 31) + 64                                              # elements between two rows


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


def test_attention_of_the_most_rows_and_heads(B):
    """2^17 sequences of 64 heads: 2^23 (row, head) pairs, two chunks at most."""
    import torch
    rng = np.random.default_rng(70)
    seqs, heads, hd, page = 1 << 17, 64, 16, 128
    lens = rng.integers(0, 4, seqs).astype(np.int32)
    some = np.array([0, 1, 511, 512, 65537, seqs - 2, seqs - 1])
    lens[some] = [3, 200, 0, 256, 131, 129, 256]
    pages = torch.randn(40, page, 1, hd, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(70))
    k, v = pages.bfloat16(), (pages * 0.5).bfloat16().flip(1).contiguous()
    table = dev(rng.integers(0, 40, (seqs, 2)).astype(np.int32))
    q = torch.randn(seqs, heads * hd, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(71)).bfloat16()
    announce("attention of 2^17 sequences of 64 heads")
    out, lse = B.ds_cache_attention_rows(B.KvCache(k, v, table), q, dev(lens), want_lse=True)
    torch.cuda.synchronize()
    few = torch.cat([torch.arange(0, seqs, 997), torch.from_numpy(some)]).to("cuda:0")
    one, one_lse = B.ds_cache_attention_rows(B.KvCache(k, v, table[few].contiguous()), q[few].contiguous(),
                                             dev(lens)[few].contiguous(), want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(bits(one), bits(out[few])) and torch.equal(bits(one_lse), bits(lse[few]))
    assert bool(((lse == -np.inf).all(1) == (dev(lens) == 0)).all()) and bool(torch.isfinite(out.float()).all())
    at = few.cpu().numpy()
    want, want_lse, mag, big, seen = D.attention(host(q[few]), host(k), host(v), host(table)[at], lens[at], 1, heads, 0, hd ** -0.5)
    E, n = U * (2 * hd + 12) * big, seen[:, None]
    close(host(one_lse), want_lse, E + U * (n + 96 + 4 * np.abs(np.where(np.isfinite(want_lse), want_lse, 0))), "lse")
    close(host(one), want, np.repeat(2 * E + U * (2 * n + 96), hd, axis=1) * mag, "out", bf16=True)
    with pytest.raises(RuntimeError):                             # one sequence more
        B.ds_cache_attention_rows(B.KvCache(k, v, table.repeat(2, 1)[:seqs + 1]), torch.cat([q, q[:1]]),
                                  dev(np.append(lens, 1).astype(np.int32)))


def test_verification_of_the_most_sequences(B):
    """2^22 - 1 of them, one token of two sampled for each."""
    import torch
    n = (1 << 22) - 1
    rng = np.random.default_rng(72)
    z, u = rng.standard_normal((n, 2)).astype(np.float32), rng.random(n).astype(np.float32)
    e = np.exp(z.astype(np.float64) - z.max(1, keepdims=True))
    p = e[:, 0] / e.sum(1)
    clear = np.abs(p - u) > 1e-12 * p                             # (both sides are in fp64)
    none = torch.empty(n, 0, dtype=torch.int32, device="cuda:0")
    announce("sample for 2^22 - 1 sequences")
    got = B.ds_draft_verify_rows(dev(z), none, none.float(), dev(u))
    torch.cuda.synchronize()
    assert not host(got.accepted).any()
    token = host(got.tokens)[:, 0]
    assert np.array_equal(token[clear], np.where(p > u, 0, 1)[clear])
    logp = np.log(np.take_along_axis(e, token[:, None].astype(np.int64), 1)[:, 0] / e.sum(1))
    close(host(got.logp)[:, 0], logp, U * np.abs(logp) + 1e-12, "logp")
    more = torch.zeros(n + 1, 2, device="cuda:0")
    with pytest.raises(RuntimeError):
        B.ds_draft_verify_rows(more, torch.empty(n + 1, 0, dtype=torch.int32, device="cuda:0"),
                               torch.empty(n + 1, 0, device="cuda:0"), more[:, 0].contiguous())


@pytest.mark.parametrize("vocab,certain", [(1 << 20, False), ((1 << 20) - 1, True)])
def test_the_widest_vocabulary_in_a_batch(B, vocab, certain):
    c = clear_of_borders(Drafts(3, 1, vocab, 73, certain=certain))
    announce("verify a batch of the widest vocabulary", vocab, certain)
    got = c.run(B)
    c.check(got)
    few_at_a_time(B, c, got, 1)


def far_rows(values):
    """The rows [2, width] of a bf16 array, FAR elements apart."""
    import torch
    buf = torch.empty(FAR + 4096, dtype=torch.bfloat16, device="cuda:0")
    t = buf.as_strided((2, values.shape[1]), (FAR, 1))
    t.copy_(dev(values, torch.bfloat16))
    return t


def test_rows_of_logits_past_32_bits(B):
    import torch
    c = Drafts(1, 1, 3000, 74, kinds=("bf16", "bf16"))
    (t, ids, ua, us), kw = c.args()
    announce("verify rows 4 GiB apart")
    got = B.ds_draft_verify_rows(far_rows(host(t)), ids, ua, us, **kw)
    torch.cuda.synchronize()
    c.check(got)


def test_rows_of_heads_past_32_bits(B):
    import torch
    rng = np.random.default_rng(75)
    x = bf16_round(rng.standard_normal((2, 4 * 64)))
    pos, inv = np.array([5, 77], np.int32), D.frequencies(64).astype(np.float32)
    near, far = dev(x, torch.bfloat16), far_rows(x)
    announce("rope, append and attention of rows 4 GiB apart")
    want, _ = B.ds_rope_rows(near, None, dev(pos), dev(inv), 64)
    got, _ = B.ds_rope_rows(far, None, dev(pos), dev(inv), 64)
    B.ds_rope_rows(far, None, dev(pos), dev(inv), 64, q_out=far)
    torch.cuda.synchronize()
    assert torch.equal(bits(got), bits(want)) and torch.equal(bits(far.contiguous()), bits(want))
    outs = []
    for t in (near, far_rows(x)):
        zero = lambda: torch.zeros(6, 16, 4, 64, dtype=torch.bfloat16, device="cuda:0")  # noqa: E731
        cache = B.KvCache(zero(), zero(), dev(np.arange(6, dtype=np.int32).reshape(1, 6)))
        q = B.ds_cache_append_rows(cache, t, t, dev(pos), inv_freq=dev(inv), q=t)
        out = B.ds_cache_attention_rows(cache, t, dev(np.array([78], np.int32)))
        into = far_rows(np.zeros_like(x))
        B.ds_cache_attention_rows(cache, t, dev(np.array([78], np.int32)), out=into)
        torch.cuda.synchronize()
        assert torch.equal(bits(into.contiguous()), bits(out))
        outs.append([bits(y).clone() for y in (q, cache.k, cache.v, out)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_millions_of_rows(B):
    """Rotated, and put into a cache of one sequence of 2^20 tokens a page at a time."""
    import torch
    n = (1 << 20) + 3
    g = torch.Generator("cuda:0").manual_seed(76)
    x = torch.randn(n, 32, device="cuda:0", generator=g).bfloat16()
    pos, inv = torch.arange(n, dtype=torch.int32, device="cuda:0"), dev(D.frequencies(16).astype(np.float32))
    announce("rope and append of 2^20 + 3 rows")
    y, _ = B.ds_rope_rows(x, None, pos, inv, 16)
    pages = -(-n // 16)
    k, v = (torch.zeros(pages, 16, 2, 16, dtype=torch.bfloat16, device="cuda:0") for _ in "kv")
    table = torch.randperm(pages, device="cuda:0", generator=g).to(torch.int32)[None]
    B.ds_cache_append_rows(B.KvCache(k, v, table), x, x, pos, inv_freq=inv)
    torch.cuda.synchronize()
    stored = lambda t: t[table[0].long()].reshape(-1, 32)[:n]  # noqa: E731
    assert torch.equal(bits(stored(k)), bits(y)) and torch.equal(bits(stored(v)), bits(x))
    at = np.array([0, 65535, 65536, 65537, n - 1])
    want, mag = D.rope_heads(host(x[at]), at, host(inv), 16)
    close(host(y[at]), want, 24 * U * mag, "q", bf16=True)
