"""ds_cache_attention_rows on the GPU where its numerics have edges, against the
float64 oracle: what the weights keep, beside the cases of
test_gpu_cache_attention.py.
"""
import numpy as np
import pytest

from gpu_util import announce
from oracle import decode_rows as D
from test_gpu_cache_attention import Case
from token_util import U, bf16_round, host

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
