"""ds_embed_rows and its gradient on the GPU against the float64 oracle.

Bounds.  Forward: one fp32 product, rounded once: equal bits.  Gradient: n
fp32 additions in any order are off by at most n 2^-24 of the sum of the
terms' magnitudes, the scale's product and an addition to what was there by
2^-24 each; a bf16 gradient by half a bf16 step more.
"""
import numpy as np
import pytest

from gpu_util import announce
from oracle import token_rows as T
from token_util import U, bf16_round, bits, close, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._token_lib()
    return binding


def tokens(rng, rows, vocab, heavy=0.0, pad=0.1):
    ids = rng.integers(0, vocab, rows)
    ids[rng.random(rows) < heavy] = vocab // 2          # one token over and over
    ids[rng.random(rows) < pad] = -1
    if rows > 3:
        ids[rows // 2] = vocab                          # just past the table
    return ids


@pytest.mark.parametrize("rows,cols,vocab", [(1, 8, 1), (1, 4096, 97), (5, 520, 33), (64, 768, 500),
                                             (257, 1032, 3), (130, 2048, 50)])
@pytest.mark.parametrize("table_type,id_type", [("fp32", "int64"), ("bf16", "int32")])
def test_forward(B, rows, cols, vocab, table_type, id_type):
    import torch
    rng = np.random.default_rng(rows * 7 + cols)
    table = rng.standard_normal((vocab, cols)).astype(np.float32)
    if table_type == "bf16":
        table = bf16_round(table)
    ids = tokens(rng, rows, vocab)
    announce("embed", rows, cols, vocab, table_type, id_type)
    t = dev(table, torch.bfloat16 if table_type == "bf16" else None)
    y = B.ds_embed_rows(t, dev(ids, getattr(torch, id_type)), 27.7)
    torch.cuda.synchronize()
    want = torch.from_numpy(T.embed_rows(table, ids, 27.7)).bfloat16()
    assert torch.equal(bits(y.cpu()), bits(want))


def test_forward_of_nothing(B):
    import torch
    t = torch.zeros(0, 64, device="cuda:0")
    assert B.ds_embed_rows(t, torch.zeros(0, dtype=torch.int64, device="cuda:0")).shape == (0, 64)
    announce("embed from an empty table")
    y = B.ds_embed_rows(t, torch.zeros(3, dtype=torch.int64, device="cuda:0"))
    torch.cuda.synchronize()
    assert not y.float().any()
    y = B.ds_embed_rows(torch.ones(4, 64, device="cuda:0"), torch.tensor([4, -1, 0], device="cuda:0"), -1.0)
    torch.cuda.synchronize()
    assert not bits(y[:2]).any() and (y[2] == -1).all()         # +0 under a negative scale


def test_forward_table_past_4_gib(B):
    """Offsets that pass 32 bits: the last rows of a 4.3 GB bf16 table."""
    import torch
    vocab, cols = 131080, 16384
    announce("embed, table of", vocab * cols * 2, "bytes")
    t = torch.zeros(vocab, cols, dtype=torch.bfloat16, device="cuda:0")
    at = [0, 131071, 131072, 131079]
    for i in at:
        t[i] = i % 251
    y = B.ds_embed_rows(t, torch.tensor(at, device="cuda:0"), 1.0)
    torch.cuda.synchronize()
    assert [float(v) for v in y[:, 0]] == [float(i % 251) for i in at]
    assert (y == y[:, :1]).all()


def grad(B, dy, ids, vocab, scale, **kw):
    import torch
    d = B.ds_embed_rows_backward(dev(dy, torch.bfloat16), ids, vocab, scale, **kw)
    torch.cuda.synchronize()
    return d


@pytest.mark.parametrize("rows,cols,vocab,heavy", [
    (1, 8, 1, 0), (1, 4096, 97, 0), (33, 520, 7, 0), (64, 768, 5000, 0), (300, 1032, 3, 0),
    (700, 64, 1000, 0.5), (2500, 264, 40, 0.9), (5000, 16, 20011, 0.2), (4097, 40, 300, 0.0)])
@pytest.mark.parametrize("grad_type,id_type", [("fp32", "int64"), ("bf16", "int32")])
def test_gradient(B, rows, cols, vocab, heavy, grad_type, id_type):
    import torch
    rng = np.random.default_rng(rows * 3 + cols)
    dy = bf16_round(rng.standard_normal((rows, cols)))
    ids = tokens(rng, rows, vocab, heavy)
    want, mag, count = T.embed_rows_backward(dy, ids, vocab, 1.7)
    bound = (count[:, None] + 3) * U * mag
    dt = torch.float32 if grad_type == "fp32" else torch.bfloat16
    d_ids = dev(ids, getattr(torch, id_type))
    announce("embed gradient", rows, cols, vocab, grad_type, id_type)
    got = grad(B, dy, d_ids, vocab, 1.7, dtype=dt)
    close(host(got), want, bound, "dtable", bf16=grad_type == "bf16")
    again = grad(B, dy, d_ids, vocab, 1.7, dtype=dt)
    assert torch.equal(bits(got), bits(again))
    # added to what is there; rows of absent tokens keep their bits
    old = bf16_round(rng.standard_normal((vocab, cols)))
    acc = dev(old, dt)
    grad(B, dy, d_ids, vocab, 1.7, dtable=acc, accumulate=True)
    close(host(acc), old + want, bound + 2 * U * (np.abs(old) + mag), "accumulated",
          bf16=grad_type == "bf16")
    absent = torch.from_numpy(count == 0)
    assert torch.equal(bits(acc).cpu()[absent], bits(dev(old, dt)).cpu()[absent])


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 64, 65, 1000, 4096, 9001])
def test_gradient_of_one_token(B, rows):
    """Every row the same token, and next to it a token that never comes."""
    import torch
    rng = np.random.default_rng(rows)
    dy = bf16_round(rng.standard_normal((rows, 72)))
    announce("embed gradient, one token", rows)
    got = grad(B, dy, torch.full((rows,), 1, device="cuda:0"), 3, 1.0)
    close(host(got)[1], dy.astype(np.float64).sum(0), (rows + 3) * U * np.abs(dy).sum(0), "row 1")
    assert not host(got)[[0, 2]].any()


def test_gradient_of_whole_numbers_is_exact(B):
    """Sums of small whole numbers are exact in any order: every row counted once."""
    import torch
    rng = np.random.default_rng(8)
    rows, vocab = 20000, 3001
    dy = rng.integers(-3, 4, (rows, 16)).astype(np.float32)
    ids = (vocab ** rng.random(rows)).astype(np.int64) - 1       # few tokens very often
    announce("embed gradient, whole numbers", rows)
    got = grad(B, dy, dev(ids), vocab, 1.0)
    want = np.zeros((vocab, 16))
    np.add.at(want, ids, dy)
    assert np.array_equal(host(got), want)


@pytest.mark.parametrize("vocab", [600_007, 2_097_153])
def test_gradient_of_a_large_vocabulary(B, vocab):
    """More tokens than 256 workgroups count at once."""
    import torch
    rng = np.random.default_rng(vocab)
    rows = 5003
    dy = rng.integers(-3, 4, (rows, 8)).astype(np.float32)       # whole numbers: exact sums
    ids = rng.integers(0, vocab, rows)
    ids[::7] = vocab - 1
    ids[1::11] = 255
    announce("embed gradient, vocabulary of", vocab)
    got = host(grad(B, dy, dev(ids), vocab, 1.0))
    want = np.zeros((vocab, 8), np.float32)
    np.add.at(want, ids, dy)
    assert np.array_equal(got, want)


def test_gradient_of_no_rows_and_no_known_token(B):
    import torch
    announce("embed gradient of nothing")
    none = grad(B, np.zeros((0, 32), np.float32), torch.zeros(0, dtype=torch.int64, device="cuda:0"), 9, 1.0)
    assert none.shape == (9, 32) and not host(none).any()
    d = grad(B, np.ones((6, 32), np.float32), torch.full((6,), -1, device="cuda:0"), 9, 1.0)
    assert not host(d).any()
    kept = torch.ones(9, 32, device="cuda:0")
    grad(B, np.ones((6, 32), np.float32), torch.full((6,), 9, device="cuda:0"), 9, 1.0, dtable=kept,
         accumulate=True)
    assert (kept == 1).all()


def test_nonfinite_rows_stay_with_their_token(B):
    import torch
    dy = np.ones((40, 24), np.float32)
    dy[5, 3], dy[7, 4], dy[9, 2] = np.inf, np.nan, -np.inf
    ids = np.arange(40) % 8
    announce("embed gradient, non-finite")
    got = host(grad(B, dy, dev(ids), 8, 1.0))
    assert got[5, 3] == np.inf and np.isnan(got[7, 4]) and got[1, 2] == -np.inf
    assert np.isfinite(got).sum() == got.size - 3


def test_rows_past_the_batch_are_left_alone(B):
    """A guard behind every output keeps its value."""
    import torch
    rng = np.random.default_rng(9)
    out = torch.full((14, 520), 7.0, dtype=torch.bfloat16, device="cuda:0")
    table = dev(rng.standard_normal((11, 520)).astype(np.float32))
    announce("embed guards")
    B.ds_embed_rows(table, dev(np.arange(10)), 1.0, out=out[2:12])
    d = torch.full((15, 520), 7.0, device="cuda:0")
    B.ds_embed_rows_backward(dev(rng.standard_normal((10, 520)), torch.bfloat16), dev(np.arange(10)),
                             11, dtable=d[2:13])
    torch.cuda.synchronize()
    assert (out[:2] == 7).all() and (out[12:] == 7).all()
    assert (d[:2] == 7).all() and (d[13:] == 7).all()


def test_more_rows_than_one_launch(B, monkeypatch):
    import torch
    rng = np.random.default_rng(10)
    table, ids = dev(rng.standard_normal((50, 72)).astype(np.float32)), dev(rng.integers(0, 50, 999))
    want = B.ds_embed_rows(table, ids, 2.0)
    monkeypatch.setenv("DS_ROWS_TEST_MAX_GROUPS", "7")
    announce("embed in pieces")
    got = B.ds_embed_rows(table, ids, 2.0)
    torch.cuda.synchronize()
    assert torch.equal(bits(got), bits(want))
