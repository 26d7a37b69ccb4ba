"""ds_draft_verify_rows on the GPU at the edges of its numerics, beside the cases
of test_gpu_draft_verify.py.
"""
import numpy as np
import pytest

from gpu_util import announce
from token_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


def near_borders(seed: int):
    """(z, u, whether u < p): fp32 differences of two logits, fp32 random numbers
    and p = e^z / (1 + e^z), 2e-15 to 2e-12 (relative) beside each other.

    2^-53 is 1.1e-16.  On the kernel's side e^z may be off by 3 of those (the
    table's entry 2, the product 1), the sum by 1, the quotient by 1, a
    reciprocal's product, the sum of two weights and u times it by 4: 9, under
    1e-15.  A polynomial off by 2e-12 puts p on the other side of some."""
    rng = np.random.default_rng(seed)
    z = -rng.uniform(0.01, 8.0, 1 << 22).astype(np.float32)
    e = np.exp(z.astype(np.longdouble))
    p = e / (1 + e)
    u = p.astype(np.float32)
    off = np.abs(u - p) / p
    at = np.flatnonzero((off > 2e-15) & (off < 2e-12))
    assert np.finfo(np.longdouble).eps < 2e-19 and len(at) > 100
    return z[at], u[at], u[at] < p[at]


@pytest.mark.parametrize("seed", [1, 2])
def test_acceptance_near_its_border(B, seed):
    import torch
    z, u, yes = near_borders(seed)
    n = len(z)
    target = np.zeros((n, 2, 2), np.float32)
    target[:, 0, 1] = z
    announce("verify near the border of acceptance", n)
    got = B.ds_draft_verify_rows(dev(target.reshape(2 * n, 2)), dev(np.ones((n, 1), np.int32)), dev(u[:, None]),
                                 dev(np.full(n, 0.25, np.float32)))
    torch.cuda.synchronize()
    assert np.array_equal(host(got.accepted) == 1, yes)
    # refused: the other token, for certain
    assert (host(got.tokens)[:, 0] == yes).all()


@pytest.mark.parametrize("seed", [3, 4])
def test_a_sample_near_its_border(B, seed):
    """Token 0 of two where its probability is above u, token 1 elsewhere."""
    import torch
    z, u, first = near_borders(seed)
    n = len(z)
    target = np.zeros((n, 2), np.float32)
    target[:, 0] = z
    announce("sample near the border of two tokens", n)
    got = B.ds_draft_verify_rows(dev(target), torch.empty(n, 0, dtype=torch.int32, device="cuda:0"),
                                 torch.empty(n, 0, device="cuda:0"), dev(u))
    torch.cuda.synchronize()
    assert np.array_equal(host(got.tokens)[:, 0] == 0, first)


@pytest.mark.parametrize("vocab", [4096, 700, 10001])
@pytest.mark.parametrize("u", [1.0, 1.5, np.inf, np.nan])
def test_random_numbers_past_the_range_give_the_last_token(B, vocab, u):
    """Rows whose upper half has weights under fp64's rounding of their total: the
    running sum is at the total long before the last token."""
    import torch
    rng = np.random.default_rng(vocab)
    z = rng.standard_normal((200, vocab)).astype(np.float32)
    z[:, vocab // 2:] -= 60
    z[100:, -5:] = -np.inf
    announce("sample past the range", vocab, u)
    got = B.ds_draft_verify_rows(dev(z), torch.empty(200, 0, dtype=torch.int32, device="cuda:0"),
                                 torch.empty(200, 0, device="cuda:0"), dev(np.full(200, u, np.float32)))
    torch.cuda.synchronize()
    want = np.where(np.arange(200) < 100, vocab - 1, vocab - 6)
    assert np.array_equal(host(got.tokens)[:, 0], want)


@pytest.mark.parametrize("certain", [False, True])
def test_target_rows_that_say_nothing_refuse_whatever_the_random_number(B, certain):
    """Below 0 it is below a probability of 0 too."""
    from test_gpu_draft_verify import Case
    c = Case(8, 2, 300, 40, certain=certain)
    c.target[0, 0] = -np.inf
    c.target[1, 0, 7] = np.nan
    c.target[2, 1] = -np.inf
    c.target[3, 1, 9] = np.inf
    c.ua[:4] = -0.5
    c.ua[4] = -1e-30
    announce("verify with random numbers below 0", certain)
    got = c.run(B)
    c.check(got)
    assert host(got.accepted)[:5].tolist() == [0, 0, 1, 1, 2]
    assert host(got.tokens)[:2, 0].tolist() == [-1, -1] and np.isfinite(host(got.logp)).all()


def test_acceptance_of_improbable_tokens_near_its_border(B):
    """Down to e^-85, where e^z may be off by 2 + 85 / 3 units of 2^-53 and what
    follows by 6: 37, under 5e-15."""
    import torch
    rng = np.random.default_rng(5)
    z = -rng.uniform(8.0, 85.0, 1 << 22).astype(np.float32)
    e = np.exp(z.astype(np.longdouble))
    p = e / (1 + e)
    u = p.astype(np.float32)
    off = np.abs(u - p) / p
    at = np.flatnonzero((off > 5e-15) & (off < 2e-12))
    z, u, yes, n = z[at], u[at], u[at] < p[at], len(at)
    assert n > 100
    target = np.zeros((n, 2, 2), np.float32)
    target[:, 0, 1] = z
    announce("verify improbable tokens near the border of acceptance", n)
    got = B.ds_draft_verify_rows(dev(target.reshape(2 * n, 2)), dev(np.ones((n, 1), np.int32)), dev(u[:, None]),
                                 dev(np.full(n, 0.25, np.float32)))
    torch.cuda.synchronize()
    assert np.array_equal(host(got.accepted) == 1, yes)
