"""ds_rope_rows and its gradient on the GPU against the float64 oracle.

Bounds, in units of 2^-24 times the magnitude of an element's two terms: the
angle (the turn is reduced in fp64 and rounded to fp32: 2 up to positions of
2^24, 12 at 2^31), sine and cosine (2 ulp each: 4), times the amplitude (1), the
two products and their sum (3): under 24.  Outputs in bf16 add half a bf16 step.
Elements that do not turn are copies, bit for bit.
"""
import numpy as np
import pytest

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
    def __init__(self, rows, nq, nk, hd, rotary, seed, amplitude=1.0):
        rng = np.random.default_rng(seed)
        self.hd, self.amplitude = hd, amplitude
        self.q, self.k = bf16_round(rng.standard_normal((rows, nq * hd))), bf16_round(rng.standard_normal((rows, nk * hd)))
        self.pos = rng.integers(0, 1 << 20, rows).astype(np.int32)
        if rows > 3:
            self.pos[:4] = 0, 1, (1 << 31) - 1, -5
        self.inv = D.frequencies(rotary).astype(np.float32)

    def args(self):
        import torch
        return (dev(self.q, torch.bfloat16), dev(self.k, torch.bfloat16) if self.k.shape[1] else None, dev(self.pos),
                dev(self.inv), self.hd)

    def check(self, got, interleaved, back=False):
        rotary = 2 * len(self.inv)
        for x, y, name in zip((self.q, self.k), got, "qk"):
            if y is None:
                continue
            want, mag = D.rope_heads(x, self.pos, self.inv, self.hd, interleaved, self.amplitude, back)
            close(host(y), want, 24 * U * mag, name, bf16=True)
            heads = (len(x), -1, self.hd)
            assert np.array_equal(host(y).reshape(heads)[:, :, rotary:], x.reshape(heads)[:, :, rotary:]), name


# rows, q heads, k heads, head_dim, rotary: every lane count, whole, partial and odd rotary widths
SHAPES = [(1, 1, 0, 16, 16), (5, 5, 2, 32, 2), (37, 12, 12, 64, 64), (5, 3, 1, 80, 20), (9, 4, 4, 96, 24),
          (33, 16, 4, 128, 64), (4, 7, 3, 112, 112), (6, 33, 9, 48, 34), (17, 16, 4, 256, 256), (4, 3, 3, 240, 126),
          (7, 70, 1, 16, 6), (300, 4, 1, 64, 32), (5, 0, 3, 128, 128)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,nq,nk,hd,rotary", SHAPES)
def test_forward_and_gradient(B, rows, nq, nk, hd, rotary, interleaved):
    import torch
    c = Case(rows, nq, nk, hd, rotary, rows + hd, amplitude=1.0 if rows % 2 else 1.25)
    announce("rope", rows, nq, nk, hd, rotary, interleaved)
    kw = dict(interleaved=interleaved, amplitude=c.amplitude)
    got = B.ds_rope_rows(*c.args(), **kw)
    back = B.ds_rope_rows_backward(*c.args(), **kw)
    torch.cuda.synchronize()
    c.check(got, interleaved)
    c.check(back, interleaved, back=True)
    # in place, and out of a wider row into a wider row
    a = c.args()
    again = B.ds_rope_rows(*a, **kw, q_out=a[0], k_out=a[1])
    wide = torch.full((rows, (nq + 2 * nk) * hd + 8), 7.0, dtype=torch.bfloat16, device="cuda:0")
    to = wide.clone()
    wide[:, :nq * hd] = dev(c.q, torch.bfloat16)
    wide[:, nq * hd:(nq + nk) * hd] = dev(c.k, torch.bfloat16)
    cut = lambda t: (t[:, :nq * hd], t[:, nq * hd:(nq + nk) * hd] if nk else None)  # noqa: E731
    out = B.ds_rope_rows(*cut(wide), *a[2:], **kw, q_out=cut(to)[0], k_out=cut(to)[1])
    torch.cuda.synchronize()
    for x, y, z in zip(got, again, out):
        assert x is None or (torch.equal(bits(x), bits(y)) and torch.equal(bits(x), bits(z.contiguous())))
    assert bool((to[:, (nq + nk) * hd:] == 7.0).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_what_does_not_turn_is_not_touched(B, interleaved):
    """Infinities and NaN past the rotary width, and a head whose turning values
    are infinite next to one whose are not."""
    import torch
    for rotary in (16, 20):
        c = Case(8, 3, 1, 64, rotary, 1)
        q = c.q.reshape(8, 3, 64)
        q[:, :, rotary:] = np.inf
        q[1, 1, rotary + 1::2] = np.nan
        q[2, 0, :rotary] = np.inf
        announce("rope beside infinities", rotary, interleaved)
        y, _ = B.ds_rope_rows(*c.args(), interleaved=interleaved)
        torch.cuda.synchronize()
        y = host(y).reshape(8, 3, 64)
        assert np.array_equal(y[:, :, rotary:], q[:, :, rotary:], equal_nan=True)
        fine = np.ones((8, 3), bool)
        fine[2, 0] = False
        assert np.isfinite(y[:, :, :rotary][fine]).all()


def test_many_rows_are_several_launches(B, monkeypatch):
    import torch
    c = Case(523, 4, 2, 32, 20, 9)
    announce("rope in pieces")
    whole = B.ds_rope_rows(*c.args(), interleaved=True)
    monkeypatch.setenv("DS_ROWS_TEST_MAX_GROUPS", "3")
    parts = B.ds_rope_rows(*c.args(), interleaved=True)
    torch.cuda.synchronize()
    c.check(whole, True)
    for x, y in zip(whole, parts):
        assert torch.equal(bits(x), bits(y))


def test_scaled_frequencies_and_an_unaligned_table(B):
    import torch
    c = Case(40, 4, 2, 128, 128, 3, amplitude=1.2079)
    f = B.ds_rope_frequencies(128, 10000.0, 8.0, 4096.0, 1.0, 32.0)
    assert np.allclose(f.numpy(), D.frequencies(128, 10000.0, 8.0, 4096.0, 1.0, 32.0), rtol=1e-7)
    c.inv = f.numpy()
    q, k, pos, _, hd = c.args()
    buf = torch.zeros(65, device="cuda:0")
    buf[1:] = f.to("cuda:0")
    announce("rope with scaled frequencies")
    got = B.ds_rope_rows(q, k, pos, buf[1:], hd, amplitude=c.amplitude)
    torch.cuda.synchronize()
    c.check(got, False)


def test_rows_do_not_depend_on_the_batch(B):
    import torch
    c = Case(64, 12, 4, 64, 64, 4)
    q, k, pos, inv, hd = c.args()
    announce("rope row by row")
    whole = B.ds_rope_rows(q, k, pos, inv, hd)
    for i in (0, 5, 63):
        one = B.ds_rope_rows(q[i:i + 1], k[i:i + 1], pos[i:i + 1], inv, hd)
        assert torch.equal(bits(one[0]), bits(whole[0][i:i + 1])) and torch.equal(bits(one[1]), bits(whole[1][i:i + 1]))


def test_no_rows(B):
    import torch
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda:0")
    q, k = B.ds_rope_rows(e, e, torch.empty(0, dtype=torch.int32, device="cuda:0"), torch.ones(32, device="cuda:0"), 64)
    assert q.shape == (0, 128) and k.shape == (0, 128)


@pytest.mark.parametrize("nq,nk,hd", [(70, 10, 64), (3, 70, 128), (12, 12, 16), (90, 0, 32)])
def test_many_rows_are_as_a_few(B, nq, nk, hd):
    """More heads than a pass of one to four waves, however many rows there are."""
    import torch
    c = Case(5003, nq, nk, hd, hd, 8)
    q, k, pos, inv, _ = c.args()
    announce("rope of many rows", nq, nk, hd)
    whole = B.ds_rope_rows(q, k, pos, inv, hd)
    for n in (3, 1100, 3001):                              # four, two or one wave a row, by the device's size
        a = 5003 - n
        part = B.ds_rope_rows(q[a:], None if k is None else k[a:], pos[a:], inv, hd)
        torch.cuda.synchronize()
        for x, y in zip(whole, part):
            assert y is None or torch.equal(bits(x[a:].contiguous()), bits(y))
    few = Case.__new__(Case)
    few.__dict__.update(c.__dict__)
    few.q, few.k, few.pos = c.q[-37:], c.k[-37:], c.pos[-37:]
    few.check([None if y is None else y[-37:].contiguous() for y in whole], False)
