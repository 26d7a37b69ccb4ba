"""ds_qk_rows_rms and its gradient on the GPU against the float64 oracle.

Bounds, in units of 2^-24 (one fp32 rounding) times the magnitude of the pair
an element turns with.  Forward: the sum of squares is 8 additions a lane and
a tree of at most 5 (half of that in 1/D), its division, 1/D (1.5), products
by 1/D and the weight, the turn's two products and sum, the angle's error (2
up to positions of 2^24, 12 at 2^31) in sine and cosine (2 ulp each): under
48.  Gradient: the turn back, the weight, u, and the mean of at most 256
products (8 a lane, a tree of 5) with its division: under 96.  A weight's
gradient adds N = rows * heads such terms: N + 64.  Outputs in bf16 add half
a bf16 step.
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


class Case:
    def __init__(self, rows, nq, nk, hd, seed, weights=True, far=True):
        rng = np.random.default_rng(seed)
        self.hd, self.nq, self.nk, self.rows = hd, nq, nk, rows
        self.q, self.dq_out = bf16_round(rng.standard_normal((2, rows, nq * hd)))
        self.k, self.dk_out = bf16_round(rng.standard_normal((2, rows, nk * hd)))
        self.pos = rng.integers(0, 1 << 20 if far else 64, rows).astype(np.int32)
        if rows > 2:
            self.pos[:3] = 0, 1, (1 << 31) - 1
        self.inv = (10000.0 ** (-np.arange(0, hd, 2) / hd)).astype(np.float32)
        self.qw, self.kw = (rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32) if weights
                            else (None, None))

    def dev(self):
        import torch
        b = torch.bfloat16
        opt = lambda w: None if w is None else dev(w)  # noqa: E731
        return (dev(self.q, b), dev(self.k, b) if self.nk else None, dev(self.pos), dev(self.inv),
                opt(self.qw), opt(self.kw))

    def grads(self):
        import torch
        return dev(self.dq_out, torch.bfloat16), dev(self.dk_out, torch.bfloat16) if self.nk else None


def check_forward(c, qo, ko, eps=1e-6):
    for x, w, got, name in ((c.q, c.qw, qo, "q"), (c.k, c.kw, ko, "k")):
        if got is None:
            continue
        want, mag = T.qk_rows_rms(x, c.pos, c.inv, w, c.hd, eps)
        close(host(got), want, 48 * U * mag, name, bf16=True)


def check_gradient(c, dq, dk, dqw, dkw, eps=1e-6):
    for x, w, dy, got, gotw, heads, name in ((c.q, c.qw, c.dq_out, dq, dqw, c.nq, "dq"),
                                             (c.k, c.kw, c.dk_out, dk, dkw, c.nk, "dk")):
        if got is None:
            continue
        dx, dw, mag, wmag = T.qk_rows_rms_backward(x, c.pos, c.inv, w, dy, c.hd, eps)
        close(host(got), dx, 96 * U * mag, name, bf16=True)
        if gotw is not None:
            close(host(gotw), dw, (c.rows * heads + 64) * U * wmag, name + "_weight")


SHAPES = [(1, 1, 0, 16), (3, 5, 2, 32), (37, 12, 12, 64), (5, 3, 1, 80), (9, 4, 4, 96), (33, 16, 4, 128),
          (2, 7, 3, 112), (6, 33, 9, 48), (17, 16, 4, 256), (4, 3, 3, 240), (700, 4, 1, 64)]


@pytest.mark.parametrize("rows,nq,nk,hd", SHAPES)
def test_forward(B, rows, nq, nk, hd):
    import torch
    c = Case(rows, nq, nk, hd, rows + hd)
    announce("qk_rms", rows, nq, nk, hd)
    qo, ko = B.ds_qk_rows_rms(*c.dev(), hd)
    torch.cuda.synchronize()
    check_forward(c, qo, ko)


@pytest.mark.parametrize("rows,nq,nk,hd", SHAPES + [(5000, 2, 1, 32)])
def test_gradient(B, rows, nq, nk, hd):
    import torch
    c = Case(rows, nq, nk, hd, rows + hd + 1)
    announce("qk_rms gradient", rows, nq, nk, hd)
    got = B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), hd)
    again = B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), hd)
    torch.cuda.synchronize()
    check_gradient(c, *got)
    for a, b in zip(got, again):
        assert a is None or torch.equal(bits(a), bits(b))


def test_without_weights(B):
    import torch
    c = Case(21, 4, 2, 64, 5, weights=False)
    announce("qk_rms without weights")
    check_forward(c, *B.ds_qk_rows_rms(*c.dev(), 64))
    check_gradient(c, *B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), 64))
    dq, dk, dqw, dkw = B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), 64, want_dweights=False)
    torch.cuda.synchronize()
    assert dqw is None and dkw is None
    check_gradient(c, dq, dk, None, None)


def test_gradient_against_differences(B):
    """A direction's derivative of the kernel's own forward pass, in whole
    steps of a size that bf16 inputs carry exactly.  The loss is a sum of N
    bf16 outputs times dy: each output is off by 2^-8 of itself (mean square
    about 1, so a standard error of 2^-9 sqrt(N) at most), seen through a step
    of 2 h, plus the third-order term of the step, h^2 times about N^(1/2)."""
    import torch
    hd, rows = 64, 64
    rng = np.random.default_rng(6)
    c = Case(rows, 2, 1, hd, 6, far=False)
    c.q = bf16_round(np.round(rng.standard_normal(c.q.shape) * 16) / 16 + 0.0)
    step = rng.integers(0, 2, c.q.shape) * 2.0 - 1.0
    h = 2.0 ** -4
    q, k, *rest = c.dev()
    g = dev(c.dq_out)
    loss = lambda v: float((B.ds_qk_rows_rms(dev(v, torch.bfloat16), k, *rest, hd)[0].double() * g).sum())  # noqa: E731
    announce("qk_rms gradient against differences")
    # multiples of 1/16 up to 8: q +- h is exact in bf16 for |q| < 8
    assert np.array_equal(bf16_round(c.q + h * step), c.q + h * step)
    assert np.array_equal(bf16_round(c.q - h * step), c.q - h * step)
    diff = (loss(c.q + h * step) - loss(c.q - h * step)) / (2 * h)
    dq = host(B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), hd)[0]).astype(np.float64)
    n = c.q.size
    tol = 6 * (2.0 ** -9 * np.sqrt(2 * n) / (2 * h) + h * h * np.sqrt(n))
    assert abs(diff - (dq * step).sum()) <= tol, (diff, (dq * step).sum(), tol)
    assert np.abs((dq * step)).sum() > 20 * tol        # the bound says something


def test_strided_slices_in_place(B):
    """q and k as slices of one projection; outputs, then gradients, in place."""
    import torch
    c = Case(50, 4, 2, 128, 7)
    wq, wk = 4 * 128, 2 * 128
    want = B.ds_qk_rows_rms(*c.dev(), 128)
    gwant = B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), 128)
    qkv = torch.full((50, wq + 2 * wk + 8), 3.0, dtype=torch.bfloat16, device="cuda:0")
    gkv = qkv.clone()
    for buf, a, b in ((qkv, c.q, c.k), (gkv, c.dq_out, c.dk_out)):
        buf[:, :wq] = dev(a, torch.bfloat16)
        buf[:, wq:wq + wk] = dev(b, torch.bfloat16)
    _, _, pos, inv, qw, kw = c.dev()
    q, k, dq, dk = (b[:, s] for b in (qkv, gkv) for s in (slice(0, wq), slice(wq, wq + wk)))
    announce("qk_rms strided, in place")
    _, _, dqw, dkw = B.ds_qk_rows_rms_backward(q, k, pos, inv, qw, kw, dq, dk, 128, dq=dq, dk=dk)
    B.ds_qk_rows_rms(q, k, pos, inv, qw, kw, 128, q_out=q, k_out=k)
    torch.cuda.synchronize()
    for got, w in ((q, want[0]), (k, want[1]), (dq, gwant[0]), (dk, gwant[1]), (dqw, gwant[2]),
                   (dkw, gwant[3])):
        assert torch.equal(bits(got.contiguous()), bits(w))
    assert (qkv[:, wq + wk:] == 3).all() and (gkv[:, wq + wk:] == 3).all()


def test_row_bits_do_not_depend_on_the_batch(B, monkeypatch):
    import torch
    c = Case(600, 3, 2, 96, 8)
    q, k, *rest = c.dev()
    pos = rest[0]
    qo, ko = B.ds_qk_rows_rms(q, k, *rest, 96)
    q1, k1 = B.ds_qk_rows_rms(q[313:314], k[313:314], pos[313:314], *rest[1:], 96)
    monkeypatch.setenv("DS_ROWS_TEST_MAX_GROUPS", "9")
    announce("qk_rms in pieces")
    q2, k2 = B.ds_qk_rows_rms(q, k, *rest, 96)
    torch.cuda.synchronize()
    assert torch.equal(bits(qo[313:314]), bits(q1)) and torch.equal(bits(ko[313:314]), bits(k1))
    assert torch.equal(bits(qo), bits(q2)) and torch.equal(bits(ko), bits(k2))


def test_extreme_heads(B):
    """Squares that overflow or underflow fp32, a zero head, negative positions."""
    import torch
    c = Case(6, 2, 1, 64, 9)
    c.q[0, :64] = 0
    c.q[1, :64] = bf16_round(c.q[1, :64] * np.float32(2.0 ** 100))
    c.q[2, 64:] = bf16_round(c.q[2, 64:] * np.float32(2.0 ** -100))
    c.k[3] = bf16_round(c.k[3] * np.float32(2.0 ** 120))
    c.pos[4:] = -1, -(1 << 31)
    for eps in (1e-6, 0.0):
        if eps == 0.0:
            c.q[0, :64] = 1                            # 0/0 without eps
        announce("qk_rms extremes", eps)
        qo, ko = B.ds_qk_rows_rms(*c.dev(), 64, eps)
        got = B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), 64, eps, want_dweights=False)
        torch.cuda.synchronize()
        check_forward(c, qo, ko, eps)
        check_gradient(c, *got, eps=eps)


def test_nonfinite_stays_in_its_head(B):
    import torch
    c = Case(4, 3, 1, 64, 10, far=False)
    c.q[0, 5], c.q[1, 64 + 3] = np.nan, np.inf
    announce("qk_rms non-finite")
    qo, ko = B.ds_qk_rows_rms(*c.dev(), 64)
    torch.cuda.synchronize()
    bad = ~np.isfinite(host(qo)).reshape(4, 3, 64)
    assert bad[0, 0].all() and bad[1, 1, [3, 35]].all()
    assert not bad[0, 1:].any() and not bad[1, [0, 2]].any() and not bad[2:].any()
    assert np.isfinite(host(ko)).all()


def test_no_rows(B):
    import torch
    c = Case(0, 2, 1, 64, 11)
    announce("qk_rms of no rows")
    qo, ko = B.ds_qk_rows_rms(*c.dev(), 64)
    dq, dk, dqw, dkw = B.ds_qk_rows_rms_backward(*c.dev(), *c.grads(), 64)
    torch.cuda.synchronize()
    assert qo.shape == (0, 128) and ko.shape == (0, 64) and dq.shape == qo.shape
    assert not dqw.any() and not dkw.any()
