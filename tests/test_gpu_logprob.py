"""ds_logprob_rows and its gradient on the GPU against the float64 oracle.

Bounds, with u = 2^-24.  exp(d) is off by (2 + 2 |d|) u of itself, and
sum p |d| is below 16 for any row here, so that S = sum exp(d), summed in at
most 64 steps a chunk and the joins, is off by 128 u; lse and logp add the
roundings of their own terms.  T = sum exp(d) d likewise, each term by
(70 + 2 |d|) u.  Gradient: p's exponent costs 2.5 |lp| u, its factors 10 u;
the oracle states the products these multiply.  A column sum over N rows adds
N u of its terms.  bf16 outputs add half a bf16 step.
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
    def __init__(self, rows, vocab, kind, seed, scaled=True, inv_temp=1.0, masked=0.0, sd=3.0):
        rng = np.random.default_rng(seed)
        self.rows, self.vocab, self.kind, self.inv_temp = rows, vocab, kind, inv_temp
        self.x = (rng.standard_normal((rows, vocab)) * sd).astype(np.float32)
        if kind == "bf16":
            self.x = bf16_round(self.x)
        if masked:
            self.x[rng.random((rows, vocab)) < masked] = -np.inf
        self.scale = rng.uniform(0.5, 2, vocab).astype(np.float32) if scaled else None
        self.labels = rng.integers(0, vocab, rows)
        if rows > 2:
            self.labels[1] = -100
        self.g, self.gh = rng.standard_normal((2, rows)).astype(np.float32)

    @property
    def z(self):
        return T.scaled_logits(self.x, self.scale, self.inv_temp)

    def logits(self, pad=0, before=0):
        """On the device, as a view with `pad` extra columns and `before` elements ahead."""
        import torch
        dt = torch.bfloat16 if self.kind == "bf16" else torch.float32
        ld = self.vocab + pad
        flat = torch.full((before + self.rows * ld,), float("nan"), dtype=dt, device="cuda:0")
        v = flat[before:].view(self.rows, ld)[:, :self.vocab]
        v.copy_(dev(self.x, dt))
        return v

    def forward(self, B, top_k=0, logits=None, id_type=None):
        import torch
        labels = dev(self.labels, id_type or torch.int64)
        r = B.ds_logprob_rows(self.logits() if logits is None else logits, labels,
                              None if self.scale is None else dev(self.scale), self.inv_temp, top_k)
        torch.cuda.synchronize()
        return r


def check(c, r, top_k=0):
    z = c.z
    with np.errstate(invalid="ignore"):
        logp, ent, lse, ids, top = T.logprob_rows(z, c.labels, top_k)
        m = z.max(-1, keepdims=True).astype(np.float64)
        d = np.where(z > -np.inf, z - m, 0.0)
        p = np.where(z > -np.inf, np.exp(np.where(z > -np.inf, z - lse[:, None], -1e3)), 0.0)
        a1, a2 = (p * np.abs(d)).sum(-1), (p * d * d).sum(-1)
        known = (c.labels >= 0) & (c.labels < c.vocab)
        zy = np.where(known, z[np.arange(c.rows), np.where(known, c.labels, 0)], 0.0)
    fin = lambda v: np.where(np.isfinite(v), np.abs(v), 0.0)  # noqa: E731
    base = 128 * U + 2 * U * (fin(lse) + fin(m[:, 0]))
    close(host(r.lse), lse, base, "lse")
    close(host(r.entropy), ent, 128 * U + U * (fin(ent) + 70 * fin(a1) + 2 * fin(a2)), "entropy")
    close(host(r.logp), logp, base + 2 * U * (fin(zy) + fin(logp)), "logp")
    if top_k:
        assert np.array_equal(host(r.top_ids), ids), "top ids"
        close(host(r.top_logp), top, base[:, None] + 2 * U * fin(top), "top_logp")


SIZES = [(1, 1), (3, 2), (2, 63), (5, 257), (4, 1000), (3, 8191), (3, 8192), (2, 8193), (4, 16387),
         (2, 50304), (1, 131072)]


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_forward(B, rows, vocab, kind):
    c = Case(rows, vocab, kind, rows + vocab, scaled=vocab % 2 == 0, inv_temp=1.0 if rows % 2 else 0.7)
    k = min(vocab, 7)
    announce("logprob", rows, vocab, kind)
    check(c, c.forward(B, k), k)


@pytest.mark.parametrize("rows,vocab,kind,values", [
    (1, 1 << 20, "fp32", 0), (2, 300007, "bf16", 0), (3, 262145, "fp32", 5), (257, 20001, "bf16", 0)])
def test_widest_rows(B, rows, vocab, kind, values):
    """Rows over more waves than one wave joins lists of at a time; with few
    distinct values the lists are all ties."""
    c = Case(rows, vocab, kind, vocab, scaled=rows == 2)
    if values:
        c.x = np.random.default_rng(1).integers(0, values, c.x.shape).astype(np.float32)
    announce("logprob", rows, vocab, kind)
    check(c, c.forward(B, 32), 32)


@pytest.mark.parametrize("top_k", [0, 1, 2, 5, 31, 32])
@pytest.mark.parametrize("vocab", [32, 9000, 40001])
def test_top_counts(B, top_k, vocab):
    c = Case(3, vocab, "bf16", top_k + vocab, scaled=False)
    announce("logprob top", top_k, vocab)
    check(c, c.forward(B, top_k), top_k)


@pytest.mark.parametrize("rows", [7, 300, 1500])
def test_many_rows(B, rows):
    c = Case(rows, 9001, "bf16", rows)
    announce("logprob rows", rows)
    check(c, c.forward(B, 5), 5)


@pytest.mark.parametrize("vocab", [100, 20000, 70001])
def test_ties_go_to_the_lowest_token(B, vocab):
    """Few distinct values, so that nearly all of a row ties."""
    rng = np.random.default_rng(vocab)
    c = Case(5, vocab, "fp32", vocab, scaled=False)
    c.x = rng.integers(0, 2, c.x.shape).astype(np.float32)
    c.x[1] = 0.0                                        # every token the same
    c.x[2] = np.where(rng.random(vocab) < 0.5, 0.0, -0.0)   # the zeros are equal
    c.x[3] = -np.inf
    c.x[3, -3:] = 1.0                                   # ties at the end only
    c.x[4] = np.arange(vocab)[::-1] // 7                # falling, in sevens
    announce("logprob ties", vocab)
    check(c, c.forward(B, 32), 32)


def test_rising_and_falling_rows(B):
    """Every column a new largest value, and the opposite."""
    c = Case(4, 30000, "fp32", 3, scaled=False)
    ramp = np.linspace(-20, 20, 30000).astype(np.float32)
    c.x[:] = ramp, ramp[::-1], np.roll(ramp, 15000), -np.abs(ramp)
    announce("logprob ramps")
    check(c, c.forward(B, 20), 20)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_masks(B, kind):
    """Most tokens masked, all masked, a masked label, fewer tokens than the list."""
    c = Case(6, 12345, kind, 5, masked=0.9, inv_temp=1.3)
    c.x[1] = -np.inf
    c.labels[1] = 3
    c.x[2] = -np.inf
    c.x[2, [7, 9000]] = 1.0, 2.0
    c.labels[2] = 8
    c.x[3, :8192] = -np.inf                             # a whole chunk
    c.x[4, 8192:] = -np.inf
    c.x[5] = -np.inf
    c.labels[5] = -1
    announce("logprob masks", kind)
    r = c.forward(B, 12)
    check(c, r, 12)
    assert host(r.logp)[1] == -np.inf and host(r.entropy)[1] == 0 and host(r.lse)[1] == -np.inf
    assert host(r.top_ids)[2].tolist() == [9000, 7] + [-1] * 10
    assert host(r.logp)[2] == -np.inf and host(r.logp)[5] == 0


def test_lowest_finite_masks_and_large_values(B):
    """The type's lowest value as a mask, and logits far from zero."""
    c = Case(4, 9999, "fp32", 6, scaled=False)
    low = np.finfo(np.float32).min
    c.x[0, ::2] = low
    c.x[1] = low                                        # every token at the lowest value: uniform
    c.x[2] += 30000
    c.x[3] *= 1000
    announce("logprob lowest values")
    r = c.forward(B, 4)
    check(c, r, 4)
    assert abs(host(r.entropy)[1] - np.log(9999)) < 1e-5


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [-1e9, -1e10, -1e30, -3e37, 1e8, 1e10, 1e12, 2e37, -7e14, 5e20])
def test_finite_masks_of_any_size(B, kind, value):
    """A finite mask over a whole chunk, over every token, and over all but a
    few of one row: whichever way the value's product with log2 e rounds."""
    c = Case(8, 4500, kind, 19, scaled=False)
    rnd = bf16_round if kind == "bf16" else np.float32
    c.x[0, 2048:4096] = rnd([value])[0]
    c.x[1] = rnd([value])[0]
    c.x[2, 5:] = rnd([value])[0]
    for i in range(3, 8):                               # other values, other roundings
        c.x[i] = rnd(np.array([value * (1 + 0.15 * i)], np.float32))[0]
    c.labels[:] = 2100
    announce("logprob finite masks", kind, value)
    r = c.forward(B, 4)
    check(c, r, 4)
    assert (np.abs(host(r.entropy)[[1, 3, 4, 5, 6, 7]] - np.log(4500)) < 1e-5).all()


def test_nonfinite(B):
    c = Case(5, 9000, "fp32", 7, scaled=False)
    c.x[0, 17] = np.nan
    c.x[1, 8500] = np.inf
    c.labels[0] = 4
    c.x[3] = np.nan
    announce("logprob non-finite")
    r = c.forward(B, 3)
    for got in (r.lse, r.entropy, r.logp):
        bad = ~np.isfinite(host(got))
        assert bad[[0, 3]].all() and not bad[[2, 4]].any()
    assert np.isnan(host(r.lse)[1]) and host(r.top_ids)[1][0] == 8500
    z = np.where(np.isnan(c.x), -np.inf, c.x)
    assert host(r.top_ids)[0].tolist() == np.argsort(-z[0], kind="stable")[:3].tolist()
    assert host(r.top_ids)[3].tolist() == [-1] * 3


@pytest.mark.parametrize("kind,pad,before", [("bf16", 3, 0), ("bf16", 1, 5), ("fp32", 5, 0), ("fp32", 1, 3),
                                             ("bf16", 7, 8), ("bf16", 0, 1)])
def test_any_row_alignment(B, kind, pad, before):
    """Rows at any element's address: bits as for aligned rows, NaNs beside
    the row never read into it."""
    import torch
    c = Case(9, 8200 + 5, kind, pad + before)
    c.g[:] = 1
    announce("logprob alignment", kind, pad, before)
    want, got = c.forward(B, 5), c.forward(B, 5, c.logits(pad, before))
    for a, b in zip(want, got):
        assert torch.equal(bits(a), bits(b))
    args = dev(c.labels), want.lse, want.entropy, dev(c.g), dev(c.gh), dev(c.scale)
    out = c.logits(pad, before)
    a, da = B.ds_logprob_rows_backward(c.logits(), *args)
    b, db = B.ds_logprob_rows_backward(c.logits(pad, before), *args, dlogits=out)
    torch.cuda.synchronize()
    assert torch.equal(bits(a), bits(b.contiguous())) and torch.equal(bits(da), bits(db))


def test_row_bits_do_not_depend_on_the_batch(B):
    import torch
    c = Case(700, 20011, "bf16", 9)
    x, labels, scale = c.logits(), dev(c.labels), dev(c.scale)
    announce("logprob batch invariance")
    whole = B.ds_logprob_rows(x, labels, scale, 1.0, 9)
    for rows in (1, 3, 130):
        part = B.ds_logprob_rows(x[400:400 + rows], labels[400:400 + rows], scale, 1.0, 9)
        torch.cuda.synchronize()
        for a, b in zip(whole, part):
            assert torch.equal(bits(a[400:400 + rows]), bits(b))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_thousands_of_rows(B, kind):
    """From 4,096 rows on a workgroup takes four of them: bits as for fewer."""
    import torch
    c = Case(4099, 2500, kind, 17)
    x, labels, scale = c.logits(), dev(c.labels), dev(c.scale)
    announce("logprob of 4,099 rows", kind)
    whole = B.ds_logprob_rows(x, labels, scale, 1.0, 9)
    for r0, rows in ((0, 5), (1021, 1400), (4094, 5)):
        part = B.ds_logprob_rows(x[r0:r0 + rows], labels[r0:r0 + rows], scale, 1.0, 9)
        torch.cuda.synchronize()
        for a, b in zip(whole, part):
            assert torch.equal(bits(a[r0:r0 + rows]), bits(b))
    check(c, whole, 9)


def test_outputs_one_at_a_time(B):
    import torch
    c = Case(4, 10007, "bf16", 10)
    announce("logprob without labels, int32 labels")
    want = c.forward(B, 3)
    r = B.ds_logprob_rows(c.logits(), None, dev(c.scale))
    torch.cuda.synchronize()
    assert r.logp is None and r.top_ids is None
    assert torch.equal(r.lse, want.lse) and torch.equal(r.entropy, want.entropy)
    assert torch.equal(c.forward(B, id_type=torch.int32).logp, want.logp)
    L, x, lse = B._token_lib(), c.logits(), torch.full((6,), 7.0, device="cuda:0")
    ws = torch.empty(max(16, L.ds_logprob_rows_workspace(4, 10007, 0)), dtype=torch.uint8, device="cuda:0")
    st = L.ds_logprob_rows(x.data_ptr(), B.DS_TYPE_BF16, 10007, dev(c.scale).data_ptr(), 1.0, None, 8,
                           None, None, lse.data_ptr() + 4, None, None, 0, 4, 10007, ws.data_ptr(),
                           ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == B.DS_OK and torch.equal(lse[1:5], want.lse) and lse[0] == 7 and lse[5] == 7


def backward(B, c, r, g=True, gh=True, **kw):
    import torch
    d, ds = B.ds_logprob_rows_backward(
        kw.pop("logits", None) if "logits" in kw else c.logits(), dev(c.labels), r.lse, r.entropy,
        dev(c.g) if g else None, dev(c.gh) if gh else None,
        None if c.scale is None else dev(c.scale), c.inv_temp, **kw)
    torch.cuda.synchronize()
    return d, ds


def check_backward(c, r, d, ds, g=True, gh=True):
    dx, dsc, unit, ds_unit, ds_mag = T.logprob_rows_backward(
        c.x, c.z, c.labels, host(r.lse), host(r.entropy), c.g if g else None, c.gh if gh else None,
        c.scale, c.inv_temp)
    close(host(d), dx, 10 * U * unit, "dlogits", bf16=c.kind == "bf16")
    if ds is not None:
        close(host(ds), dsc, 10 * U * ds_unit + (c.rows + 4) * U * ds_mag, "dscale")


@pytest.mark.parametrize("rows,vocab", SIZES[:-1] + [(70, 3000), (600, 515), (1030, 40)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradient(B, rows, vocab, kind):
    import torch
    c = Case(rows, vocab, kind, rows + vocab + 1, scaled=rows != 3, inv_temp=0.8 if rows % 2 else 1.0)
    announce("logprob gradient", rows, vocab, kind)
    r = c.forward(B)
    d, ds = backward(B, c, r)
    assert (ds is None) == (c.scale is None)
    check_backward(c, r, d, ds)
    d2, ds2 = backward(B, c, r)
    assert torch.equal(bits(d), bits(d2)) and (ds is None or torch.equal(bits(ds), bits(ds2)))


@pytest.mark.parametrize("g,gh", [(True, False), (False, True), (False, False)])
def test_gradient_of_one_output(B, g, gh):
    c = Case(40, 2049, "fp32", 12)
    announce("logprob gradient of", g, gh)
    r = c.forward(B)
    check_backward(c, r, *backward(B, c, r, g, gh), g, gh)


def test_gradient_in_place_and_masked(B):
    import torch
    c = Case(20, 9001, "bf16", 13, masked=0.5)
    c.x[3] = -np.inf
    announce("logprob gradient in place, masked")
    r = c.forward(B)
    want, ds = backward(B, c, r)
    check_backward(c, r, want, ds)
    dead = ~np.isfinite(c.x)
    assert not host(want)[dead].any() and not host(want)[3].any()
    x = c.logits()
    got, ds2 = backward(B, c, r, logits=x, dlogits=x)
    assert got is x and torch.equal(bits(x), bits(want)) and torch.equal(bits(ds), bits(ds2))


def test_gradient_of_tokens_masked_by_their_scale(B):
    """z is -infinity although x is not: a product past fp32's range, and
    +infinity under a negative scale.  No gradient, as a label too."""
    c = Case(12, 3001, "fp32", 20)
    c.scale[40], c.scale[2500] = -2.0, -1.5
    c.x[0, 40] = 3e38
    c.x[4, 2500] = np.inf
    c.x[5, 2500] = np.inf
    c.labels[[0, 4, 5]] = 40, 2500, 7
    announce("logprob gradient, masked by the scale")
    with np.errstate(over="ignore"):
        r = c.forward(B, 3)
        check(c, r, 3)
        d, ds = backward(B, c, r)
        c.x[[4, 5], 2500] = np.where(np.isinf(c.x[[4, 5], 2500]), np.float32(3e38), 0)   # z is the same
        check_backward(c, r, d, ds)
    assert host(d)[0, 40] == 0 and not host(d)[[4, 5], 2500].any()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [-3.3e38, -1e30, -1e9, 1e12])
def test_gradient_of_rows_masked_with_finite_values(B, kind, value):
    """Such a row gets no gradient and adds none to dscale; a finite mask over
    part of a row is like any logit."""
    c = Case(10, 2500, kind, 21, inv_temp=0.9)
    c.scale[:] = 1
    c.x[2] = value
    c.x[5, :2100] = -abs(value)
    c.labels[2], c.labels[5] = 9, 2400
    if kind == "bf16":
        c.x = bf16_round(c.x)
    announce("logprob gradient, finite masks", kind, value)
    r = c.forward(B, 3)
    check(c, r, 3)
    d, ds = backward(B, c, r)
    assert not host(d)[2].any()
    c.x[2] = -np.inf                                    # what the row counts as
    check_backward(c, r, d, ds)


def test_gradient_of_a_large_batch(B):
    """Past 256 MiB of logits in and out the loads change; the bits do not."""
    import torch
    rows, vocab = 2103, 32003
    g = torch.Generator(device="cuda:0").manual_seed(18)
    x = torch.randn(rows, vocab, device="cuda:0", generator=g).mul_(3).bfloat16()
    labels = torch.randint(0, vocab, (rows,), device="cuda:0", generator=g)
    scale = torch.rand(vocab, device="cuda:0", generator=g) + 0.5
    dl, dh = torch.randn(2, rows, device="cuda:0", generator=g)
    announce("logprob gradient, large", rows, vocab)
    r = B.ds_logprob_rows(x, labels, scale)
    whole, ds = B.ds_logprob_rows_backward(x, labels, r.lse, r.entropy, dl, dh, scale)
    total = torch.zeros(vocab, dtype=torch.float64, device="cuda:0")
    size = torch.zeros_like(total)
    for i in range(0, rows, 300):
        s = slice(i, i + 300)
        part, dsp = B.ds_logprob_rows_backward(x[s], labels[s], r.lse[s], r.entropy[s], dl[s], dh[s], scale)
        assert torch.equal(bits(whole[s]), bits(part)), i
        total += dsp.double()
        # what dscale sums, from the bf16 gradients: good enough for a magnitude
        size += (part.double() / scale * x[s].double()).abs().sum(0)
    torch.cuda.synchronize()
    # two orders of the same fp32 sums over 2,103 rows
    close(host(ds), host(total), 2 * rows * U * host(size) * 1.01, "dscale")


def test_gradient_leaves_the_padding(B):
    import torch
    c = Case(6, 1001, "fp32", 14)
    r = c.forward(B)
    buf = torch.full((8, 1010), 5.0, device="cuda:0")
    announce("logprob gradient into a view")
    backward(B, c, r, dlogits=buf[1:7, 3:1004])
    assert (buf[[0, 7]] == 5).all() and (buf[:, :3] == 5).all() and (buf[:, 1004:] == 5).all()


def test_gradient_against_differences(B):
    """Central differences of the kernel's own forward pass along a direction.
    With steps of 2^-7 the third-order term is h^2 / 6 times the third
    derivative (at most about 2 |g| + 30 |gh| a row), and the forward's error
    of some 150 u a row is seen through 2 h."""
    rng = np.random.default_rng(15)
    c = Case(30, 700, "fp32", 15, scaled=True, sd=1.0)
    step = rng.choice([-1.0, 1.0], c.x.shape).astype(np.float32)
    h = np.float32(2.0 ** -7)
    announce("logprob gradient against differences")
    r = c.forward(B)
    d, ds = backward(B, c, r)
    x0, s0 = c.x, c.scale

    def loss():
        f = c.forward(B)
        return float((host(f.logp).astype(np.float64) * c.g + host(f.entropy).astype(np.float64) * c.gh).sum())

    def along(set_to):
        set_to(h)
        hi = loss()
        set_to(-h)
        lo = loss()
        set_to(np.float32(0))
        return (hi - lo) / (2 * float(h))

    def move_x(t):
        c.x = x0 + t * step

    def move_s(t):
        c.scale = s0 + t * step[0]

    size = (np.abs(c.g) * 2 + np.abs(c.gh) * 30).sum()
    tol = size * float(h) ** 2 * 4 + 150 * U * (np.abs(c.g) + np.abs(c.gh)).sum() * 10 / (2 * float(h))
    assert abs(along(move_x) - (host(d) * step).sum()) <= tol
    assert abs(along(move_s) - (host(ds) * step[0]).sum()) <= 4 * tol     # logits of a few units


def test_offsets_past_32_bits(B):
    """Rows that start past 4 GiB: a strided view whose last rows lie there."""
    import torch
    vocab, ld, rows = 1003, 1 << 20, 2100                   # 4.4 GB of bf16 between first and last
    announce("logprob rows past 4 GiB")
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda:0")
    x = buf.view(rows, ld)[:, :vocab]
    g = torch.Generator(device="cuda:0").manual_seed(3)
    x.copy_(torch.randn(rows, vocab, device="cuda:0", generator=g))
    small = x.contiguous()
    labels = torch.randint(0, vocab, (rows,), device="cuda:0", generator=g)
    ones = torch.ones(rows, device="cuda:0")
    a, b = (B.ds_logprob_rows(t, labels, top_k=4) for t in (x, small))
    da, db = (B.ds_logprob_rows_backward(t, labels, a.lse, a.entropy, ones, ones)[0] for t in (x, small))
    torch.cuda.synchronize()
    for s, t in zip(a, b):
        assert torch.equal(bits(s), bits(t))
    assert torch.equal(bits(da), bits(db))


def test_no_rows(B):
    import torch
    c = Case(0, 100, "bf16", 16)
    announce("logprob of no rows")
    r = c.forward(B, 3)
    d, ds = backward(B, c, r)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 3) and d.shape == (0, 100)
    assert not ds.any()


@pytest.mark.parametrize("rows,vocab,kind", [(300, 2048, "fp32"), (300, 2048, "bf16"), (200, 5000, "fp32"),
                                             (200, 9000, "bf16"), (4099, 2100, "fp32"), (4098, 4096, "bf16"),
                                             (12, 131072, "fp32")])
def test_confident_rows(B, rows, vocab, kind):
    """One token 2 to 14 above all others, as in a trained model, in another
    lane than the first.

    With m = z_top and s the sum of the others' exp(z - m), S = 1 + s.  The top
    is its lane's last value of the chunk, so what rounds a sum of 1 or more is
    its own exponential (2 u), 6 sums over the lanes, the chunk's correction
    (6 u) and one addition in each of the 6 joins: 20 u, and 24 u with the
    logarithm and its subtraction.  Every other term, s in all, is off by its
    exponential's (2 + 2 |d|) u and by 70 u of sums at most."""
    rng = np.random.default_rng(rows + vocab)
    c = Case(rows, vocab, kind, vocab + 1, scaled=rows > 4000)
    c.x[:] = rng.standard_normal(c.x.shape) * 0.5 - 3
    if c.scale is not None:
        c.scale = np.exp2(rng.integers(0, 2, vocab)).astype(np.float32)
    # the last of the 32 values of lane 20, in a whole chunk
    top = (vocab // 2048 - 1) * 2048 + ((3 * 64 + 20) * 8 + 7 if kind == "bf16" else (7 * 64 + 20) * 4 + 3)
    if c.scale is not None:
        c.scale[top] = 1
    c.x[:, top] = rng.uniform(0.5, 12.5, rows)
    if kind == "bf16":
        c.x = bf16_round(c.x)
    c.labels[::2] = top
    announce("logprob confident rows", rows, vocab, kind)
    r = c.forward(B, 3)
    check(c, r, 3)
    z = c.z.astype(np.float64)
    logp, ent, lse, ids, top_lp = T.logprob_rows(c.z, c.labels, 3)
    d = z - z[:, top:top + 1]
    assert (np.delete(d, top, 1) < 0).all()
    e = np.exp(d)
    e[:, top] = 0
    s, s1, s2 = e.sum(-1), (e * -d).sum(-1), (e * d * d).sum(-1)
    off = U * (24 + 72 * s + 2 * s1)                    # of log S
    known = (c.labels >= 0) & (c.labels < vocab)
    dy = np.where(known, np.abs(d[np.arange(rows), np.where(known, c.labels, 0)]), 0)
    close(host(r.logp), logp, off + U * (dy + np.abs(logp)), "logp")
    close(host(r.lse), lse, off + U * np.abs(lse), "lse")
    close(host(r.top_logp), top_lp, off[:, None] + 2 * U * np.abs(top_lp), "top_logp")
    close(host(r.entropy), ent, off + U * (3 * ent + 74 * s1 + 2 * s2), "entropy")


@pytest.mark.parametrize("kind,scaled", [("fp32", False), ("fp32", True), ("bf16", False), ("bf16", True)])
def test_gradient_of_one_token_far_from_the_others(B, kind, scaled):
    """Past |lse| = 2^24 one token may still hold the maximum alone (a runaway
    logit, a temperature near 0): its p is 1 and the row's gradient that of any
    row, where the forward call's entropy tells so.  A maximum that tokens share
    leaves p unknown: none, and none without the entropy either."""
    import torch
    c = Case(14, 4500, kind, 23, scaled=scaled, inv_temp=0.75)
    rnd = bf16_round if kind == "bf16" else np.float32
    if scaled:
        c.scale[:] = np.exp2(np.random.default_rng(3).integers(-1, 2, 4500)).astype(np.float32)
    top, alone, shared = 3001, [0, 1, 2, 3, 4, 5, 12], [6, 7, 8, 13]
    c.x[0, top] = 4e8
    c.x[1, top] = 2e30
    c.x[2] = rnd([-3e30])[0] * (1 + np.arange(4500) % 7)    # far below, but for one
    c.x[2, top] = rnd([-2e8])[0]
    c.x[3] *= 1e9                                       # a temperature near 0
    c.x[3, top] = 2e11
    c.x[4, top] = 3e8                                   # its label the top, below a lesser one, ...
    c.x[5] = -np.inf                                    # ... the only token that is not masked
    c.x[5, top] = -4e8
    c.x[12, top] = 4e8
    c.labels[[0, 2, 3, 4, 5, 12]] = top, 17, top, top, 9, -7
    c.labels[1] = 4499
    c.x[6, [5, top]] = 1e10 / (1 if c.scale is None else c.scale[[5, top]])     # two hold the maximum
    c.x[7] = -1e30 / (1 if c.scale is None else c.scale)                        # all do
    c.x[8, :] = -np.inf
    c.x[8, :3] = -1e9 / (1 if c.scale is None else c.scale[:3])
    c.x[13, :] = 5e8 / (1 if c.scale is None else c.scale)
    c.labels[shared] = 5, 9, 2, 3
    c.x = rnd(c.x)
    announce("logprob gradient of far rows", kind, scaled)
    r = c.forward(B, 3)
    check(c, r, 3)
    lse, ent = host(r.lse), host(r.entropy)
    assert (np.abs(lse[alone + shared]) >= 2.0 ** 24).all()
    assert (np.abs(ent[alone]) < 1e-6).all() and (ent[shared] > 0.69).all()
    d, ds = backward(B, c, r)
    assert not host(d)[shared].any() and host(d)[5, 9] == 0
    for i in (1, 2):                                    # the label's gradient and the top's
        assert host(d)[i, c.labels[i]] != 0 and host(d)[i, top] != 0
    # without the entropy no far row can tell
    blind, _ = B.ds_logprob_rows_backward(c.logits(), dev(c.labels), r.lse, None, dev(c.g), None,
                                          None if c.scale is None else dev(c.scale), 0.75)
    torch.cuda.synchronize()
    assert not host(blind)[alone + shared].any()
    c.x[shared] = -np.inf                               # what they count as
    check_backward(c, r, d, ds)


def test_gradient_of_far_rows_with_a_second_token_near(B):
    """Two tokens a few steps of fp32 apart past 2^24: lse is rounded by up to
    2^-24 of itself (1.2 here), and p known to that."""
    c = Case(2, 300, "fp32", 24, scaled=False)
    c.x[:] = np.array([[2e7], [-2e7]], np.float32) - 400
    c.x[0, [7, 250]] = 2e7, 2e7 - 4
    c.x[1, [250, 7]] = -2e7, -2e7 - 6
    c.labels[:] = 7
    announce("logprob gradient of near tokens far from 0")
    r = c.forward(B)
    d, _ = backward(B, c, r, gh=False)
    z = c.x.astype(np.float64)
    p = np.exp(z - z.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    want = c.g[:, None] * ((np.arange(300) == 7) - p)
    close(host(d), want, np.abs(c.g[:, None]) * p * np.expm1(2e7 * U) + 4 * U, "dlogits")
    assert host(d)[0, 250] != 0 and host(d)[1, 7] != 0


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradient_of_tokens_masked_by_an_infinite_scale(B, kind):
    """A scale of -infinity or +infinity with logits of the other sign masks a
    column: no gradient for its logits or its scale."""
    c = Case(40, 3001, kind, 25, inv_temp=1.2)
    c.scale[[3, 1500, 3000]] = np.inf, -np.inf, np.inf
    c.x[:, [3, 3000]] = -np.abs(c.x[:, [3, 3000]]) - 0.1
    c.x[:, 1500] = np.abs(c.x[:, 1500]) + 0.1
    if kind == "bf16":
        c.x = bf16_round(c.x)
    c.labels[[4, 9]] = 3, 1500
    announce("logprob gradient, infinite scale", kind)
    r = c.forward(B, 3)
    check(c, r, 3)
    d, ds = backward(B, c, r)
    for a in (host(d)[:, [3, 1500, 3000]], host(ds)[[3, 1500, 3000]]):
        assert not a.any() and not np.isnan(a).any()
    # a masked column by another way: the rest must not tell the difference
    c.x[:, [3, 1500, 3000]], c.scale[[3, 1500, 3000]] = -np.inf, 1
    check_backward(c, r, d, ds)


@pytest.mark.parametrize("rows", [300000, 1 << 20])
def test_column_sums_of_many_tiles(B, rows):
    """One row's share of dscale is near 2^30, the others' near 1: thousands of tiles
    of at most 32 rows.  A tile's sum rounds 32 times; adding the tiles and
    rounding the total adds 2 more, however many there are."""
    import torch
    announce("logprob column sums over", rows)
    g = torch.Generator(device="cuda:0").manual_seed(26)
    x = torch.randn(rows, 6, device="cuda:0", generator=g)
    labels = torch.randint(0, 6, (rows,), device="cuda:0", generator=g)
    scale = torch.rand(6, device="cuda:0", generator=g) + 0.5
    dl = torch.rand(rows, device="cuda:0", generator=g) + 0.5
    dl[0] = 2.0 ** 31
    # labels of one half of the tokens and x < 0 in the other: one sign there
    labels %= 3
    labels[0] = 0
    x[:, 3:].abs_().neg_()
    x[0] = -1
    r = B.ds_logprob_rows(x, labels, scale)
    d, ds = B.ds_logprob_rows_backward(x, labels, r.lse, None, dl, None, scale)
    torch.cuda.synchronize()
    z = (x * scale).double()
    lp = z - r.lse.double()[:, None]
    p = torch.exp(lp)
    hot = torch.zeros_like(p).scatter_(1, labels[:, None], 1.0)
    t = dl.double()[:, None] * (hot - p) * x.double()
    unit = dl.double()[:, None] * (p * (lp.abs() + 1) + hot) * x.double().abs()
    bound = 10 * U * unit.sum(0) + 34 * U * t.abs().sum(0)
    lost = t[32:].abs().sum(0)                          # what a sum that sticks at the first would miss
    assert (lost[3:] > 2 * bound[3:]).all()
    close(host(ds), host(t.sum(0)), host(bound), "dscale")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_more_rows_than_one_launch(B, kind):
    """The forward call launches 2^20 rows at a time."""
    import torch
    rows, vocab, at = (1 << 20) + 37, 11, [0, 5, (1 << 20) - 3, 1 << 20]
    announce("logprob, two launches", kind)
    g = torch.Generator(device="cuda:0").manual_seed(27)
    x = torch.randn(rows, vocab, device="cuda:0", generator=g).mul_(2)
    x = x.bfloat16() if kind == "bf16" else x
    labels = torch.randint(-1, vocab, (rows,), device="cuda:0", generator=g)
    for ids, scale in ((labels, None), (labels.int(), torch.rand(vocab, device="cuda:0", generator=g) + 0.5)):
        whole = B.ds_logprob_rows(x, ids, scale, 0.9, 4)
        for i in at:
            n = min(40, rows - i)
            part = B.ds_logprob_rows(x[i:i + n], ids[i:i + n], scale, 0.9, 4)
            torch.cuda.synchronize()
            for a, b in zip(whole, part):
                assert torch.equal(bits(a[i:i + n]), bits(b)), i
        z = (x.float() if scale is None else x.float() * scale) * 0.9
        lse = torch.logsumexp(z.double(), -1)
        assert float((whole.lse.double() - lse).abs().max()) < 256 * U * 16


def test_gradient_of_more_tiles_than_one_launch(B):
    """The gradient launches 2^20 tiles' strips at a time: 32 rows each here."""
    import torch
    rows, vocab = (1 << 25) + 32 * 3 + 5, 3
    announce("logprob gradient, two launches")
    g = torch.Generator(device="cuda:0").manual_seed(28)
    x = torch.randn(rows, vocab, device="cuda:0", generator=g).bfloat16()
    labels = torch.randint(0, vocab, (rows,), device="cuda:0", generator=g, dtype=torch.int32)
    scale = torch.rand(vocab, device="cuda:0", generator=g) + 0.5
    dl, dh = torch.rand(2, rows, device="cuda:0", generator=g) + 0.5
    r = B.ds_logprob_rows(x, labels, scale)
    d, ds = B.ds_logprob_rows_backward(x, labels, r.lse, r.entropy, dl, dh, scale)
    total = torch.zeros(vocab, dtype=torch.float64, device="cuda:0")
    size = torch.zeros_like(total)
    for i, n in ((0, 1 << 24), (1 << 24, (1 << 24) - 7), ((1 << 25) - 7, rows - (1 << 25) + 7)):
        s = slice(i, i + n)
        part, dsp = B.ds_logprob_rows_backward(x[s], labels[s], r.lse[s], r.entropy[s], dl[s], dh[s], scale)
        torch.cuda.synchronize()
        assert torch.equal(bits(d[s]), bits(part)), i
        total += dsp.double()
        size += (part.float() / scale * x[s].float()).abs().sum(0, dtype=torch.float64)
    # two groupings of the same fp32 terms: 32 roundings a tile and 2 of the totals each
    close(host(ds), host(total), 2 * 34 * U * host(size) * 1.01, "dscale")
