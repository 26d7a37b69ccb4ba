"""The token rows together, as a model's step uses them: a unit-row embedding
made by the weight op, looked up, normalised, projected to heads, its heads
normed and rotated, logits scored, and all of it backwards to the master
weights' gradient.  Every stage is held to the float64 oracle on the inputs it
really had, with that stage's bounds; the whole step is then captured into
graphs, replayed, run on other streams and from threads, bit for bit.
"""
import threading

import numpy as np
import pytest

from gpu_util import announce
from oracle import token_rows as T
from token_util import U, bits, close, host

pytestmark = pytest.mark.gpu

ROWS, VOCAB, DIM, HEADS, KV, HD = 150, 1003, 256, 4, 2, 64


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._token_lib()
    return binding


class Model:
    """Weights and one batch; step() returns every stage's tensors by name."""

    def __init__(self, seed):
        import torch
        g = torch.Generator(device="cuda:0").manual_seed(seed)
        n = lambda *s, sd=1.0: torch.randn(*s, device="cuda:0", generator=g) * sd  # noqa: E731
        self.w = n(VOCAB, DIM, sd=0.02)
        self.gain = 1 + 0.1 * n(VOCAB)
        self.proj = n(DIM, (HEADS + 2 * KV) * HD, sd=DIM ** -0.5)
        self.qw, self.kw = 1 + 0.1 * n(HD), 1 + 0.1 * n(HD)
        self.head_scale = 1 + 0.1 * n(VOCAB)
        self.inv_freq = (10000.0 ** (-torch.arange(0, HD, 2, dtype=torch.float64) / HD)).float().to("cuda:0")
        self.ids = torch.zeros(ROWS, dtype=torch.int64, device="cuda:0")
        self.labels = torch.zeros_like(self.ids)
        self.pos = torch.arange(ROWS, dtype=torch.int32, device="cuda:0")
        self.g = torch.full((ROWS,), -1.0 / ROWS, device="cuda:0")
        self.gh = torch.full((ROWS,), 0.01 / ROWS, device="cuda:0")
        self.batch(seed)

    def batch(self, seed):
        import torch
        g = torch.Generator(device="cuda:0").manual_seed(seed)
        self.ids.copy_(torch.randint(0, VOCAB, (ROWS,), device="cuda:0", generator=g) ** 2 // VOCAB)
        self.ids[ROWS // 3:ROWS // 2] = 7                       # one token over and over
        self.ids[-5:] = -1                                      # padding
        self.labels.copy_(self.ids.roll(-1))
        self.labels[-6:] = -100

    def step(self, B, stream=None):
        """Forward and backward.  The projections between are torch products in
        fp32, and the heads' outputs go straight into the residual."""
        import torch
        s = {}
        radius = DIM ** 0.5
        _, (s["w_eff"],) = B.ds_weight_rownorm_gain([self.w], [self.gain], [radius], stream=stream)
        s["x"] = B.ds_embed_rows(s["w_eff"], self.ids, DIM ** -0.5, stream=stream)
        s["qkv"] = (s["x"].float() @ self.proj).bfloat16()
        wq, wk = HEADS * HD, KV * HD
        q, k = s["qkv"][:, :wq], s["qkv"][:, wq:wq + wk]
        s["q"], s["k"] = B.ds_qk_rows_rms(q, k, self.pos, self.inv_freq, self.qw, self.kw, HD, stream=stream)
        mixed = s["x"].float() + s["q"].float() * 0.1
        mixed[:, :wk] += s["k"].float() * 0.1
        s["h"] = B.ds_l2_rows(mixed.bfloat16(), stream=stream)
        s["logits"] = (s["h"].float() @ s["w_eff"].float().t().contiguous() * 2).bfloat16()
        r = B.ds_logprob_rows(s["logits"], self.labels, self.head_scale, 1.5, 5, stream=stream)
        s.update(logp=r.logp, entropy=r.entropy, lse=r.lse, top_ids=r.top_ids, top_logp=r.top_logp)
        s["dlogits"], s["dscale"] = B.ds_logprob_rows_backward(
            s["logits"], self.labels, r.lse, r.entropy, self.g, self.gh, self.head_scale, 1.5, stream=stream)
        s["dh"] = (s["dlogits"].float() @ s["w_eff"].float() * 2).bfloat16()
        s["dmixed"] = B.ds_l2_rows_backward(mixed.bfloat16(), None, s["dh"], stream=stream)
        s["dq"], s["dk"], s["dqw"], s["dkw"] = B.ds_qk_rows_rms_backward(
            q, k, self.pos, self.inv_freq, self.qw, self.kw, s["dmixed"], s["dmixed"][:, :wk].contiguous(),
            HD, stream=stream)
        dqkv = torch.cat([s["dq"], s["dk"]], 1).float() * 0.1
        s["dx"] = (s["dmixed"].float() + dqkv @ self.proj[:, :wq + wk].t().contiguous()).bfloat16()
        # the tied head's part of the table's gradient, then the lookup's on top
        s["head_grad"] = (s["dlogits"].float().t().contiguous() @ s["h"].float() * 2).bfloat16()
        s["dw_eff"] = B.ds_embed_rows_backward(s["dx"], self.ids, VOCAB, DIM ** -0.5,
                                               dtable=s["head_grad"].clone(), accumulate=True, stream=stream)
        (s["dw"],), (s["dgain"],) = B.ds_weight_rownorm_gain_backward(
            [self.w], [self.gain], [s["dw_eff"]], [radius], stream=stream)
        return s


def same(a, b):
    import torch
    for name in a:
        assert torch.equal(bits(a[name].contiguous()), bits(b[name].contiguous())), name


def test_every_stage_on_its_real_inputs(B):
    import torch
    m = Model(1)
    announce("token chain")
    s = m.step(B)
    torch.cuda.synchronize()
    s = {k: host(v) for k, v in s.items()}
    ids, labels, pos, inv = host(m.ids), host(m.labels), host(m.pos), host(m.inv_freq)
    want = torch.from_numpy(T.embed_rows(s["w_eff"], ids, DIM ** -0.5)).bfloat16().float().numpy()
    assert np.array_equal(s["x"], want)
    wq, wk = HEADS * HD, KV * HD
    parts = (("q", s["qkv"][:, :wq], host(m.qw), s["dmixed"], HEADS),
             ("k", s["qkv"][:, wq:wq + wk], host(m.kw), s["dmixed"][:, :wk], KV))
    for n, x, w, dy, heads in parts:
        y, mag = T.qk_rows_rms(x, pos, inv, w, HD, 1e-6)
        close(s[n], y, 48 * U * mag, n, bf16=True)
        dx, dw, mag, wmag = T.qk_rows_rms_backward(x, pos, inv, w, dy, HD, 1e-6)
        close(s["d" + n], dx, 96 * U * mag, "d" + n, bf16=True)
        close(s[f"d{n}w"], dw, (ROWS * heads + 64) * U * wmag, f"d{n}w")
    scale = host(m.head_scale)
    z = T.scaled_logits(s["logits"], scale, 1.5)
    logp, ent, lse, top_ids, top = T.logprob_rows(z, labels, 5)
    bound = (128 + 2 * np.abs(lse) + 2 * np.abs(z).max(1)) * U
    close(s["lse"], lse, bound, "lse")
    close(s["logp"], logp, bound + 2 * U * np.abs(logp), "logp")
    d = np.abs(z.max(1, keepdims=True) - z.astype(np.float64))
    p = np.exp(z - lse[:, None])
    close(s["entropy"], ent, (128 + np.abs(ent) + 70 * (p * d).sum(1) + 2 * (p * d * d).sum(1)) * U, "entropy")
    assert np.array_equal(s["top_ids"], top_ids)
    close(s["top_logp"], top, bound[:, None] + 2 * U * np.abs(top), "top_logp")
    dx, ds, unit, ds_unit, ds_mag = T.logprob_rows_backward(
        s["logits"], z, labels, s["lse"], s["entropy"], host(m.g), host(m.gh), scale, 1.5)
    close(s["dlogits"], dx, 10 * U * unit, "dlogits", bf16=True)
    close(s["dscale"], ds, 10 * U * ds_unit + (ROWS + 4) * U * ds_mag, "dscale")
    d, mag, count = T.embed_rows_backward(s["dx"], ids, VOCAB, DIM ** -0.5)
    close(s["dw_eff"], s["head_grad"] + d, (count[:, None] + 5) * U * (mag + np.abs(s["head_grad"])),
          "dw_eff", bf16=True)
    assert np.isfinite(s["dw"]).all() and np.isfinite(s["dgain"]).all()
    # tangent to the rows, by the weight op's own gradient
    w = host(m.w).astype(np.float64)
    along = np.abs((s["dw"] * w).sum(1)) / (np.linalg.norm(s["dw"], axis=1) * np.linalg.norm(w, axis=1) + 1e-30)
    assert along.max() < 1e-4


def test_captured_and_replayed(B):
    """Two graphs of the step, replayed in turn with eager work between."""
    import torch
    models = [Model(2), Model(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for m in models:
            m.step(B)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    announce("token chain: capture")
    for m in models:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(B))
        graphs.append(g)
    for rep in range(3):
        for m, i in ((models[0], 0), (models[1], 1), (models[0], 0)):
            m.batch(100 + 10 * rep + i)
            m.w.mul_(1.01)
            torch.cuda.synchronize()
            announce("token chain: replay", rep, i)
            graphs[i].replay()
            torch.cuda.synchronize()
            same(outs[i], m.step(B))


def test_on_a_stream_given_by_the_call(B):
    import torch
    m = Model(4)
    want = m.step(B)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    announce("token rows on a stream given by the call")
    wq = HEADS * HD
    torch.cuda._sleep(20_000_000)                     # the current stream is busy
    x = B.ds_embed_rows(want["w_eff"], m.ids, DIM ** -0.5, stream=side)
    q, k = B.ds_qk_rows_rms(want["qkv"][:, :wq], want["qkv"][:, wq:wq + KV * HD], m.pos, m.inv_freq, m.qw, m.kw,
                            HD, stream=side)
    dq, dk, dqw, dkw = B.ds_qk_rows_rms_backward(
        want["qkv"][:, :wq], want["qkv"][:, wq:wq + KV * HD], m.pos, m.inv_freq, m.qw, m.kw, want["dmixed"],
        want["dmixed"][:, :KV * HD].contiguous(), HD, stream=side.cuda_stream)
    r = B.ds_logprob_rows(want["logits"], m.labels, m.head_scale, 1.5, 5, stream=side)
    dl, ds = B.ds_logprob_rows_backward(want["logits"], m.labels, want["lse"], want["entropy"], m.g, m.gh,
                                        m.head_scale, 1.5, stream=side)
    dt = B.ds_embed_rows_backward(want["dx"], m.ids, VOCAB, DIM ** -0.5, stream=side)
    side.synchronize()                                # not the current stream
    got = dict(x=x, q=q, k=k, dq=dq, dk=dk, dqw=dqw, dkw=dkw, lse=r.lse, entropy=r.entropy, logp=r.logp,
               top_ids=r.top_ids, top_logp=r.top_logp, dlogits=dl, dscale=ds)
    same(got, {n: want[n] for n in got})
    again = B.ds_embed_rows_backward(want["dx"], m.ids, VOCAB, DIM ** -0.5)
    torch.cuda.synchronize()
    assert torch.equal(bits(dt), bits(again))


def test_threads_on_their_own_streams(B):
    import torch
    models = [Model(10 + i) for i in range(4)]
    wants = [m.step(B) for m in models]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(5):
                    got = models[i].step(B)
            st.synchronize()
            same(got, wants[i])
        except BaseException as e:      # noqa: BLE001 -- handed to the main thread
            errors.append((i, repr(e)))

    announce("token chain from four threads")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors, errors
