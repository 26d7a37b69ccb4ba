"""A decoding step of a small model with drafted tokens: embedding rows, heads
normed, rotated and appended to a paged cache, attention over it, logits, the
drafts verified and the accepted tokens fed back.  Every stage is held to the
float64 oracle on the inputs it really had; the step is then captured into
graphs that are replayed over growing sequences, run on other streams and from
threads, bit for bit.
"""
import threading

import numpy as np
import pytest

from decode_util import values_of
from gpu_util import announce
from oracle import decode_rows as D
from token_util import HALF_BF16, U, bits, close, dev, host

pytestmark = pytest.mark.gpu

SEQS, DRAFTS, VOCAB, DIM, HEADS, KV, HD, PAGE, PER_SEQ = 5, 2, 503, 256, 8, 2, 64, 16, 40
NEW = DRAFTS + 1


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


class Model:
    """One layer, its cache and the sequences' state; step() is one pass."""

    def __init__(self, B, seed, kind="bf16"):
        import torch
        g = torch.Generator(device="cuda:0").manual_seed(seed)
        self.gen = g
        n = lambda *s, sd=1.0: torch.randn(*s, device="cuda:0", generator=g) * sd  # noqa: E731
        self.table = n(VOCAB, DIM).bfloat16()
        self.proj = n(DIM, (HEADS + 2 * KV) * HD, sd=DIM ** -0.5)
        self.out = n(HEADS * HD, DIM, sd=(HEADS * HD) ** -0.5)
        self.draft_head = n(DIM, VOCAB, sd=0.1)
        self.qw, self.kw = 1 + 0.1 * n(HD), 1 + 0.1 * n(HD)
        self.inv_freq = B.ds_rope_frequencies(HD // 2, factor=4.0, original=256.0, low=1.0, high=8.0, device="cuda:0")
        dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        k, v = (torch.zeros(SEQS * PER_SEQ, KV, PAGE, HD, dtype=dtype, device="cuda:0").transpose(1, 2) for _ in "kv")
        scales = (None, None) if kind == "bf16" else (torch.full((KV,), 0.01, device="cuda:0"),) * 2
        pages = torch.randperm(SEQS * PER_SEQ, device="cuda:0", generator=g).int().reshape(SEQS, PER_SEQ)
        self.cache = B.KvCache(k, v, pages, *scales)
        # the state: the last known token and the drafts after it, of sequences of different lengths
        self.held = torch.tensor([0, 1, 200, 254, 300], dtype=torch.int32, device="cuda:0")[:SEQS].clone()
        self.ids = torch.randint(0, VOCAB, (SEQS, NEW), device="cuda:0", generator=g)
        self.ua, self.us = torch.rand(SEQS, DRAFTS, device="cuda:0", generator=g), torch.rand(SEQS, device="cuda:0", generator=g)
        for b in (k, v):                                          # what the sequences hold already
            b.copy_((n(*b.shape) / (1 if kind == "bf16" else 0.02)).clamp(-448, 448).to(dtype))

    def step(self, B, stream=None):
        import torch
        s = {}
        steps = torch.arange(NEW, dtype=torch.int32, device="cuda:0")
        s["pos"] = (self.held[:, None] + steps).flatten()
        s["lens"] = self.held + NEW
        s["x"] = B.ds_embed_rows(self.table, self.ids.flatten(), 1.0, stream=stream)
        s["qkv"] = (s["x"].float() @ self.proj).bfloat16()
        wq, wk = HEADS * HD, KV * HD
        q, k, v = s["qkv"][:, :wq], s["qkv"][:, wq:wq + wk], s["qkv"][:, wq + wk:]
        s["q"] = B.ds_cache_append_rows(self.cache, k, v, s["pos"], inv_freq=self.inv_freq, amplitude=1.1, q=q,
                                        rms_eps=1e-6, q_weight=self.qw, k_weight=self.kw, stream=stream)
        s["a"], s["lse"] = B.ds_cache_attention_rows(self.cache, s["q"], s["lens"], want_lse=True, stream=stream)
        h = B.ds_l2_rows((s["x"].float() + s["a"].float() @ self.out).bfloat16(), stream=stream)
        s["logits"] = (h.float() @ self.table.float().t().contiguous() * 2).bfloat16()
        s["draft"] = (h.float().reshape(SEQS, NEW, DIM)[:, :DRAFTS].reshape(-1, DIM) @ self.draft_head).contiguous()
        s["drafted"] = self.ids[:, 1:].contiguous()
        r = B.ds_draft_verify_rows(s["logits"], s["drafted"], self.ua, self.us, draft=s["draft"], inv_temp=0.7,
                                   stream=stream)
        s.update(accepted=r.accepted, tokens=r.tokens, logp=r.logp)
        return s

    def advance(self, s):
        """The accepted tokens are held; the next one and new drafts come after."""
        import torch
        self.held += s["accepted"] + 1
        self.ids[:, 0] = s["tokens"].gather(1, s["accepted"].long()[:, None])[:, 0].clamp(min=0)
        self.ids[:, 1:] = torch.randint(0, VOCAB, (SEQS, DRAFTS), device="cuda:0", generator=self.gen)
        self.ua.copy_(torch.rand(SEQS, DRAFTS, device="cuda:0", generator=self.gen))
        self.us.copy_(torch.rand(SEQS, device="cuda:0", generator=self.gen))


def same(a, b):
    import torch
    for name in a:
        if a[name].dtype == torch.int64:
            assert torch.equal(a[name], b[name]), name
        else:
            assert torch.equal(bits(a[name].contiguous()), bits(b[name].contiguous())), name


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_every_stage_on_its_real_inputs(B, kind):
    import torch
    m = Model(B, 1, kind)
    table = host(m.cache.page_table)
    for step in range(4):
        announce("decode chain", kind, step)
        s = m.step(B)
        torch.cuda.synchronize()
        t = {k: host(x) for k, x in s.items()}
        pos, wq, wk = t["pos"], HEADS * HD, KV * HD
        inv = host(m.inv_freq)
        y = D.normed_heads(t["qkv"][:, :wq], host(m.qw), HD, 1e-6)
        y, mag = D.rope_heads(y, pos, inv, HD, amplitude=1.1)
        close(t["q"], y, 52 * U * np.maximum(mag, np.abs(y)), "q", bf16=True)
        k, v = values_of(m.cache.k), values_of(m.cache.v)
        y = D.normed_heads(t["qkv"][:, wq:wq + wk], host(m.kw), HD, 1e-6)
        y, mag = D.rope_heads(y, pos, inv, HD, amplitude=1.1)
        scale = 1.0 if kind == "bf16" else 0.01
        half = HALF_BF16 if kind == "bf16" else 2.0 ** -4
        for row in range(SEQS * NEW):
            page, off = D.token_place(table, SEQS * PER_SEQ, PAGE, row // NEW, int(pos[row]))
            for got, want, what in ((k, y, "k"), (v, t["qkv"][:, wq + wk:], "v")):
                x = np.clip(want[row].reshape(KV, HD) / scale, -448 if scale != 1 else -np.inf, 448 if scale != 1 else np.inf)
                bound = 60 * U * np.abs(mag[row]).max() / scale + half * np.abs(x) + (2.0 ** -10 if scale != 1 else 0)
                close(got[page, off], x, bound, what)
        opt = None if kind == "bf16" else host(m.cache.k_scale)
        out, lse, mag, big, seen = D.attention(t["q"], k, v, table, t["lens"], NEW, HEADS, 0, HD ** -0.5, opt, opt)
        E = U * (2 * HD + 12) * big
        close(t["lse"], lse, E + U * (seen[:, None] + 96 + 4 * np.abs(lse)), "lse")
        close(t["a"], out, np.repeat(2 * E + 2.0 ** -16 + U * (2 * seen[:, None] + 96), HD, 1) * mag, "attention", bf16=True)
        for i in range(SEQS):
            z = D.scaled_logits(t["logits"].reshape(SEQS, NEW, VOCAB)[i], None, 0.7)
            d = D.scaled_logits(t["draft"].reshape(SEQS, DRAFTS, VOCAB)[i], None, 1.0)
            want, lp, margin = D.verify_sequence(z, d, t["drafted"][i], host(m.ua)[i], host(m.us)[i])
            if margin > 1e-9:
                assert t["tokens"][i].tolist() == want + [-1] * (NEW - len(want)) and t["accepted"][i] == len(want) - 1
                close(t["logp"][i][:len(want)], lp, U * np.abs(lp) + 1e-12, "logp")
        m.advance(s)
    assert (host(m.held) > np.array([0, 1, 200, 254, 300]) + 3).all()


def test_captured_and_replayed(B):
    """Two graphs, replayed in turn over growing sequences with eager work between."""
    import torch
    models = [Model(B, 2), Model(B, 3, "e4m3")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for m in models:
            m.step(B)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    announce("decode chain: capture")
    for m in models:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(B))
        graphs.append(g)
    for rep in range(4):
        for i in (0, 1, 0):
            announce("decode chain: replay", rep, i)
            graphs[i].replay()
            torch.cuda.synchronize()
            got = {k: x.clone() for k, x in outs[i].items()}
            cached = [bits(x.contiguous()) if x.element_size() > 1 else x.contiguous().view(torch.uint8)
                      for x in (models[i].cache.k, models[i].cache.v)]
            want = models[i].step(B)
            torch.cuda.synchronize()
            same(got, want)
            for x, y in zip((models[i].cache.k, models[i].cache.v), cached):
                assert torch.equal(bits(x.contiguous()) if x.element_size() > 1 else x.contiguous().view(torch.uint8), y)
            models[i].advance(want)


def test_two_graphs_on_two_streams(B):
    """Both replayed at once: their workspaces are their own."""
    import torch
    models = [Model(B, 4), Model(B, 5)]
    wants = [m.step(B) for m in models]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for m in models:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(B))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    announce("decode chain: two graphs at once")
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        same(got, want)


def test_on_a_stream_given_by_the_call(B):
    import torch
    m = Model(B, 6)
    want = m.step(B)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    announce("decode rows on a stream given by the call")
    wq, wk = HEADS * HD, KV * HD
    q, k, v = want["qkv"][:, :wq], want["qkv"][:, wq:wq + wk], want["qkv"][:, wq + wk:]
    rq, rk = B.ds_rope_rows(q, k, want["pos"], m.inv_freq, HD)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                                 # the current stream is busy
    for st in (side, side.cuda_stream):
        got = dict(q=B.ds_cache_append_rows(m.cache, k, v, want["pos"], inv_freq=m.inv_freq, amplitude=1.1, q=q,
                                            rms_eps=1e-6, q_weight=m.qw, k_weight=m.kw, stream=st))
        got["a"], got["lse"] = B.ds_cache_attention_rows(m.cache, want["q"], want["lens"], want_lse=True, stream=st)
        r = B.ds_draft_verify_rows(want["logits"], want["drafted"], m.ua, m.us, draft=want["draft"], inv_temp=0.7, stream=st)
        got.update(accepted=r.accepted, tokens=r.tokens, logp=r.logp)
        sq, sk = B.ds_rope_rows(q, k, want["pos"], m.inv_freq, HD, stream=st)
        side.synchronize()                                        # not the current stream
        same(got, {n: want[n] for n in got})
        same(dict(q=sq, k=sk), dict(q=rq, k=rk))


def test_threads_on_their_own_streams(B):
    import torch
    models = [Model(B, 10 + i, "bf16" if i % 2 else "e4m3") for i in range(4)]
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

    announce("decode chain from four threads")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors, errors


def test_rope_in_a_training_step(B):
    """The rotation and its gradient around autograd: the gradient of a loss of
    the rotated heads, against differences in the oracle's rotation."""
    import torch

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, pos, inv):
            ctx.save_for_backward(pos, inv)
            return B.ds_rope_rows(q, k, pos, inv, HD, interleaved=True)

        @staticmethod
        def backward(ctx, dq, dk):
            return (*B.ds_rope_rows_backward(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors, HD, interleaved=True),
                    None, None)

    g = torch.Generator(device="cuda:0").manual_seed(7)
    q, k, a, b = (torch.randn(6, 2 * HD, device="cuda:0", generator=g).bfloat16() for _ in range(4))
    q.requires_grad_(), k.requires_grad_()
    pos = torch.tensor([0, 3, 77, 1000, 50000, 7], dtype=torch.int32, device="cuda:0")
    inv = B.ds_rope_frequencies(24, device="cuda:0")
    announce("rope in a training step")
    y, z = Rope.apply(q, k, pos, inv)
    ((y.float() * a.float()).sum() + (z.float() * b.float()).sum()).backward()
    for x, w in ((q, a), (k, b)):
        f = lambda v: (D.rope_heads(v, host(pos), host(inv), HD, True)[0] * host(w)).sum()  # noqa: E731
        x0, dx = host(x).astype(np.float64), host(x.grad)
        for at in [(0, 0), (1, 5), (2, 23), (3, 24), (4, 64), (5, 127)]:
            hi, lo = x0.copy(), x0.copy()
            hi[at] += 0.5
            lo[at] -= 0.5                                         # linear: any step is exact
            want = f(hi) - f(lo)
            assert abs(dx[at] - want) <= HALF_BF16 * abs(want) + 24 * U * 8
