"""ds_decode_rows.h without a GPU: symbols, workspace sizes, argument checks,
the frequency table (a host call).

Every refused call returns before its first HIP call (fake pointer values are
never dereferenced).  Calls with valid arguments are made only where no HIP
device exists, where they must stop at DS_ERR_DEVICE.
"""
import ctypes
import os

import numpy as np
import pytest

from oracle import decode_rows as D
from scale_invariant_row_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH),
                                reason="library not built (python -m scale_invariant_row_amd.build)")

P = [0x10000000 * (i + 1) for i in range(24)]       # fake, aligned, far apart
BIG = 1 << 26
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return B._decode_lib()


def test_exports_every_declared_function(L):
    names = B.header_functions(B.DECODE_HEADER)
    assert set(names) == {
        "ds_rope_rows", "ds_rope_rows_backward", "ds_rope_frequencies", "ds_cache_append_rows",
        "ds_cache_attention_rows", "ds_cache_attention_rows_workspace", "ds_draft_verify_rows",
        "ds_draft_verify_rows_workspace"}
    for n in names:
        assert hasattr(L, n), n


def test_the_cache_struct_is_the_headers():
    assert ctypes.sizeof(B.KvCacheDesc) == 5 * 8 + 4 * 8 + 7 * 4 + 4
    text = open(B.DECODE_HEADER).read()
    body = text[text.index("typedef struct ds_kv_cache {"):text.index("} ds_kv_cache;")]
    names = [n.strip(" *") for line in body.splitlines()[1:] for n in line.strip().rstrip(";").split(" ", 2 if
             line.strip().startswith("const") else 1)[-1].split(",") if n.strip()]
    assert names == [f for f, _ in B.KvCacheDesc._fields_]


# 7 pages of 16 tokens, 2 heads of 64; 3 sequences of up to 4 pages
CACHE = dict(k=P[20], v=P[21], k_scale=None, v_scale=None, page_table=P[22], page_stride=2048, token_stride=128,
             head_stride=64, ld_table=4, type=B.DS_TYPE_BF16, n_pages=7, page_size=16, n_heads=2, head_dim=64,
             n_seqs=3, pages_per_seq=4)


class Call:
    """Keyword arguments over a valid call; those of the cache go into its struct."""

    def __init__(self, name, **base):
        self.name, self.base = name, base

    def __call__(self, L, **over):
        assert set(over) <= set(self.base) | (set(CACHE) if "cache" in self.base else set()), over
        args = {**self.base, **{n: v for n, v in over.items() if n in self.base}}
        if args.get("cache") == "cache":
            cache = B.KvCacheDesc(**{**CACHE, **{n: v for n, v in over.items() if n in CACHE and n not in self.base}})
            args["cache"] = ctypes.addressof(cache)
        return getattr(L, self.name)(*args.values())


rope = Call("ds_rope_rows", q=P[0], ldq=256, k=P[1], ldk=128, pos=P[2], inv=P[3], rotary=64, pairs=0, amp=1.0,
            qo=P[6], ldqo=256, ko=P[7], ldko=128, rows=10, nq=4, nk=2, hd=64, stream=None)
rope_bwd = Call("ds_rope_rows_backward", **rope.base)
append = Call("ds_cache_append_rows", cache="cache", q=P[0], ldq=256, kk=P[1], ldk=128, vv=P[2], ldv=128, pos=P[3],
              seqs=P[4], inv=P[5], rotary=64, pairs=0, amp=1.0, rms=1, qw=P[6], kw=P[7], eps=1e-6, qo=P[8],
              ldqo=256, rows=10, nq=4, stream=None)
attend = Call("ds_cache_attention_rows", cache="cache", q=P[0], ldq=256, nq=4, lens=P[1], new=2, window=0,
              scale=0.125, out=P[2], ldo=256, lse=P[3], ws=P[4], nws=BIG, stream=None)
verify = Call("ds_draft_verify_rows", t=P[0], tt=B.DS_TYPE_BF16, ldt=1000, scale=P[1], tau=1.0, d=P[2],
              dt=B.DS_TYPE_F32, ldd=1000, dscale=P[3], dtau=1.0, ids=P[4], id_bytes=8, ua=P[5], us=P[6], acc=P[7],
              tok=P[8], logp=P[9], seqs=5, drafts=3, vocab=1000, ws=P[10], nws=BIG, stream=None)
EVERY = [rope, rope_bwd, append, attend, verify]


def no_device():
    import torch
    return torch.cuda.device_count() == 0


@pytest.mark.skipif("not no_device()")
@pytest.mark.parametrize("call", EVERY, ids=lambda c: c.name)
def test_valid_arguments_reach_the_device(L, call):
    assert call(L) == B.DS_ERR_DEVICE


N, S, A, G, W = B.DS_ERR_NULL, B.DS_ERR_SHAPE, B.DS_ERR_ALIGN, B.DS_ERR_ARG, B.DS_ERR_WORKSPACE
BAD_CACHE = [
    (dict(type=B.DS_TYPE_F32), G), (dict(type=3), G), (dict(n_heads=0), S), (dict(n_heads=-1), S),
    (dict(head_dim=24), S), (dict(head_dim=272), S), (dict(head_dim=0), S), (dict(n_pages=-1), S),
    (dict(page_size=0), S), (dict(page_size=24), S), (dict(page_size=8192), S), (dict(page_size=-16), S),
    (dict(pages_per_seq=-1), S), (dict(n_seqs=-1), S), (dict(pages_per_seq=1 << 27, ld_table=1 << 27), S),
    (dict(ld_table=3), S), (dict(page_stride=2044), S), (dict(page_stride=-2048), S),
    (dict(token_stride=1 << 61), S), (dict(k=None), N), (dict(v=None), N), (dict(page_table=None), N),
    (dict(k=P[20] + 8), A), (dict(v=P[21] + 2), A), (dict(page_table=P[22] + 2), A),
    (dict(k_scale=P[23] + 1), A), (dict(v_scale=P[23] + 2), A), (dict(head_stride=56), G),
    (dict(token_stride=64), G), (dict(page_stride=1024), G), (dict(v=P[20]), G), (dict(v=P[20] + 1024), G),
    (dict(type=B.DS_TYPE_E4M3, page_stride=2056), S),
]


@pytest.mark.parametrize("call,over,code", [
    *[(c, o, e) for c in (append, attend) for o, e in BAD_CACHE],
    *[(c, o, e) for c in (rope, rope_bwd) for o, e in [
        (dict(q=None), N), (dict(ko=None), N), (dict(pos=None), N), (dict(inv=None), N), (dict(rotary=0), S),
        (dict(rotary=63), S), (dict(rotary=66), S), (dict(rotary=-2), S), (dict(hd=24), S), (dict(hd=272), S),
        (dict(nq=-1), S), (dict(rows=-1), S), (dict(ldq=248), S), (dict(ldko=132), S), (dict(rows=1 << 61), S),
        (dict(pairs=2), G), (dict(amp=NAN), G), (dict(amp=INF), G), (dict(q=P[0] + 2), A), (dict(pos=P[2] + 1), A),
        (dict(inv=P[3] + 2), A), (dict(qo=P[0] + 16), G), (dict(qo=P[1]), G), (dict(qo=P[2]), G),
        (dict(ko=P[3]), G), (dict(qo=P[0], ldqo=264), G), (dict(ko=P[6] + 128), G)]],
    (append, dict(cache=None), N), (append, dict(q=None), N), (append, dict(kk=None), N), (append, dict(vv=None), N),
    (append, dict(pos=None), N), (append, dict(inv=None), N), (append, dict(qo=None), N), (append, dict(rotary=65), S),
    (append, dict(rotary=128), S), (append, dict(rows=-1), S), (append, dict(seqs=None), S), (append, dict(nq=-1), S),
    (append, dict(ldv=120), S), (append, dict(ldk=132), S), (append, dict(pairs=-1), G), (append, dict(rms=2), G),
    (append, dict(rms=0), G), (append, dict(eps=-1.0), G), (append, dict(eps=NAN), G), (append, dict(amp=INF), G),
    (append, dict(kk=P[1] + 8), A), (append, dict(qw=P[6] + 4), A), (append, dict(seqs=P[4] + 2), A),
    (append, dict(qo=P[1]), G), (append, dict(qo=P[20] + 16), G), (append, dict(vv=P[21]), G), (append, dict(kk=P[20]), G),
    (append, dict(pos=P[20] + 64), G), (append, dict(inv=P[21] + 64), G), (append, dict(kw=P[21] + 64), G),
    (append, dict(page_table=P[20] + 4), G), (append, dict(k_scale=P[21] + 4), G), (append, dict(qo=P[22]), G),
    (append, dict(qo=P[0], ldqo=264), G), (append, dict(q=P[20]), G),
    (attend, dict(cache=None), N), (attend, dict(q=None), N), (attend, dict(out=None), N), (attend, dict(lens=None), N),
    (attend, dict(ws=None, n_pages=300, pages_per_seq=100, ld_table=100), N), (attend, dict(nq=3), S),
    (attend, dict(nq=0), S), (attend, dict(nq=-2), S), (attend, dict(new=0), S), (attend, dict(new=17), S),
    (attend, dict(window=-1), G), (attend, dict(scale=NAN), G), (attend, dict(scale=-INF), G),
    (attend, dict(n_seqs=1 << 22), S), (attend, dict(ldq=248), S), (attend, dict(ldo=260), S),
    (attend, dict(nws=16, pages_per_seq=100, ld_table=100), W),
    (attend, dict(ws=P[4] + 4, pages_per_seq=100, ld_table=100), A), (attend, dict(lens=P[1] + 1), A),
    (attend, dict(lse=P[3] + 2), A), (attend, dict(out=P[0]), G), (attend, dict(out=P[20]), G),
    (attend, dict(out=P[1]), G), (attend, dict(lse=P[0] + 4), G), (attend, dict(lse=P[2]), G),
    (attend, dict(lse=P[21]), G), (attend, dict(out=P[22]), G),
    (attend, dict(ws=P[0], pages_per_seq=100, ld_table=100), G),
    (attend, dict(ws=P[20], pages_per_seq=100, ld_table=100), G),
    (verify, dict(t=None), N), (verify, dict(ids=None), N), (verify, dict(ua=None), N), (verify, dict(us=None), N),
    (verify, dict(acc=None), N), (verify, dict(tok=None), N), (verify, dict(logp=None), N), (verify, dict(ws=None), N),
    (verify, dict(nws=64), W), (verify, dict(ldt=999), S), (verify, dict(ldd=999), S), (verify, dict(drafts=33), S),
    (verify, dict(drafts=-1), S), (verify, dict(vocab=0), S), (verify, dict(seqs=-1), S), (verify, dict(seqs=1 << 24), S),
    (verify, dict(vocab=1 << 21, ldt=1 << 21, ldd=1 << 21), S), (verify, dict(ldt=1 << 60), S),
    (verify, dict(tt=2), G), (verify, dict(dt=3), G), (verify, dict(id_bytes=2), G), (verify, dict(tau=0.0), G),
    (verify, dict(tau=NAN), G), (verify, dict(dtau=-1.0), G), (verify, dict(dtau=INF), G), (verify, dict(t=P[0] + 1), A),
    (verify, dict(d=P[2] + 2), A), (verify, dict(ids=P[4] + 4), A), (verify, dict(ua=P[5] + 1), A),
    (verify, dict(tok=P[8] + 2), A), (verify, dict(ws=P[10] + 8), A), (verify, dict(tok=P[0]), G),
    (verify, dict(acc=P[9] + 4), G), (verify, dict(logp=P[2] + 64), G), (verify, dict(ws=P[0]), G),
    (verify, dict(ws=P[4]), G), (verify, dict(acc=P[6]), G), (verify, dict(tok=P[5]), G),
], ids=lambda v: getattr(v, "name", None) or (str(v) if isinstance(v, dict) else None))
def test_refused(L, call, over, code):
    assert call(L, **over) == code


@pytest.mark.parametrize("call", EVERY, ids=lambda c: c.name)
def test_no_rows_is_a_noop(L, call):
    """Nothing to write: pointers are not looked at, no device is needed."""
    none = {k: None for k, v in call.base.items() if isinstance(v, int) and v in P}
    over = dict(none, nws=0) if "nws" in call.base else none
    over.update(rms=1) if call is append else None
    if call is attend:
        over.update(n_seqs=0, page_table=None)
    else:
        over["seqs" if call is verify else "rows"] = 0
    assert call(L, **over) == B.DS_OK


@pytest.mark.skipif("not no_device()")
def test_what_is_allowed(L):
    dev = B.DS_ERR_DEVICE
    assert rope(L, qo=P[0], ko=P[1]) == dev                                     # in place
    assert rope(L, q=P[0], ldq=512, k=P[0] + 512, ldk=512, qo=P[0], ldqo=512, ko=P[0] + 512, ldko=512) == dev
    assert rope(L, k=None, ko=None, nk=0) == dev and rope(L, rotary=2, inv=P[3] + 4) == dev
    assert append(L, q=None, qo=None, nq=0) == dev and append(L, qo=P[0]) == dev
    assert append(L, inv=None, rotary=0) == dev and append(L, rms=0, qw=None, kw=None) == dev
    assert append(L, seqs=None, rows=12) == dev                                 # four of each sequence
    assert append(L, n_pages=0, k=None, v=None) == dev                          # nothing to store into
    assert append(L, pages_per_seq=0, page_table=None) == dev
    # head-major pages; k and v in turn in one buffer; a lone head, page and token of any stride
    assert append(L, token_stride=64, head_stride=1024) == dev
    assert append(L, page_stride=4096, v=P[20] + 4096) == dev
    assert append(L, token_stride=256, page_stride=4096, v=P[20] + 256) == dev
    assert attend(L, n_heads=1, n_pages=1, page_size=1, page_stride=0, token_stride=0, head_stride=0) == dev
    # scales that lie between k and v in memory
    assert append(L, type=B.DS_TYPE_E4M3, k_scale=P[20] + 65536, v_scale=P[20] + 65600) == dev
    assert attend(L, lse=None, ws=None, nws=0) == dev                           # 64 tokens: nothing to join
    assert attend(L, window=1 << 30) == dev and attend(L, n_pages=0, k=None, v=None) == dev
    assert verify(L, d=None, dscale=None, ldd=0, dtau=0.0) == dev
    assert verify(L, drafts=0, d=None, ids=None, ua=None) == dev
    assert verify(L, scale=None, dscale=None) == dev and verify(L, tt=B.DS_TYPE_F32, dt=B.DS_TYPE_BF16) == dev


def test_workspace_sizes_refuse_what_the_calls_refuse(L):
    cache = B.KvCacheDesc(**CACHE)
    size = lambda *a, **over: L.ds_cache_attention_rows_workspace(  # noqa: E731
        ctypes.addressof(B.KvCacheDesc(**{**CACHE, **over})), *a)
    assert size(4, 1, 0) == 0 and size(3, 1, 0) == S and size(4, 0, 0) == S and size(4, 1, -1) == G
    assert size(4, 1, 0, page_size=3) == S and L.ds_cache_attention_rows_workspace(None, 4, 1, 0) == N
    assert size(4, 1, 0, pages_per_seq=8) == 0                                  # one chunk of 128: nothing to join
    assert size(4, 1, 0, pages_per_seq=17) == 3 * 4 * 3 * 66 * 4                # three
    assert size(4, 1, 97, pages_per_seq=1000) == 0                              # a window within one
    assert size(4, 1, 98, pages_per_seq=1000) == 3 * 4 * 2 * 66 * 4
    assert size(4, 1, 0, pages_per_seq=1 << 25) == size(4, 1, 0, pages_per_seq=1 << 12)   # 128 chunks at most
    assert size(4, 1, 0, n_seqs=1 << 21) == 0 and size(4, 1, 0, n_seqs=(1 << 21) + 1) == S
    del cache
    f = L.ds_draft_verify_rows_workspace
    assert f(0, 3, 1000, 1) == 0 and f(5, 3, 1000, 0) > 0 and f(5, 3, 1000, 1) > f(5, 3, 1000, 0)
    assert f(-1, 3, 1000, 1) == S and f(5, 33, 1000, 1) == S and f(5, 3, 0, 1) == S and f(5, 3, 1000, 2) == G


def test_frequencies(L):
    for kw in (dict(), dict(factor=4.0), dict(base=500000.0, factor=8.0, original=8192.0, low=1.0, high=4.0),
               dict(factor=32.0, original=4096.0, low=1.0, high=32.0)):
        for rotary in (2, 20, 128, 256):
            got = B.ds_rope_frequencies(rotary, **kw).double().numpy()
            want = D.frequencies(rotary, **kw)
            assert np.abs(got / want - 1).max() <= 2.0 ** -24 * (1 + 1e-6)
    out = (ctypes.c_float * 128)()
    ok = (64, 10000.0, 1.0, 4096.0, 0.0, 0.0)
    assert L.ds_rope_frequencies(ctypes.addressof(out), *ok) == B.DS_OK
    for i, v, code in ((0, 3, S), (0, 0, S), (0, 258, S), (1, 0.0, G), (1, NAN, G), (2, 0.5, G), (2, INF, G),
                       (3, 0.0, G), (4, -1.0, G), (5, -1.0, G), (5, NAN, G)):
        bad = list(ok)
        bad[i] = v
        assert L.ds_rope_frequencies(ctypes.addressof(out), *bad) == code, bad
    assert L.ds_rope_frequencies(ctypes.addressof(out), 64, 1e4, 1.0, 1.0, 2.0, 2.0) == G
    assert L.ds_rope_frequencies(None, *ok) == N and L.ds_rope_frequencies(ctypes.addressof(out) + 2, *ok) == A
    with pytest.raises(RuntimeError, match="DS_ERR_SHAPE"):
        B.ds_rope_frequencies(7)
