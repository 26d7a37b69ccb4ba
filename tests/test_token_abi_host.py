"""ds_token_rows.h without a GPU: symbols, workspace sizes, argument checks.

Every refused call returns before its first HIP call (fake pointer values are
never dereferenced).  Calls with valid arguments are made only where no HIP
device exists, where they must stop at DS_ERR_DEVICE.
"""
import os

import pytest

from scale_invariant_row_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH),
                                reason="library not built (python -m scale_invariant_row_amd.build)")

P = [0x10000000 * (i + 1) for i in range(24)]       # fake, aligned, far apart
BIG = 1 << 26                                       # a workspace size that suffices everywhere
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return B._token_lib()


def test_exports_every_declared_function(L):
    names = B.header_functions(B.TOKEN_HEADER)
    assert set(names) == {
        "ds_embed_rows", "ds_embed_rows_backward", "ds_embed_rows_backward_workspace",
        "ds_qk_rows_rms", "ds_qk_rows_rms_backward", "ds_qk_rows_rms_backward_workspace",
        "ds_logprob_rows", "ds_logprob_rows_workspace", "ds_logprob_rows_backward",
        "ds_logprob_rows_backward_workspace"}
    for n in names:
        assert hasattr(L, n), n


def test_workspace_status_has_a_text():
    assert B.ds_status_string(B.DS_ERR_WORKSPACE).startswith("DS_ERR_WORKSPACE")


class Call:
    """Keyword arguments over a valid call."""

    def __init__(self, name, **base):
        self.name, self.base = name, base

    def __call__(self, L, **over):
        assert set(over) <= set(self.base), over
        return getattr(L, self.name)(*{**self.base, **over}.values())


embed = Call("ds_embed_rows", table=P[0], type=B.DS_TYPE_F32, vocab=100, ids=P[1], id_bytes=8,
             scale=1.0, out=P[2], rows=10, cols=64, stream=None)
embed_bwd = Call("ds_embed_rows_backward", dy=P[0], ids=P[1], id_bytes=8, scale=1.0, dtable=P[2],
                 type=B.DS_TYPE_F32, accumulate=0, vocab=100, rows=10, cols=64, ws=P[3], nws=BIG,
                 stream=None)
qk = Call("ds_qk_rows_rms", q=P[0], ldq=256, k=P[1], ldk=128, pos=P[2], inv=P[3], qw=P[4], kw=P[5],
          qo=P[6], ldqo=256, ko=P[7], ldko=128, rows=10, nq=4, nk=2, hd=64, eps=1e-6, stream=None)
qk_bwd = Call("ds_qk_rows_rms_backward", q=P[0], ldq=256, k=P[1], ldk=128, pos=P[2], inv=P[3],
              qw=P[4], kw=P[5], dqo=P[6], lddqo=256, dko=P[7], lddko=128, dq=P[8], lddq=256,
              dk=P[9], lddk=128, dqw=P[10], dkw=P[11], rows=10, nq=4, nk=2, hd=64, eps=1e-6,
              ws=P[12], nws=BIG, stream=None)
score = Call("ds_logprob_rows", x=P[0], type=B.DS_TYPE_BF16, ld=1000, scale=P[1], tau=1.0,
             labels=P[2], label_bytes=8, logp=P[3], ent=P[4], lse=P[5], ids=P[6], top=P[7],
             top_k=5, rows=10, vocab=1000, ws=P[8], nws=BIG, stream=None)
score_bwd = Call("ds_logprob_rows_backward", x=P[0], type=B.DS_TYPE_BF16, ld=1000, scale=P[1],
                 tau=1.0, labels=P[2], label_bytes=8, lse=P[3], ent=P[4], dlogp=P[5], dent=P[6],
                 dx=P[7], ldo=1000, dscale=P[8], rows=10, vocab=1000, ws=P[9], nws=BIG, stream=None)
EVERY = [embed, embed_bwd, qk, qk_bwd, score, score_bwd]


def no_device():
    import torch
    return torch.cuda.device_count() == 0


@pytest.mark.skipif("not no_device()")
@pytest.mark.parametrize("call", EVERY, ids=lambda c: c.name)
def test_valid_arguments_reach_the_device(L, call):
    assert call(L) == B.DS_ERR_DEVICE


@pytest.mark.parametrize("call,over,code", [
    (embed, dict(table=None), B.DS_ERR_NULL), (embed, dict(ids=None), B.DS_ERR_NULL),
    (embed, dict(out=None), B.DS_ERR_NULL), (embed, dict(rows=-1), B.DS_ERR_SHAPE),
    (embed, dict(cols=60), B.DS_ERR_SHAPE), (embed, dict(cols=0), B.DS_ERR_SHAPE),
    (embed, dict(cols=65544), B.DS_ERR_SHAPE), (embed, dict(vocab=-1), B.DS_ERR_SHAPE),
    (embed, dict(vocab=1 << 31), B.DS_ERR_SHAPE), (embed, dict(rows=1 << 60), B.DS_ERR_SHAPE),
    (embed, dict(type=2), B.DS_ERR_ARG), (embed, dict(id_bytes=2), B.DS_ERR_ARG),
    (embed, dict(scale=NAN), B.DS_ERR_ARG), (embed, dict(scale=INF), B.DS_ERR_ARG),
    (embed, dict(table=P[0] + 8), B.DS_ERR_ALIGN), (embed, dict(out=P[2] + 2), B.DS_ERR_ALIGN),
    (embed, dict(ids=P[1] + 4), B.DS_ERR_ALIGN), (embed, dict(out=P[0] + 64), B.DS_ERR_ARG),
    (embed, dict(out=P[1]), B.DS_ERR_ARG),
    (embed_bwd, dict(dy=None), B.DS_ERR_NULL), (embed_bwd, dict(ids=None), B.DS_ERR_NULL),
    (embed_bwd, dict(dtable=None), B.DS_ERR_NULL), (embed_bwd, dict(rows=1 << 31), B.DS_ERR_SHAPE),
    (embed_bwd, dict(rows=1 << 30, cols=1024), B.DS_ERR_SHAPE),       # 2 TiB of rows
    (embed_bwd, dict(vocab=1 << 28, cols=1024), B.DS_ERR_SHAPE),      # 1 TiB of table
    (embed_bwd, dict(cols=12), B.DS_ERR_SHAPE), (embed_bwd, dict(accumulate=2), B.DS_ERR_ARG),
    (embed_bwd, dict(type=7), B.DS_ERR_ARG), (embed_bwd, dict(scale=-INF), B.DS_ERR_ARG),
    (embed_bwd, dict(dy=P[0] + 8), B.DS_ERR_ALIGN), (embed_bwd, dict(dtable=P[0]), B.DS_ERR_ARG),
    (embed_bwd, dict(dtable=P[1] + 16), B.DS_ERR_ARG),
    (qk, dict(q=None), B.DS_ERR_NULL), (qk, dict(ko=None), B.DS_ERR_NULL),
    (qk, dict(pos=None), B.DS_ERR_NULL), (qk, dict(inv=None), B.DS_ERR_NULL),
    (qk, dict(hd=24), B.DS_ERR_SHAPE), (qk, dict(hd=272), B.DS_ERR_SHAPE),
    (qk, dict(hd=0), B.DS_ERR_SHAPE), (qk, dict(nq=-1), B.DS_ERR_SHAPE),
    (qk, dict(ldq=248), B.DS_ERR_SHAPE), (qk, dict(ldko=132), B.DS_ERR_SHAPE),
    (qk, dict(rows=1 << 61), B.DS_ERR_SHAPE), (qk, dict(eps=-1.0), B.DS_ERR_ARG),
    (qk, dict(eps=NAN), B.DS_ERR_ARG), (qk, dict(q=P[0] + 2), B.DS_ERR_ALIGN),
    (qk, dict(qw=P[4] + 4), B.DS_ERR_ALIGN), (qk, dict(pos=P[2] + 1), B.DS_ERR_ALIGN),
    (qk, dict(qo=P[0] + 16), B.DS_ERR_ARG), (qk, dict(qo=P[1]), B.DS_ERR_ARG),
    (qk, dict(ko=P[6] + 128), B.DS_ERR_ARG), (qk, dict(qo=P[3]), B.DS_ERR_ARG),
    (qk, dict(qo=P[0], ldqo=264), B.DS_ERR_ARG),
    (qk_bwd, dict(dqo=None), B.DS_ERR_NULL), (qk_bwd, dict(dk=None), B.DS_ERR_NULL),
    (qk_bwd, dict(ws=None), B.DS_ERR_NULL), (qk_bwd, dict(nws=16), B.DS_ERR_WORKSPACE),
    (qk_bwd, dict(ws=P[12] + 4), B.DS_ERR_ALIGN), (qk_bwd, dict(dqw=P[10] + 2), B.DS_ERR_ALIGN),
    (qk_bwd, dict(dq=P[7]), B.DS_ERR_ARG), (qk_bwd, dict(dq=P[6] + 32), B.DS_ERR_ARG),
    (qk_bwd, dict(dqw=P[11] + 4), B.DS_ERR_ARG), (qk_bwd, dict(dqw=P[0] + 4), B.DS_ERR_ARG),
    (qk_bwd, dict(dkw=P[8]), B.DS_ERR_ARG), (qk_bwd, dict(ws=P[8]), B.DS_ERR_ARG),
    (qk_bwd, dict(ws=P[10]), B.DS_ERR_ARG), (qk_bwd, dict(hd=8), B.DS_ERR_SHAPE),
    (qk_bwd, dict(lddqo=8), B.DS_ERR_SHAPE),
    (score, dict(x=None), B.DS_ERR_NULL), (score, dict(labels=None), B.DS_ERR_NULL),
    (score, dict(ids=None), B.DS_ERR_NULL), (score, dict(top=None), B.DS_ERR_NULL),
    (score, dict(vocab=0), B.DS_ERR_SHAPE), (score, dict(vocab=1 << 21, ld=1 << 21), B.DS_ERR_SHAPE),
    (score, dict(ld=999), B.DS_ERR_SHAPE), (score, dict(top_k=33), B.DS_ERR_SHAPE),
    (score, dict(top_k=-1), B.DS_ERR_SHAPE), (score, dict(vocab=3, ld=3), B.DS_ERR_SHAPE),
    (score, dict(rows=-2), B.DS_ERR_SHAPE), (score, dict(tau=0.0), B.DS_ERR_ARG),
    (score, dict(tau=-1.0), B.DS_ERR_ARG), (score, dict(tau=NAN), B.DS_ERR_ARG),
    (score, dict(type=3), B.DS_ERR_ARG), (score, dict(label_bytes=1), B.DS_ERR_ARG),
    (score, dict(x=P[0] + 1), B.DS_ERR_ALIGN), (score, dict(type=B.DS_TYPE_F32, x=P[0] + 2), B.DS_ERR_ALIGN),
    (score, dict(labels=P[2] + 4), B.DS_ERR_ALIGN), (score, dict(logp=P[3] + 2), B.DS_ERR_ALIGN),
    (score, dict(logp=P[0] + 4), B.DS_ERR_ARG), (score, dict(ent=P[5] + 4), B.DS_ERR_ARG),
    (score, dict(top=P[6] + 8), B.DS_ERR_ARG), (score, dict(lse=P[1]), B.DS_ERR_ARG),
    (score_bwd, dict(lse=None), B.DS_ERR_NULL), (score_bwd, dict(labels=None), B.DS_ERR_NULL),
    (score_bwd, dict(ent=None), B.DS_ERR_NULL), (score_bwd, dict(dx=None), B.DS_ERR_NULL),
    (score_bwd, dict(scale=None), B.DS_ERR_ARG), (score_bwd, dict(ldo=10), B.DS_ERR_SHAPE),
    (score_bwd, dict(dx=P[0] + 2), B.DS_ERR_ARG), (score_bwd, dict(dx=P[0], ldo=1008), B.DS_ERR_ARG),
    (score_bwd, dict(dscale=P[1]), B.DS_ERR_ARG), (score_bwd, dict(dscale=P[7] + 4), B.DS_ERR_ARG),
    (score_bwd, dict(dx=P[3]), B.DS_ERR_ARG), (score_bwd, dict(dscale=P[8] + 1), B.DS_ERR_ALIGN),
    (score_bwd, dict(tau=INF), B.DS_ERR_ARG),
], ids=lambda v: getattr(v, "name", None) or (str(v) if isinstance(v, dict) else None))
def test_refused(L, call, over, code):
    assert call(L, **over) == code


@pytest.mark.parametrize("call", EVERY, ids=lambda c: c.name)
def test_no_rows_is_a_noop(L, call):
    """Nothing to write: pointers are not looked at, no device is needed."""
    none = {k: None for k, v in call.base.items() if isinstance(v, int) and v in P}
    over = dict(none, rows=0)
    if call is embed_bwd:
        over["vocab"] = 0
    if "nws" in call.base:
        over["nws"] = 0
    assert call(L, **over) == B.DS_OK


@pytest.mark.skipif("not no_device()")
def test_in_place_and_fused_slices_are_allowed(L):
    assert qk(L, qo=P[0], ko=P[1]) == B.DS_ERR_DEVICE
    # q and k as slices of one projection row, outputs in place
    assert qk(L, q=P[0], ldq=512, k=P[0] + 512, ldk=512, qo=P[0], ldqo=512, ko=P[0] + 512,
              ldko=512) == B.DS_ERR_DEVICE
    assert qk_bwd(L, dq=P[6], dk=P[7]) == B.DS_ERR_DEVICE
    assert qk_bwd(L, dq=P[0], dk=P[1]) == B.DS_ERR_DEVICE
    assert qk_bwd(L, dqw=None, dkw=None, ws=None, nws=0) == B.DS_ERR_DEVICE
    assert score_bwd(L, dx=P[0]) == B.DS_ERR_DEVICE
    assert score_bwd(L, dscale=None, ws=None, nws=0) == B.DS_ERR_DEVICE
    assert score_bwd(L, dlogp=None, labels=None) == B.DS_ERR_DEVICE
    assert embed(L, table=None, vocab=0) == B.DS_ERR_DEVICE


def test_workspace_sizes_refuse_what_the_calls_refuse(L):
    assert L.ds_embed_rows_backward_workspace(100, -1, 64) == B.DS_ERR_SHAPE
    assert L.ds_embed_rows_backward_workspace(100, 1 << 31, 64) == B.DS_ERR_SHAPE
    assert L.ds_qk_rows_rms_backward_workspace(10, 4, 2, 24) == B.DS_ERR_SHAPE
    assert L.ds_logprob_rows_workspace(10, 0, 0) == B.DS_ERR_SHAPE
    assert L.ds_logprob_rows_workspace(10, 100, 40) == B.DS_ERR_SHAPE
    assert L.ds_logprob_rows_backward_workspace(-1, 100) == B.DS_ERR_SHAPE
    for n in (L.ds_embed_rows_backward_workspace(100, 0, 64),
              L.ds_qk_rows_rms_backward_workspace(0, 4, 2, 64),
              L.ds_logprob_rows_workspace(0, 100, 5), L.ds_logprob_rows_backward_workspace(0, 100)):
        assert 0 <= n < BIG
