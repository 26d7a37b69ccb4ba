"""Batches of the decoding step captured into graphs and run beside each other:
every replay, on inputs changed in place, gives the eager call's bits."""
import numpy as np
import pytest

from gpu_util import announce
from test_gpu_cache_attention import Case as Attend
from test_gpu_draft_verify import Case as Drafts
from token_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


def captured(call):
    import torch
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


def same(a, b):
    import torch
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("seqs,drafts,vocab,certain", [(300, 2, 9001, False), (64, 4, 40000, True), (5, 3, 9001, False)])
def test_verification_replayed(B, seqs, drafts, vocab, certain):
    import torch
    c = Drafts(seqs, drafts, vocab, 80, certain=certain, noise=0.4)
    a, kw = c.args()
    announce("verify replayed", seqs, drafts, vocab, certain)
    graph, out = captured(lambda: B.ds_draft_verify_rows(*a, **kw))
    for seed in range(4):
        rng = np.random.default_rng(seed)
        a[2].copy_(dev(rng.random((seqs, drafts)).astype(np.float32)))
        a[3].copy_(dev(rng.random(seqs).astype(np.float32)))
        a[0].copy_(a[0].roll(7, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, B.ds_draft_verify_rows(*a, **kw))


@pytest.mark.parametrize("heads,group,new,kind,window", [(2, 4, 1, "bf16", 0), (2, 7, 5, "bf16", 0), (3, 2, 3, "e4m3", 300)])
def test_attention_replayed(B, heads, group, new, kind, window):
    import torch
    c = Attend([2000, 700, 40, 5], heads, group, 64, 16, 81, new, window, kind)
    cache, q, lens = c.paged(B).cache, dev(c.q, torch.bfloat16), dev(c.lens)
    call = lambda: B.ds_cache_attention_rows(cache, q, lens, window=window, want_lse=True)  # noqa: E731
    announce("attention replayed", heads, group, new, kind, window)
    graph, out = captured(call)
    for lengths in ([2000, 700, 40, 5], [1, 0, 2000, 1999], [128, 129, 127, 2000], [0, 0, 0, 0]):
        lens.copy_(dev(np.array(lengths, np.int32)))
        q.mul_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, call())


def test_batches_beside_each_other(B):
    """Verification and attention of two batches each on four streams."""
    import torch
    drafts = [Drafts(200, 2, 9001, 82 + i, certain=bool(i)) for i in range(2)]
    attends = [Attend([3000, 90, 700], 2, 4 + 3 * i, 64, 16, 84 + i, 2) for i in range(2)]
    calls = []
    for c in drafts:
        a, kw = c.args()
        calls.append(lambda a=a, kw=kw: B.ds_draft_verify_rows(*a, **kw))
    for c in attends:
        cache, q, lens = c.paged(B).cache, dev(c.q, torch.bfloat16), dev(c.lens)
        calls.append(lambda cache=cache, q=q, lens=lens: B.ds_cache_attention_rows(cache, q, lens, want_lse=True))
    announce("batches on four streams")
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(8):
        for i, (call, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(call())
    torch.cuda.synchronize()
    for results, w in zip(got, want):
        assert all(same(r, w) for r in results)
