"""The decoding step's binding refuses bad arguments before any launch.

CPU tensors throughout: shape, dtype and stride checks run before the device
check, so each bad argument is named on its own, and a well-formed call stops
at the device check without reaching the library.
"""
import pytest
import torch

from scale_invariant_row_amd import binding as B

ROWS, HD, HEADS = 6, 64, 2
bf16 = torch.bfloat16


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def cache(**over):
    a = dict(k=z(5, 16, HEADS, HD, dtype=bf16), v=z(5, 16, HEADS, HD, dtype=bf16),
             page_table=z(3, 4, dtype=torch.int32))
    return B.KvCache(**{**a, **over})


def q(heads=4, rows=ROWS, **kw):
    return z(rows, heads * HD, dtype=kw.get("dtype", bf16))


pos = z(ROWS, dtype=torch.int32)
CALLS = {
    "rope": (B.ds_rope_rows, dict(q=q(), k=q(2), positions=pos, inv_freq=z(HD // 2), head_dim=HD)),
    "rope_bwd": (B.ds_rope_rows_backward, dict(dq_out=q(), dk_out=q(2), positions=pos, inv_freq=z(5), head_dim=HD)),
    "append": (B.ds_cache_append_rows, dict(cache=cache(), k=q(2), v=q(2), positions=pos, seqs=pos, inv_freq=z(8),
                                            q=q(), rms_eps=1e-6, q_weight=z(HD), k_weight=z(HD))),
    "attend": (B.ds_cache_attention_rows, dict(cache=cache(), q=q(), lens=z(3, dtype=torch.int32))),
    "verify": (B.ds_draft_verify_rows, dict(target=z(8, 50), drafted=z(2, 3, dtype=torch.int64), u_accept=z(2, 3),
                                            u_sample=z(2), draft=z(6, 50, dtype=bf16), scale=z(50),
                                            draft_scale=z(50))),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_well_formed_stops_at_the_device(name):
    f, a = CALLS[name]
    with pytest.raises(ValueError, match="must be on a HIP device"):
        f(**a)


@pytest.mark.parametrize("name,over,word", [
    ("rope", dict(q=q(dtype=torch.float32)), "q: expected a bf16"), ("rope", dict(q=q().t()), "unit column stride"),
    ("rope", dict(k=q(2, rows=5)), "k: expected 6 rows"), ("rope", dict(q=z(ROWS, 100, dtype=bf16)), "whole number"),
    ("rope", dict(positions=pos.long()), "positions"), ("rope", dict(inv_freq=z(33)), "inv_freq"),
    ("rope", dict(inv_freq=z(0)), "inv_freq"), ("rope", dict(inv_freq=z(32, dtype=torch.float64)), "inv_freq"),
    ("rope", dict(head_dim=0), "head_dim"), ("rope", dict(q_out=q(3)), "q_out"),
    ("rope", dict(k=None, k_out=q(2)), "k_out: given without"),
    ("rope_bwd", dict(dk_out=q(2, rows=7)), "dk_out: expected 6 rows"), ("rope_bwd", dict(dq=q(5)), "dq"),
    ("append", dict(k=q(3)), "k: expected 2 heads"), ("append", dict(v=q(1)), "v: expected 2 heads"),
    ("append", dict(v=q(2, rows=5)), "v: expected 6 rows"), ("append", dict(q=q(rows=7)), "q: expected 6 rows"),
    ("append", dict(positions=pos[:5]), "positions"), ("append", dict(seqs=pos.float()), "seqs"),
    ("append", dict(inv_freq=z(40)), "inv_freq"), ("append", dict(rms_eps=None), "rms_eps"),
    ("append", dict(q_weight=z(HD + 1)), "q_weight"), ("append", dict(k_weight=z(HD, dtype=bf16)), "k_weight"),
    ("append", dict(q=None, q_weight=None, q_out=q()), "q_out"), ("append", dict(q_out=q(3)), "q_out"),
    ("append", dict(seqs=None, k=q(2, rows=5), v=q(2, rows=5), q=None, positions=pos[:5]), "seqs: needed"),
    ("attend", dict(q=q(3)), "multiple of the cache's 2"), ("attend", dict(q=q(rows=7)), "equally many rows"),
    ("attend", dict(q=q(rows=0)), "equally many rows"), ("attend", dict(q=q(rows=51)), "at most 16"),
    ("attend", dict(lens=z(4, dtype=torch.int32)), "lens"), ("attend", dict(lens=z(3)), "lens"),
    ("attend", dict(window=-1), "window"), ("attend", dict(out=q(2)), "out"), ("attend", dict(out=q(rows=5)), "out"),
    ("verify", dict(target=z(7, 50)), "target: expected 8 rows"), ("verify", dict(target=z(8, 50).double()), "target"),
    ("verify", dict(drafted=z(2, 3)), "drafted"), ("verify", dict(drafted=z(6, dtype=torch.int64)), "drafted"),
    ("verify", dict(drafted=z(1, 33, dtype=torch.int32)), "at most 32"),
    ("verify", dict(u_accept=z(2, 4)), "u_accept"), ("verify", dict(u_sample=z(3)), "u_sample"),
    ("verify", dict(draft=z(6, 51)), "draft: expected"), ("verify", dict(draft=z(8, 50)), "draft: expected"),
    ("verify", dict(scale=z(49)), "scale"), ("verify", dict(draft_scale=z(49)), "draft_scale"),
])
def test_bad_argument_is_named(name, over, word):
    f, a = CALLS[name]
    with pytest.raises((ValueError, TypeError), match=word):
        f(**{**a, **over})


@pytest.mark.parametrize("over,word", [
    (dict(k=z(5, 16, HEADS, HD)), "k: expected bf16 or e4m3"), (dict(v=z(5, 16, HEADS, HD)), "v: expected bf16"),
    (dict(k=z(5, 16, HD, dtype=bf16)), "k: expected a"), (dict(v=z(4, 16, HEADS, HD, dtype=bf16)), "v: must be like k"),
    (dict(v=z(5, HEADS, 16, HD, dtype=bf16).transpose(1, 2)), "laid out like k"),
    (dict(k=z(5, 16, HD, HEADS, dtype=bf16).transpose(2, 3)), "unit stride"),
    (dict(page_table=z(3, 4)), "page_table"), (dict(page_table=z(12, dtype=torch.int32)), "page_table"),
    (dict(page_table=z(4, 3, dtype=torch.int32).t()), "page_table"), (dict(k_scale=z(3)), "k_scale"),
    (dict(v_scale=z(2, dtype=bf16)), "v_scale"),
])
def test_bad_cache_is_named(over, word):
    with pytest.raises((ValueError, TypeError), match=word):
        cache(**over)


def test_a_dimension_past_32_bits_is_refused():
    wide = z(1, 1, 1, 16, dtype=bf16).expand((1 << 32) + 1, 1, 1, 16)
    with pytest.raises(ValueError, match="2\\^31"):
        cache(k=wide, v=wide)
    with pytest.raises(ValueError, match="2\\^31"):
        cache(page_table=z(1, 4, dtype=torch.int32).expand((1 << 32) + 3, 4))


def test_a_caches_description():
    c = cache()
    assert (c.desc.page_stride, c.desc.token_stride, c.desc.head_stride) == (16 * HEADS * HD, HEADS * HD, HD)
    t = z(5, HEADS, 16, HD, dtype=torch.float8_e4m3fn).transpose(1, 2)
    c = cache(k=t, v=t.clone(memory_format=torch.preserve_format), page_table=z(3, 9, dtype=torch.int32)[:, :4])
    assert (c.desc.token_stride, c.desc.head_stride, c.desc.type) == (HD, 16 * HD, B.DS_TYPE_E4M3)
    assert (c.desc.ld_table, c.desc.pages_per_seq, c.desc.n_seqs, c.desc.page_size) == (9, 4, 3, 16)
    c = cache(k=z(1, 1, 1, 16, dtype=bf16), v=z(1, 1, 1, 16, dtype=bf16), page_table=z(1, 9, dtype=torch.int32)[:, :4])
    assert (c.desc.page_stride, c.desc.token_stride, c.desc.head_stride, c.desc.ld_table) == (0, 0, 0, 4)


def test_a_cache_stays_as_it_was_made():
    c = cache()
    with pytest.raises(AttributeError, match="make another"):
        c.k = c.v
    c.page_table.set_(z(3, 4, dtype=torch.int32))                 # other memory under the same tensor
    for f, a in (CALLS["append"], CALLS["attend"]):
        with pytest.raises(ValueError, match="other memory"):
            f(**{**a, "cache": c})
