"""The token rows' binding refuses bad arguments before any launch.

CPU tensors throughout: shape, dtype and stride checks run before the device
check, so each bad argument is named on its own, and a well-formed call stops
at the device check without reaching the library.
"""
import pytest
import torch

from scale_invariant_row_amd import binding as B

ROWS, HD = 6, 64
bf16 = torch.bfloat16


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


CALLS = {
    "embed": (lambda **a: B.ds_embed_rows(**a),
              dict(table=z(9, 16), ids=z(ROWS, dtype=torch.int64))),
    "embed_bwd": (lambda **a: B.ds_embed_rows_backward(**a),
                  dict(dy=z(ROWS, 16, dtype=bf16), ids=z(ROWS, dtype=torch.int32), vocab=9)),
    "qk": (lambda **a: B.ds_qk_rows_rms(**a),
           dict(q=z(ROWS, 3 * HD, dtype=bf16), k=z(ROWS, HD, dtype=bf16),
                positions=z(ROWS, dtype=torch.int32), inv_freq=z(HD // 2), q_weight=z(HD),
                k_weight=z(HD), head_dim=HD)),
    "score": (lambda **a: B.ds_logprob_rows(**a),
              dict(logits=z(ROWS, 50), labels=z(ROWS, dtype=torch.int64))),
    "score_bwd": (lambda **a: B.ds_logprob_rows_backward(**a),
                  dict(logits=z(ROWS, 50), labels=z(ROWS, dtype=torch.int64), lse=z(ROWS),
                       entropy=z(ROWS), dlogp=z(ROWS))),
}
CALLS["qk_bwd"] = (lambda **a: B.ds_qk_rows_rms_backward(**a),
                   dict(CALLS["qk"][1], dq_out=z(ROWS, 3 * HD, dtype=bf16), dk_out=z(ROWS, HD, dtype=bf16)))


@pytest.mark.parametrize("name", sorted(CALLS))
def test_well_formed_stops_at_the_device(name):
    f, a = CALLS[name]
    with pytest.raises(ValueError, match="HIP device"):
        f(**a)


@pytest.mark.parametrize("name,over,error,match", [
    ("embed", dict(table=z(9, 16, dtype=torch.float16)), TypeError, "^table"),
    ("embed", dict(table=z(16, 9).t()), ValueError, "^table"),
    ("embed", dict(ids=z(ROWS)), ValueError, "^ids"),
    ("embed", dict(ids=z(2, ROWS, dtype=torch.int64)), ValueError, "^ids"),
    ("embed", dict(ids=z(2 * ROWS, dtype=torch.int64)[::2]), ValueError, "^ids"),
    ("embed", dict(out=z(ROWS, 16)), TypeError, "^out"),
    ("embed", dict(out=z(ROWS, 8, dtype=bf16)), ValueError, "^out"),
    ("embed_bwd", dict(dy=z(ROWS, 16)), TypeError, "^dy"),
    ("embed_bwd", dict(ids=z(ROWS + 1, dtype=torch.int32)), ValueError, "^ids"),
    ("embed_bwd", dict(vocab=-1), ValueError, "^vocab"),
    ("embed_bwd", dict(dtable=z(8, 16)), ValueError, "^dtable"),
    ("embed_bwd", dict(dtable=z(9, 16, dtype=torch.float64)), TypeError, "^dtable"),
    ("embed_bwd", dict(dtable=z(9, 16), dtype=bf16), ValueError, "^dtable"),
    ("embed_bwd", dict(accumulate=True), ValueError, "^dtable"),
    ("embed_bwd", dict(dtype=torch.float16), TypeError, "^dtype"),
    ("qk", dict(q=z(ROWS, 3 * HD)), ValueError, "^q"),
    ("qk", dict(q=z(ROWS, 3 * HD + 8, dtype=bf16)), ValueError, "^q: its width"),
    ("qk", dict(k=z(ROWS + 1, HD, dtype=bf16)), ValueError, "^k: expected 6 rows"),
    ("qk", dict(k=z(HD, ROWS, dtype=bf16).t()), ValueError, "^k: expected a bf16"),
    ("qk", dict(positions=z(ROWS, dtype=torch.int64)), ValueError, "^positions"),
    ("qk", dict(inv_freq=z(HD)), ValueError, "^inv_freq"),
    ("qk", dict(q_weight=z(HD, dtype=bf16)), ValueError, "^q_weight"),
    ("qk", dict(k_weight=z(2 * HD)[::2]), ValueError, "^k_weight"),
    ("qk", dict(q_out=z(ROWS, 2 * HD, dtype=bf16)), ValueError, "^q_out"),
    ("qk", dict(k=None, k_out=z(ROWS, HD, dtype=bf16)), ValueError, "^k_out: given without k"),
    ("qk", dict(head_dim=0), ValueError, "^head_dim"),
    ("qk_bwd", dict(dq_out=z(ROWS, HD, dtype=bf16)), ValueError, "^dq_out"),
    ("qk_bwd", dict(dk_out=None), ValueError, "^dk_out"),
    ("qk_bwd", dict(dq=z(ROWS - 1, 3 * HD, dtype=bf16)), ValueError, "^dq"),
    ("qk_bwd", dict(dk=z(ROWS, 2 * HD, dtype=bf16)), ValueError, "^dk"),
    ("score", dict(logits=z(ROWS, 50, dtype=torch.float16)), TypeError, "^logits"),
    ("score", dict(logits=z(50, ROWS).t()), ValueError, "^logits"),
    ("score", dict(labels=z(ROWS)), ValueError, "^labels"),
    ("score", dict(labels=z(5, dtype=torch.int64)), ValueError, "^labels"),
    ("score", dict(scale=z(49)), ValueError, "^scale"),
    ("score", dict(top_k=33), ValueError, "^top_k"),
    ("score", dict(top_k=-1), ValueError, "^top_k"),
    ("score", dict(logits=z(ROWS, 4), top_k=5), ValueError, "^top_k"),
    ("score_bwd", dict(labels=None), ValueError, "^labels"),
    ("score_bwd", dict(lse=None), ValueError, "^lse"),
    ("score_bwd", dict(entropy=None, dentropy=z(ROWS)), ValueError, "^entropy"),
    ("score_bwd", dict(dlogp=z(ROWS, dtype=torch.float64)), ValueError, "^dlogp"),
    ("score_bwd", dict(dlogits=z(ROWS, 51)), ValueError, "^dlogits"),
    ("score_bwd", dict(dlogits=z(ROWS, 50, dtype=bf16)), ValueError, "^dlogits"),
    ("score_bwd", dict(scale=z(50, dtype=bf16)), ValueError, "^scale"),
])
def test_bad_argument_named(name, over, error, match):
    f, a = CALLS[name]
    with pytest.raises(error, match=match):
        f(**{**a, **over})
