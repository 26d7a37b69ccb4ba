"""The decoding step's binding: calls that an ordinary program makes
at the edge of what is allowed."""
import os

import numpy as np
import pytest
import torch

from oracle import decode_rows as D
from scale_invariant_row_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH),
                                reason="library not built (python -m scale_invariant_row_amd.build)")


def test_frequencies_are_made_on_the_host_whatever_the_default_device():
    """The library writes them with host code: memory of another device is none."""
    with torch.device("meta"):
        f = B.ds_rope_frequencies(64, 10000.0)
    assert f.device.type == "cpu"
    assert np.allclose(f.numpy(), D.frequencies(64), rtol=1e-6)


def empty_step(device):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
    c = B.KvCache(z(5, 16, 2, 64), z(5, 16, 2, 64), z(0, 4, dtype=torch.int32))
    return B.ds_cache_append_rows(c, z(0, 128), z(0, 128), z(0, dtype=torch.int32), q=z(0, 256))


def test_a_step_of_no_sequences_may_append():
    """No rows to equally many sequences, none: as attention takes it."""
    with pytest.raises(ValueError, match="cache: must be on a HIP device"):   # and no other refusal
        empty_step("cpu")


@pytest.mark.gpu
def test_a_step_of_no_sequences_appends_nothing():
    assert empty_step("cuda:0").shape == (0, 256)
