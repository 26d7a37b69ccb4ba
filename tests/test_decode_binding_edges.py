"""The decoding step's binding without a GPU: calls that an ordinary program makes
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
