"""The decoding step's oracle at the edges of its arguments."""
import numpy as np

from oracle import decode_rows as D


def test_a_target_row_that_says_nothing_refuses_a_random_number_below_0():
    z = np.zeros((3, 5), np.float32)
    z[0] = -np.inf
    z[1, 2] = np.nan
    for row, d in ((0, None), (1, None), (0, np.zeros((1, 5), np.float32))):
        tokens, logp, _ = D.verify_sequence(z[[row, 2]], d, [3], [-0.5], 0.5)
        assert tokens == [-1] and logp == [0.0]
