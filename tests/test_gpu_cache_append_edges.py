"""ds_cache_append_rows on the GPU at the edges of its scales, beside the cases of
test_gpu_cache_append.py."""
import numpy as np
import pytest

from decode_util import Paged, values_of
from gpu_util import announce
from token_util import bf16_round, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from scale_invariant_row_amd import binding
    binding._decode_lib()
    return binding


SCALES = [1.0, 2.0 ** -120, 2.0 ** -127, 1.3e-38, 2.9e-39, 2.0 ** -129, 7e-41, 1.4e-45, 2.0 ** 120, 2.5e38, 3.4e38, np.inf]


def test_quotients_by_scales_of_any_size(B):
    """Values up to 600 times a head's scale, zeros among them: the fp32 quotient,
    rounded to e4m3 once (numpy's division keeps denormals, as the kernel's)."""
    import torch
    rng = np.random.default_rng(50)
    heads, hd, rows = len(SCALES), 32, 40
    scale = np.array(SCALES, np.float32)
    finite = np.where(np.isfinite(scale), scale, 1.0).astype(np.float64)
    x = finite[:, None] * 2.0 ** rng.uniform(-12, 9.2, (rows, heads, hd)) * rng.choice([-1, 1], (rows, heads, hd))
    x = bf16_round(np.clip(x, -3e38, 3e38).reshape(rows, -1)).reshape(rows, heads, hd)
    x[:, :, ::7] = 0
    x[3, :, 5], x[4, :, 6] = np.inf, -np.inf
    x[5, :, 8] = np.nan
    cache = Paged(B, np.zeros((rows, 1, heads, hd)), np.zeros((rows, 1, heads, hd)), np.arange(rows)[None], "e4m3",
                  k_scale=scale, v_scale=scale[::-1].copy())
    t = dev(x.reshape(rows, -1), torch.bfloat16)
    back = dev(x[:, ::-1].reshape(rows, -1), torch.bfloat16)
    announce("append by scales of any size")
    B.ds_cache_append_rows(cache.cache, t, back, dev(np.arange(rows, dtype=np.int32)), seqs=dev(np.zeros(rows, np.int32)))
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        quotient = x.astype(np.float32) / scale[:, None]
    want = torch.from_numpy(quotient).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(values_of(cache.k)[:, 0], want, equal_nan=True)
    assert np.array_equal(values_of(cache.v)[:, 0], want[:, ::-1], equal_nan=True)
