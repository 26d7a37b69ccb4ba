"""Helpers of the token row tests: inputs with exact bf16 values, comparisons
against a float64 value with a stated bound."""
import numpy as np

U = 2.0 ** -24              # half a step of fp32, relative
HALF_BF16 = 2.0 ** -8       # half a step of bf16, relative


def bf16_round(a) -> np.ndarray:
    """Float array -> the nearest bf16 values, as float32."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().float().numpy()


def dev(a, dtype=None):
    """numpy -> tensor on cuda:0 (floats as fp32 unless ``dtype`` is given)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    return t if dtype is None else t.to(dtype)


def host(t) -> np.ndarray:
    import torch
    if t.dtype == torch.bfloat16:
        t = t.float()
    return t.detach().cpu().numpy()


def close(got, want, bound, what: str, bf16: bool = False):
    """|got - want| <= bound (+ half a bf16 step of want), and the same
    non-finite values in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, f"{what}: shape {got.shape}, expected {want.shape}"
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), \
        f"{what}: non-finite values differ at {np.argwhere(np.isfinite(got) != fine)[:4].tolist()}"
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), f"{what}: non-finite values"
    b = np.broadcast_to(np.asarray(bound, np.float64), want.shape) + 1e-36
    if bf16:
        b = b * (1 + HALF_BF16) + HALF_BF16 * np.abs(np.where(fine, want, 0.0))
    with np.errstate(invalid="ignore"):
        off = np.where(fine, np.abs(got - want), 0.0)
    bad = off > np.where(fine, b, np.inf)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} beyond the bound, first at {i}: got "
                             f"{got[i]!r}, want {want[i]!r}, bound {b[i]:.3g}")


def bits(t):
    """A tensor's bits as whole numbers, for exact comparisons."""
    import torch
    return t.view({2: torch.int16, 4: torch.int32}[t.element_size()])
