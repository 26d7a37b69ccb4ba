"""Helpers of the decoding step's GPU tests: paged caches filled from numpy
values, in either order of memory and either type."""
import numpy as np

from oracle import decode_rows as D
from token_util import bf16_round, dev

HALF_E4M3 = 2.0 ** -4       # half a step of e4m3, relative
LEAST_E4M3 = 2.0 ** -10     # half a step below its normal range, absolute


def e4m3_round(a) -> np.ndarray:
    """Float array -> the nearest e4m3 values (the largest past the range), as float32."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).clamp(-D.E4M3_MAX, D.E4M3_MAX)
    return t.to(torch.float8_e4m3fn).float().numpy()


def values_of(t) -> np.ndarray:
    """A cache tensor's values as float64 on the host."""
    return t.float().cpu().numpy().astype(np.float64)


class Paged:
    """A cache of n_pages pages whose k and v (float arrays [pages, page, heads,
    hd]) are on the GPU as `kind`, in memory order `order`:
      "token": [pages, page, heads, hd]   "head": [pages, heads, page, hd]
      "both":  k and v in one buffer, [pages, page, k|v, heads, hd]
      "wide":  as "token", with unused elements after every head, token and page
    """

    def __init__(self, B, k, v, table, kind="bf16", order="token", k_scale=None, v_scale=None):
        import torch
        self.kind, self.k_scale, self.v_scale = kind, k_scale, v_scale
        self.table = np.asarray(table, np.int32)
        dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        pages, page, heads, hd = k.shape
        at = np.uint8 if kind != "bf16" else None

        def make(a):
            t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda:0")
            return t.to(dtype) if at is None else t.clamp(-448, 448).to(dtype)

        tk, tv = make(k), make(v)
        self.store = None
        if order == "head":
            tk, tv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (tk, tv))
        elif order in ("both", "wide"):
            raw = torch.uint8 if dtype == torch.float8_e4m3fn else torch.int16
            if order == "both":
                self.store = torch.full((pages, page, 2, heads, hd), 85, dtype=raw, device="cuda:0")
                views = self.store[:, :, 0], self.store[:, :, 1]
            else:
                self.store = torch.full((2, pages, page + 1, heads + 1, hd + 16), 85, dtype=raw, device="cuda:0")
                views = tuple(self.store[i][:, :page, :heads, :hd] for i in (0, 1))
            for view, t in zip(views, (tk, tv)):
                view.copy_(t.view(raw))
            tk, tv = (view.view(dtype) for view in views)
        self.k, self.v = tk, tv
        opt = lambda s: None if s is None else dev(np.asarray(s, np.float32))  # noqa: E731
        self.cache = B.KvCache(tk, tv, dev(self.table), opt(k_scale), opt(v_scale))

    def bits(self):
        """Everything that the buffers hold, gaps too."""
        import torch
        raw = torch.uint8 if self.kind != "bf16" else torch.int16
        if self.store is not None:
            return [self.store.cpu().numpy()]
        return [t.contiguous().view(raw).cpu().numpy() for t in (self.k, self.v)]


def random_pages(rng, shape, kind, sd=1.0):
    """(k, v) values that the cache's type holds exactly."""
    a = rng.standard_normal((2, *shape)) * sd
    return bf16_round(a) if kind == "bf16" else e4m3_round(a)
