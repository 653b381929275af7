"""Paged K+V caches for the tests: device tensors and the float64 oracle's copy of the same cache."""
import numpy as np
import torch

from oracle import paged_oracle as P

GARBAGE_PAGE = 1 << 29  # table entries behind a sequence's pages: reading one would be seen


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


class PagedState:
    """B sequences of given cached lengths in shuffled pages; rows behind a sequence's end are NaN."""

    def __init__(self, S, kind, Hkv, dh, page, lens, room, seed=0, dev="cuda", spare=2):
        rng = np.random.default_rng(seed)
        self.S, self.kind, self.Hkv, self.dh, self.page = S, kind, Hkv, dh, page
        self.lens_h = [int(x) for x in lens]
        self.room = [int(x) for x in room]  # rows a sequence can grow to
        B = len(self.lens_h)
        need = [-(-r // page) for r in self.room]
        max_pages = max(need + [1]) + 1
        num_pages = sum(need) + spare
        order = list(rng.permutation(num_pages))
        self.table_h = np.full((B, max_pages), GARBAGE_PAGE, dtype=np.int64)
        for b in range(B):
            for i in range(need[b]):
                self.table_h[b, i] = order.pop()
        pools = []
        for which in range(2):
            x = rng.standard_normal((num_pages, Hkv, page, dh)) * np.exp(0.4 * rng.standard_normal((1, Hkv, 1, 1)))
            pools.append(torch.from_numpy(x).to(torch.bfloat16))
        live = torch.zeros(num_pages, page, dtype=torch.bool)
        for b in range(B):
            for t in range(self.lens_h[b]):
                live[int(self.table_h[b, t // page]), t % page] = True
        mask = live[:, None, :, None]
        self.pages, self.scales, self.oracle = [], [], []
        for x in pools:
            x = torch.where(mask, x, torch.zeros_like(x))
            if kind == "bf16":
                self.oracle.append(P.Pages(f64(x)))
                self.pages.append(torch.where(mask, x, torch.full_like(x, float("nan"))).to(dev))
                self.scales.append(None)
            else:
                amax = f64(x.abs().amax(dim=(2, 3)))
                sc = np.vectorize(P.needed_scale)(amax)
                vals = P.round_e4m3(f64(x) / sc[:, :, None, None])
                codes = torch.from_numpy(vals).to(torch.float32).to(torch.float8_e4m3fn)
                codes = torch.where(mask, codes.view(torch.uint8), torch.full_like(codes.view(torch.uint8), 0x7F))
                self.oracle.append(P.Pages(vals * sc[:, :, None, None], sc))
                self.pages.append(codes.view(torch.float8_e4m3fn).to(dev))
                self.scales.append(torch.from_numpy(sc).to(torch.float32).to(dev))
        self.table = torch.from_numpy(self.table_h).to(torch.int32).to(dev)
        self.lens = torch.tensor(self.lens_h, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.cache = S.PagedKV(self.pages[0], self.pages[1], self.table, self.scales[0], self.scales[1])
        self.rng, self.dev, self.B = rng, dev, B

    def rows(self, n, heads, scale=1.0):
        """bf16 rows [sum n][heads][dh] on the device."""
        x = self.rng.standard_normal((sum(n), heads, self.dh)) * scale
        return torch.from_numpy(x).to(torch.bfloat16).to(self.dev)

    def starts(self, n, first=0):
        return torch.tensor(np.concatenate([[first], first + np.cumsum(n)]), dtype=torch.int32, device=self.dev)

    def values(self, which):
        """What the device's pages stand for."""
        x = f64(self.pages[which].to(torch.float32))
        return x if self.kind == "bf16" else x * f64(self.scales[which])[:, :, None, None]


def angles(n_pos, rot, dev="cuda"):
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n_pos)[:, None] * f
    return tuple(torch.from_numpy(x.astype(np.float32)).to(dev) for x in (np.cos(a), np.sin(a)))
