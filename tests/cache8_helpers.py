"""Inputs shared by the tests of the 8-bit cache and of attention over a shared prefix."""

import numpy as np
import torch

from oracle import serving as S
from tests.serving_helpers import f64, random_cache

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def quantised(x):
    """Rows on the host as (float8_e4m3fn codes, uint8 bytes), by the oracle."""
    codes, b = S.quantise(f64(x))
    return torch.from_numpy(codes).view(E4M3), torch.from_numpy(b)


def values(codes, b, dtype=F32):
    """What they stand for; exact in either type. Cells that hold anything at all give NaN or a number."""
    return torch.from_numpy(S.stand_for(codes.view(torch.uint8).numpy(), b.numpy())).to(dtype)


class Cache8:
    """A cache in 8 bits on the host, and the same in fp32."""

    def __init__(self, k, v, seed=0):
        """k, v: a cache as random_cache makes it; cells that hold no token are NaN there and get
        any codes and any bytes here."""
        g = np.random.default_rng(seed)
        self.parts = []
        for x in (k, v):
            empty = torch.isnan(x.float()).all(-1)
            codes, b = quantised(torch.where(empty[..., None], 0.0, x.float()))
            junk = torch.from_numpy(g.integers(0, 256, tuple(codes.shape), dtype=np.uint8))
            junk[..., 1::7] = 127
            codes = torch.where(empty[..., None], junk, codes.view(torch.uint8)).view(E4M3)
            b = torch.where(empty, torch.from_numpy(g.integers(0, 256, tuple(b.shape), dtype=np.uint8)), b)
            self.parts.append((codes, b))
        self.refresh()

    def refresh(self):
        (self.kc, self.kb), (self.vc, self.vb) = self.parts
        self.k, self.v = values(self.kc, self.kb), values(self.vc, self.vb)

    def on_gpu(self, B, dtype):
        return B.KVCache8(self.kc.cuda(), self.vc.cuda(), self.kb.cuda(), self.vb.cuda(), dtype)


def random_cache8(lens, h_kv, dh, page, seed, spread=0.7, **kw):
    """(Cache8, table): as random_cache, the rows of different sizes."""
    k, v, table = random_cache(lens, h_kv, dh, page, F32, seed, **kw)
    g = torch.Generator().manual_seed(seed + 1000)
    k, v = (x * torch.exp(spread * torch.randn(x.shape[:-1] + (1,), generator=g)) for x in (k, v))
    return Cache8(k, v, seed), table
