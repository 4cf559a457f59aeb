"""Batches and error bounds of the history cache, for its GPU tests."""

import numpy as np
import torch

import recommender_model_attention_gb300 as gd
from oracle import cache as orc
from oracle import ref
from prefix_util import ACT_ERR, check_f32, check_lse, offsets

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dtype))).cuda()


class Batch:
    """Samples with `new` rows on `hist` events each, on random pages of a cache
    whose memory held NaNs in every byte before."""

    def __init__(self, new, hist, H=2, Hkv=2, d=128, store="bf16", dtype=None, page=16, seed=0, gain=1.5,
                 parents=None, extra_width=0):
        self.new, self.hist = np.asarray(new, dtype=np.int64), np.asarray(hist, dtype=np.int64)
        self.H, self.Hkv, self.d, self.store, self.page = H, Hkv, d, store, page
        self.few = len(self.new) == 0 or int(self.new.sum()) * (H // Hkv) // len(self.new) <= 32
        self.dt = DT[dtype or ("f32" if store == "f32" else "bf16")]
        rng = np.random.Generator(np.random.PCG64(seed))
        total = self.new + self.hist
        pages = -(-total // page)
        n = int(pages.sum()) + 2
        order = rng.permutation(n).astype(np.int32)
        self.table_host = np.full((len(total), int(pages.max(initial=0)) + extra_width), -1, dtype=np.int32)
        at = 0
        for b, p in enumerate(pages):
            self.table_host[b, :p] = order[at:at + p]
            at += int(p)
        self.cache = gd.KVCache(n, Hkv, d, page=page, store=store)
        for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            t.fill_(255)
        self.table = dev(self.table_host)
        self.off_host, self.off, self.starts = offsets(self.new), dev(offsets(self.new)), dev(self.hist)
        g = torch.Generator().manual_seed(seed)

        def rows(n, heads, s):
            x = torch.randn((n, heads, d), generator=g)
            return (x * (s * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6))).to(self.dt)
        T = int(total.sum())
        self.k_all, self.v_all = rows(T, Hkv, 1.0), rows(T, Hkv, 1.0)
        self.q = rows(int(self.new.sum()), H, gain).cuda()
        self.parents_host = None if parents is None else np.asarray(parents, dtype=np.int32)
        self.parents = None if parents is None else dev(self.parents_host)

    def split(self, x):
        """Per sample, its events' rows."""
        return np.split(x, np.cumsum(self.new + self.hist)[:-1])

    def fill(self):
        """History first, then the new rows, as a server does."""
        total = self.new + self.hist
        first = np.cumsum(total) - total
        at = lambda n, s: np.concatenate([f + a + np.arange(c) for f, a, c in zip(first, s, n)]).astype(np.int64)  # noqa: E731
        h, w = at(self.hist, 0 * self.hist), at(self.new, self.hist)
        for idx, off, st in ((h, dev(offsets(self.hist)), None), (w, self.off, self.starts)):
            gd.gdpa_cache_write(self.cache, self.k_all[idx].cuda(), self.v_all[idx].cuda(), self.table, off, st)
        return self

    def want(self, alpha, act, **kw):
        k, v = (self.split(orc.held(ref.to_f64(x), self.store)) for x in (self.k_all, self.v_all))
        return orc.attend(self.off_host, self.hist, ref.to_f64(self.q), k, v, alpha, act,
                          parents=self.parents_host, **kw)

    def run(self, act="softmax", alpha=None, **kw):
        """(O, lse or None) of the library."""
        args = (self.cache, self.q, self.table, self.off, self.starts)
        if act == "softmax":
            return gd.gdpa_cache_softmax_fwd(*args, alpha=alpha, parents=self.parents, **kw)
        return gd.gdpa_cache_fwd(*args, act=act, alpha=alpha, parents=self.parents, **kw), None

    def check(self, act="softmax", alpha=None, **kw):
        o, lse = self.run(act, alpha, **kw)
        self.cache.check()
        want, wlse, size = self.want(self.d ** -0.5 if alpha is None else alpha, act, **kw)
        check_o(o, want, size, act, self)
        if lse is not None:
            check_lse(lse, wlse)
        return o, lse


def check_o(got, want, size, act, b):
    """float32 rows, or bf16 ones of a head dim that the CUDA cores take: 1e-5 of
    the largest value and the output's rounding.  bf16 on the tensor cores: half
    a step (2^-8) of the value for its own rounding; of every term, half a step of
    its weight's type (bf16 2^-8; f16 2^-11 for 8-bit caches and at most 32 rows a
    sample and key head on average) and 2^-12 for the float32 sums behind it; the
    activation's error; 2% for products of these."""
    if b.dt == torch.float32:
        return check_f32(got, want, "o")
    err = np.abs(ref.to_f64(got) - want)
    terms, one, x = size
    if b.d in (64, 128):
        c1, cx = ACT_ERR.get(act, ((0.0, 0.0),))[0]
        weight = 2.0 ** -11 if b.store == "e4m3" and b.few else 2.0 ** -8
        bound = 1.02 * (2.0 ** -8 * np.abs(want) + (weight + 2.0 ** -12) * terms + c1 * one + cx * x) + 1e-30
    else:
        bound = 2.0 ** -8 * np.abs(want) + 1.02e-5 * np.max(np.abs(want), initial=0.0) + 1e-30
    assert np.all(err <= bound), "worst error %.3g of its bound" % np.max(err / bound)


__all__ = ["Batch", "DT", "check_f32", "check_lse", "check_o", "dev", "gd", "offsets", "orc", "ref"]
