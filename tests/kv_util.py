"""A paged int8 cache on the host and on the device, for the cache tests."""
import numpy as np
import torch

from oracle import decode
from packed_bit_gemv_tern_amd import tern
from gpu_util import DEV, to_dev


class Paged:
    """A cache of random codes and scales, page tables of distinct pages."""

    def __init__(self, seqs, columns, heads, D, P, seed=0, spare=2, scales=None):
        rng = np.random.default_rng([seqs, columns, heads, D, P, seed])
        pages = seqs * columns + spare
        k = rng.integers(-127, 128, (pages, heads, P, D)).astype(np.int8)
        v = rng.integers(-127, 128, (pages, heads, D, P)).astype(np.int8)
        ks, vs = (rng.uniform(0.005, 0.03, (2, pages, heads)) if scales is None else scales(rng, (2, pages, heads)))
        self.host = decode.Cache(k, v, ks.astype(np.float32), vs.astype(np.float32))
        self.table = rng.permutation(pages)[: seqs * columns].reshape(seqs, columns).astype(np.int32)
        self.heads, self.D, self.P, self.rng = heads, D, P, rng

    def upload(self):
        h = self.host
        self.k, self.v, self.ks, self.vs = (to_dev(a) for a in (h.k, h.v, h.k_scale, h.v_scale))
        self.cache = tern.make_kv_cache(self.k, self.v, self.ks, self.vs, h.pages, self.heads, self.D, self.P)
        return self

    def batch(self, new, length, rows=None, max_new=None, max_len=0, start=None):
        """The device batch of the given new and total tokens, its offsets,
        and its rows (also kept here)."""
        start = np.concatenate([[0], np.cumsum(new)]) if start is None else np.asarray(start)
        self.start, self.length = start.astype(np.int32), np.asarray(length, np.int32)
        self.rows = int(start[-1]) if rows is None else rows
        self.max_new = max(new) if max_new is None else max_new
        self.keep = to_dev(self.table), to_dev(self.start), to_dev(self.length)
        return tern.make_kv_batch(self.keep[0], self.table.shape[1], self.keep[1], self.keep[2], len(self.length),
                                  self.rows, self.max_new, max_len)

    def check(self):
        """The whole device cache against the host's."""
        torch.cuda.synchronize()
        h = self.host
        for name, dev, host in (("k_scale", self.ks, h.k_scale), ("v_scale", self.vs, h.v_scale), ("k", self.k, h.k),
                                ("v", self.v, h.v)):
            got = dev.cpu().numpy()
            bad = np.argwhere(got != host) if got.dtype == np.int8 else np.argwhere(
                got.view(np.uint32) != host.view(np.uint32))
            assert not len(bad), "%s differs at %s (%d places)" % (name, bad[0].tolist(), len(bad))
