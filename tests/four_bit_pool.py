"""A 4-bit paged cache for the GPU tests, with its values in 64 bits, beside the pools of the other types."""
import numpy as np
import torch

import dense_reference as ref
import four_bit_reference as four
import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import DEV, E4M3, Pool, i32

E2M1 = torch.uint8


class Pool4(Pool):
    """Sequences of `lens` cells with random codes, scales (some of them zero) and exponents that differ from row to
    row.  Every row that belongs to no cell has NaN scales.  The values in 64 bits in self.k[s], self.v[s]; units:
    the cells' powers of two."""

    def __init__(self, lens, H, d, page, seed, spare=2, pad=0, extra_cols=1, exps=(116, 124), width=None):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.d, self.page = lens, H, d, page
        counts = [-(-n // page) for n in lens]
        n_pages = sum(counts) + spare
        order = rng.permutation(n_pages)
        table = np.full((len(lens), width or max(counts + [0]) + extra_cols), -7, np.int32)
        at = 0
        for i, c in enumerate(counts):
            table[i, :c] = order[at:at + c]
            at += c
        self.table = i32(table)
        rows = n_pages * page
        self.np = {}
        for x in "KV":
            codes = rng.integers(0, 256, (rows, H * d // 2 + pad)).astype(np.uint8)
            scale = rng.integers(0x28, 0x50, (n_pages, H, page, d // 16)).astype(np.uint8)  # 2^-2 .. 2^3
            scale[rng.random(scale.shape) < 0.05] = 0
            exp = rng.integers(exps[0], exps[1], (rows, H)).astype(np.uint8)
            live = np.zeros(rows, bool)
            for i, n in enumerate(lens):
                live[self.np_rows(table[i], np.arange(n))] = True
            page_of, off = np.arange(rows) // page, np.arange(rows) % page
            scale[page_of[~live], :, off[~live]] = 0x7f
            self.np[x] = codes, scale, exp
        t = {x: [torch.from_numpy(y).to(DEV) for y in self.np[x]] for x in "KV"}
        self.K, self.V = (t[x][0][:, :H * d // 2].unflatten(1, (H, d // 2)) for x in "KV")
        self.Ke, self.Ve = t["K"][2], t["V"][2]
        self.Ks, self.Vs = (t[x][1].view(E4M3) for x in "KV")
        self.cache = qsa.PagedCache(self.K, self.V, page, K_exp=self.Ke, V_exp=self.Ve, K_scale=self.Ks, V_scale=self.Vs)
        self.k, self.v, self.units = [], [], []
        for i, n in enumerate(lens):
            k, v = self.values(i, np.arange(n))
            self.k.append(k)
            self.v.append(v)
            self.units.append(2.0 ** (self.np["V"][2][self.np_rows(table[i], np.arange(n))].astype(float) - 127))
        self.kv_len = i32(lens)

    def np_rows(self, table_row, pos):
        return np.asarray(table_row)[pos // self.page].astype(np.int64) * self.page + pos % self.page

    def values(self, i, pos):
        """Stored values of cells as the GPU has them now, 64 bits."""
        r = self.np_rows(self.table[i].cpu().numpy(), np.asarray(pos))
        out = []
        for codes, scale, exp in ((self.K, self.Ks, self.Ke), (self.V, self.Vs, self.Ve)):
            c = four.unpack(codes.cpu().numpy()[r])
            s = scale.view(torch.uint8).cpu().numpy()[r // self.page, :, r % self.page]
            out.append(four.values(c, s, exp.cpu().numpy()[r]))
        return out


def any_pool(lens, H, d, page, dtype, seed, **kw):
    """A pool of float32, bfloat16, float8_e4m3fn, or (uint8) of 4-bit rows."""
    return Pool4(lens, H, d, page, seed, **kw) if dtype == E2M1 else Pool(lens, H, d, page, dtype, seed, **kw)


def kind_of(dtype):
    """What the bound on an attention's error goes by: rows of codes have the term of small fp16 weights."""
    return E4M3 if dtype == E2M1 else dtype
