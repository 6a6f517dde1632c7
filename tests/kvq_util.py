"""A small 8-bit KV cache on the GPU and its oracle twin, for the kvq tests."""
import numpy as np
import torch

from oracle import kvq as ok

HD, PAGE, SUB = 128, 128, 16


def bf16(x):
    """fp64 array rounded to bf16, as (tensor on the GPU, fp64 array)."""
    t = torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


class Cache:
    """n_seqs sequences of up to `pages` pages in scattered pool pages; every
    byte of the pool starts as garbage (NaN codes among it)."""

    def __init__(self, heads, n_seqs, pages, seed=0, spare=2, mapped=None):
        from block_diffusion_speculative_injection_gb300 import capi
        self.capi = capi
        rng = np.random.default_rng(seed)
        self.heads, self.n_seqs, self.pages = heads, n_seqs, pages
        n_pages = n_seqs * pages + spare
        ids = rng.permutation(n_pages)[:n_seqs * pages].reshape(n_seqs, pages).astype(np.int32)
        if mapped is not None:
            for q, m in enumerate(mapped):
                ids[q, m:] = -1
        self.table = ids
        self.t = {}
        for x in "kv":
            junk = rng.integers(0, 256, (n_pages, heads, PAGE, HD), dtype=np.uint8)
            junk[rng.random(junk.shape) < 0.02] = 0x7F
            self.t[x + "8"] = torch.from_numpy(junk).cuda()
            self.t[x + "e"] = torch.from_numpy(
                rng.integers(-40, 41, (n_pages, heads, PAGE // SUB), dtype=np.int8)).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.h = capi.KvqCache(self.t["k8"], self.t["v8"], self.t["ke"], self.t["ve"],
                               torch.from_numpy(ids).cuda(), self.status)
        slots = pages * PAGE
        self.val = {x: np.zeros((n_seqs, slots, heads, HD)) for x in "kv"}
        self.exp = {x: np.zeros((n_seqs, slots // SUB, heads), dtype=int) for x in "kv"}

    def append(self, starts, rows_k, rows_v, counts=None, seqs=None, pad=0, oracle=True):
        """rows_k, rows_v: fp64 [batch][rows][heads][128]."""
        B, R = rows_k.shape[:2]
        both = np.concatenate([rows_k, rows_v, np.zeros((B, R, pad, HD))], axis=2)
        t, exact = bf16(both)
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
        self.capi.dflash_kvq_append(self.h, B, R, i32(seqs), i32(starts), i32(counts),
                                    t[:, :, :self.heads], t[:, :, self.heads:2 * self.heads])
        if oracle:
            for b in range(B):
                q = b if seqs is None else seqs[b]
                c = R if counts is None else counts[b]
                for x, at in (("k", 0), ("v", self.heads)):
                    ok.append(self.val[x][q], self.exp[x][q], starts[b],
                              exact[b, :c, at:at + self.heads])
        torch.cuda.synchronize()

    def codes(self, x):
        """[n_seqs][slots][heads][128] codes and [n_seqs][slots/16][heads]
        exponents as they lie in the pool (unmapped: page 0's)."""
        pg = torch.from_numpy(np.maximum(self.table, 0)).long().cuda()
        c = self.t[x + "8"][pg].permute(0, 1, 3, 2, 4).reshape(self.n_seqs, -1, self.heads, HD)
        e = self.t[x + "e"][pg].permute(0, 1, 3, 2).reshape(self.n_seqs, -1, self.heads)
        return c.cpu().numpy(), e.cpu().numpy().astype(int)

    def values(self, x):
        c, e = self.codes(x)
        return ok.E4M3[c] * 2.0 ** np.repeat(e, SUB, axis=1)[..., None]


def ancestors(parents, words):
    """Ancestor sets and their bit form [n][words] int64 (node 0 the root)."""
    sets, bits = [], np.zeros((len(parents), words), dtype=np.uint64)
    for i, p in enumerate(parents):
        s = {i} | (sets[p] if p >= 0 else set())
        sets.append(s)
        for m in s:
            bits[i, m >> 6] |= np.uint64(1) << np.uint64(m & 63)
    return sets, bits.view(np.int64)
