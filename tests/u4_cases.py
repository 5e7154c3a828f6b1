"""Inputs of the 4-bit-cache tests: caches with whatever garbage a cache may
hold in rows that are not the sequence's, and the error a result may have."""

import numpy as np
import torch

import oracle

NAN_PAIR = float("nan")


def deal_pages(rng, need, spare=3):
    total = sum(need) + spare
    perm = rng.permutation(total)
    table = np.full((len(need), max(max(need), 1) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, total


def random_rows(g, shape, d, spread=1.0):
    """Codes, and pairs as they come from rows of about `spread`: (packed uint8 [*shape, d / 2], bf16 [*shape, 2])."""
    codes = torch.randint(0, 256, (*shape, d // 2), generator=g, dtype=torch.uint8)
    scale = spread * (0.25 + 0.2 * torch.rand(shape, generator=g))
    low = -scale * (6.5 + 2 * torch.rand(shape, generator=g))
    return codes, torch.stack([scale, low], -1).to(torch.bfloat16)


class U4Case:
    """A 4-bit cache on the CPU: K, V codes and pairs in cache layout, `values(b)` the logical rows in 64 bits."""

    def __init__(self, hq, hkv, d, lens, n_new=1, page=0, window=0, seed=0, garbage=True, capacity=None, spread=1.0):
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.B, self.hq, self.hkv, self.d, self.n, self.page, self.window = len(lens), hq, hkv, d, n_new, page, window
        self.lens = list(lens)
        most = max(max(lens), 1)
        self.table = None
        if page:
            table, pages = deal_pages(rng, [-(-max(x, 1) // page) for x in lens])
            if window:  # pages before the window are released
                for b, x in enumerate(lens):
                    table[b, : max(0, x - n_new + 1 - window) // page] = -1
            self.table = torch.from_numpy(table)
            shape = (pages, hkv, page)
        else:
            shape = (self.B, hkv, capacity or -(-most // 4) * 4)
        self.k, self.ksm = random_rows(g, shape, d, spread)
        self.v, self.vsm = random_rows(g, shape, d, spread)
        if garbage:
            keep = torch.zeros(shape, dtype=torch.bool)
            for b, x in enumerate(lens):
                lo = max(0, x - n_new + 1 - window) if window else 0
                for t in range(lo, x):
                    keep[self.slot(b, t)] = True
            for x in (self.ksm, self.vsm):
                x[~keep] = torch.tensor([float("nan"), float("inf")], dtype=torch.bfloat16)
        self.q = torch.randn(self.B, n_new, hq, d, generator=g)

    def slot(self, b, t):
        """Index of row t of sequence b, over all kv heads."""
        if self.table is None:
            return (b, slice(None), t)
        return (int(self.table[b, t // self.page]), slice(None), t % self.page)

    def values(self, b, upto=None):
        """K, V [Hkv, L, d] in 64 bits; rows whose page has been released read as 0 (no query sees them)."""
        n = self.lens[b] if upto is None else upto
        out = []
        for codes, sm in ((self.k, self.ksm), (self.v, self.vsm)):
            x = np.zeros((self.hkv, n, self.d))
            for t in range(n):
                if self.table is not None and int(self.table[b, t // self.page]) < 0:
                    continue
                at = self.slot(b, t)
                p = sm[at].double().numpy()
                x[:, t] = oracle.dequantize_u4(oracle.unpack_u4(codes[at].numpy()), p[..., 0], p[..., 1])
            out.append(np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0))
        return out

    def layout(self, m, dev="cuda"):
        move = lambda x: None if x is None else x.to(dev)  # noqa: E731
        self.dev = dict(k=move(self.k), v=move(self.v), ksm=move(self.ksm), vsm=move(self.vsm), table=move(self.table))
        t = self.dev
        if self.page:
            return m.layout_paged(t["k"], t["v"], t["table"], self.hq, self.window, t["ksm"], t["vsm"], cache_dtype=m.MQA_U4)
        return m.layout_contiguous(t["k"], t["v"], self.hq, self.window, t["ksm"], t["vsm"], cache_dtype=m.MQA_U4)


def attention_reference(case, b, scale, q=None):
    """(out, lse, tolerance of out, tolerance of lse) of sequence b, [n, Hq, d] and [n, Hq].

    q is rounded to fp16, an odd value by half a step, 2^-11 of itself, an even one less 1/16 of its odd neighbour by half
    a step of that: a score is off by at most D = |scale| 2^-11 sum |q| (|k| + |its even neighbour| / 16) <= |scale| 2^-11
    sum (|q| + |the pair's other| / 16) |k| (tiny values more, by 2^-25 of a row's largest), a weight by a factor within exp(+-2 D) of the
    others', the output by (exp(2 D) - 1) max |v - out| <= (exp(2 D) - 1) range(v); p s to 11 bits: 2^-11 of sum p s c <=
    range of a row. Products and sums in fp32, some 2^-24 each over cancelling terms of up to 16 times the values: 2^-18
    of (1 + |score|) in a score and of the values in the output."""
    K, V = case.values(b)
    q = case.q[b].double().numpy() if q is None else np.asarray(q, np.float64)
    first = case.lens[b] - case.n
    out, lse = oracle.attention_values(q, K, V, first, scale, case.window)
    g = case.hq // case.hkv
    n = case.n
    tol_o, tol_l = np.empty_like(out), np.empty_like(lse)
    for i in range(n):
        end = first + i + 1
        begin = max(0, end - case.window) if case.window else 0
        for h in range(case.hq):
            k, v = K[h // g, begin:end], V[h // g, begin:end]
            mag = np.abs(q[i, h])
            mag = mag + mag.reshape(-1, 2)[:, ::-1].reshape(-1) / 16 + mag.max() * 2.0 ** -14
            score = abs(scale) * (np.abs(k) @ mag).max()
            D = score * 2.0 ** -11 + (1 + score) * 2.0 ** -18
            spread = v.max() - v.min() + 1e-30
            tol_o[i, h] = np.expm1(2 * D) * spread + spread * (2.0 ** -11 + 2.0 ** -17) + np.abs(v).max() * 2.0 ** -18
            tol_l[i, h] = D + 2.0 ** -18
    return out, lse, tol_o, tol_l


def rounding(out, dtype):
    """The half step of the output's own rounding."""
    return np.abs(out) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)
