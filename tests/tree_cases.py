"""Inputs of the tree-speculation tests: random trees, masks, caches with
whatever garbage a cache may hold in rows that are not the sequence's."""

import numpy as np
import torch


def random_parents(rng, n, branch=3):
    par, kids = [-1], [0] * n
    for i in range(1, n):
        a = int(rng.integers(0, i))
        while kids[a] >= branch:
            a += 1
        par.append(a)
        kids[a] += 1
    return par


def mask_words(bits: np.ndarray) -> np.ndarray:
    """[..., n, n] truth values -> [..., n, ceil(n / 32)] int32 words."""
    n = bits.shape[-1]
    w = (n + 31) // 32
    pad = np.zeros(bits.shape[:-1] + (32 * w,), np.uint64)
    pad[..., :n] = bits
    words = (pad.reshape(bits.shape[:-1] + (w, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def deal_pages(rng, need, spare):
    total = sum(need) + spare
    perm = rng.permutation(total)
    table = np.full((len(need), max(max(need), 1) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, total


class TreeCase:
    """One call's inputs on the CPU. pos, nodes: lists; mask: "tree", "random"
    (any relation, empty rows among them) or "none" (every row empty)."""

    def __init__(self, hq, hkv, d, pos, nodes, n, cache="bf16", page=0, window=0, mask="tree", seed=0, garbage=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.B, self.hq, self.hkv, self.d, self.n = len(pos), hq, hkv, d, n
        self.pos, self.nodes, self.cache, self.page, self.window = list(pos), list(nodes), cache, page, window
        B = self.B
        self.parents = np.array([random_parents(rng, n) for _ in pos], np.int32)
        bits = np.zeros((B, n, n), bool)
        self.depth = np.zeros((B, n), np.int32)
        for b in range(B):
            for i in range(n):
                a = self.parents[b, i]
                if a >= 0:
                    bits[b, i] = bits[b, a]
                    self.depth[b, i] = self.depth[b, a] + 1
                bits[b, i, i] = True
        if mask == "random":
            bits = rng.random((B, n, n)) < 0.4
            bits[:, 0] = False
        elif mask == "none":
            bits[:] = False
        self.bits = bits
        self.words = mask_words(bits)
        tokens = max(p + k for p, k in zip(pos, nodes))
        self.max_len = max(tokens, 1)
        self.table = None
        if page:
            self.table, total = deal_pages(rng, [-(-(p + k) // page) for p, k in zip(pos, nodes)], 2)
            shape = (total, hkv, page, d)
        else:
            shape = (B, hkv, (self.max_len + 3) // 2 * 2, d)
        self.ksz = self.vsz = None

        def normal(s):
            return torch.randn(s, generator=g).to(torch.bfloat16)

        if cache == "u8":
            self.k, self.v = (torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8) for _ in "kv")
            self.ksz, self.vsz = (torch.stack([(5 + 2 * torch.rand(shape[:-1], generator=g)) / 255,
                                               torch.randint(100, 156, shape[:-1], generator=g).float()], -1).contiguous()
                                  for _ in "kv")
        else:
            self.k, self.v = normal(shape), normal(shape)
            if cache == "e5m2":
                self.k, self.v = self.k.to(torch.float8_e5m2), self.v.to(torch.float8_e5m2)
        self.q_new, self.k_new, self.v_new = normal((B, n, hq, d)), normal((B, n, hkv, d)), normal((B, n, hkv, d))
        if garbage:
            self._garbage()

    def _garbage(self):
        """NaN (u8: NaN and infinite scales) in every row that no sequence owns."""
        used = torch.zeros(self.k.shape[:-1], dtype=torch.bool)
        for b in range(self.B):
            for t in range(self.pos[b] + self.nodes[b]):
                if self.page:
                    used[int(self.table[b, t // self.page]), :, t % self.page] = True
                else:
                    used[b, :, t] = True
        for x, sz in ((self.k, self.ksz), (self.v, self.vsz)):
            if sz is not None:
                sz[~used] = float("nan")
            elif x.dtype == torch.float8_e5m2:
                x.view(torch.uint8)[~used] = 0x7F
            else:
                x[~used] = float("nan")

    def gpu(self, m, device="cuda"):
        """(layout, tensors) on the GPU; the tensors are copies."""
        import types

        t = types.SimpleNamespace()
        for name in ("k", "v", "ksz", "vsz", "q_new", "k_new", "v_new"):
            x = getattr(self, name)
            setattr(t, name, None if x is None else x.clone().to(device))
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=device)  # noqa: E731
        t.pos, t.depth, t.num, t.mask = i32(self.pos), i32(self.depth), i32(self.nodes), i32(self.words)
        t.table = None if self.table is None else i32(self.table)
        if self.page:
            lay = m.layout_paged(t.k, t.v, t.table, self.hq, self.window, t.ksz, t.vsz)
        else:
            lay = m.layout_contiguous(t.k, t.v, self.hq, self.window, t.ksz, t.vsz)
        return lay, t


def raw(x):
    """A cache tensor as numpy: float64 values, or codes."""
    x = x.detach().cpu()
    if x.dtype == torch.float8_e5m2:
        return x.view(torch.uint8).numpy()
    return x.numpy() if x.dtype == torch.uint8 else x.to(torch.float64).numpy()
