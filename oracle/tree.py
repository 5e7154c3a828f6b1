"""fp64 CPU oracle of one round of tree speculation: the tree step, the
verification of drafted tokens, and keeping the accepted path.

Sources: "Arsitektur Inferensi LLM ..." (tveniu.com), section 7: drafted tokens
are checked by the target model in one pass and the output keeps the target's
distribution. The page describes a chain; a tree is several chains that share
their beginnings, so that a node sees the cached tokens and its own chain
only. Verification is speculative sampling tried over a node's children one
after the other, written below as it is defined (a residual distribution per
rejection), not in the closed form a fast implementation would use.
"""

from __future__ import annotations

import numpy as np

from .decode import (
    F64,
    _f64,
    append_contiguous,
    append_paged,
    dequantize_e5m2,
    dequantize_u8,
    quantize_e5m2,
    quantize_u8,
    rope_rotate,
    round_bf16,
)


def mask_matrix(words, n: int) -> np.ndarray:
    """[..., n, W] 32-bit words -> [..., n, n] truth values."""
    w = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    return ((w[..., None] >> np.arange(32)) & 1).astype(bool).reshape(w.shape[:-1] + (-1,))[..., :n]


def tree_rotate(x, pos, depth, base: float) -> np.ndarray:
    """x [B, n, H, d] with node i of sequence b rotated by pos[b] + depth[b, i], unrounded."""
    x = _f64(x)
    out = np.empty_like(x)
    for b in range(x.shape[0]):
        for i in range(x.shape[1]):
            out[b, i] = rope_rotate(x[b, i], int(pos[b]) + int(depth[b][i]), base)
    return out


def tree_append(K, V, cache: str, k_new, v_new, pos, depth, nodes, base: float, table=None, page_size: int = 0,
                k_sz=None, v_sz=None):
    """The caches (and a u8 cache's scale / zero rows) with every node's row
    written at pos[b] + i: copies. cache: "bf16" (values), "e5m2", "u8" (codes)."""
    K, V = np.array(K, copy=True), np.array(V, copy=True)
    ksz = None if k_sz is None else np.array(k_sz, copy=True)
    vsz = None if v_sz is None else np.array(v_sz, copy=True)
    k_rot, v_new = tree_rotate(k_new, pos, depth, base), _f64(v_new)
    for b in range(k_rot.shape[0]):
        for i in range(int(nodes[b])):
            p = int(pos[b]) + i
            if cache == "bf16":
                ks, vs = round_bf16(k_rot[b, i]), v_new[b, i]
            elif cache == "e5m2":
                ks, vs = quantize_e5m2(k_rot[b, i]), quantize_e5m2(v_new[b, i])
            else:
                ks, sk, zk = quantize_u8(k_rot[b, i].astype(np.float32))
                vs, sv, zv = quantize_u8(v_new[b, i].astype(np.float32))
            if table is None:
                append_contiguous(K, V, b, p, ks, vs)
                if cache == "u8":
                    append_contiguous(ksz, vsz, b, p, np.stack([sk, zk], -1), np.stack([sv, zv], -1))
            else:
                append_paged(K, V, table[b], page_size, p, ks, vs)
                if cache == "u8":
                    append_paged(ksz, vsz, table[b], page_size, p, np.stack([sk, zk], -1), np.stack([sv, zv], -1))
    return K, V, ksz, vsz


def tree_attention(q, keys, values, pos, depth, nodes, mask, scale: float, window: int = 0):
    """q [B, n, H_q, d]; keys / values [B, H_kv, T, d], the logical caches with
    the nodes at rows pos[b] + i; mask [B, n, n] truth values. Returns dict
    (out [B, n, H_q, d], lse [B, n, H_q], size [B, n, H_q, d] = sum w |v|,
    reach [B, n, H_q] = max over attended keys of scale sum |q k|); rows of
    nodes past nodes[b] are NaN."""
    q, keys, values = _f64(q), _f64(keys), _f64(values)
    B, n, hq, d = q.shape
    G = hq // keys.shape[1]
    out, size = np.full((B, n, hq, d), np.nan), np.full((B, n, hq, d), np.nan)
    lse, reach = np.full((B, n, hq), np.nan), np.full((B, n, hq), np.nan)
    for b in range(B):
        P, N = int(pos[b]), int(nodes[b])
        for i in range(N):
            cached = [t for t in range(P) if not window or t > P + int(depth[b][i]) - window]
            own = [P + t for t in range(N)
                   if mask[b][i][t] and (not window or int(depth[b][t]) > int(depth[b][i]) - window)]
            at = np.array(cached + own, dtype=np.int64)
            for h in range(hq):
                if at.size == 0:
                    out[b, i, h], size[b, i, h], lse[b, i, h], reach[b, i, h] = 0.0, 0.0, -np.inf, 0.0
                    continue
                k, v = keys[b, h // G, at], values[b, h // G, at]
                s = scale * (k @ q[b, i, h])
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                w = w / total
                out[b, i, h], size[b, i, h] = w @ v, w @ np.abs(v)
                lse[b, i, h] = m + np.log(total)
                reach[b, i, h] = scale * (np.abs(k) @ np.abs(q[b, i, h])).max()
    return {"out": out, "lse": lse, "size": size, "reach": reach}


def logical(cache: str, x, sz=None, table=None, page_size: int = 0, tokens: int = 0) -> np.ndarray:
    """A cache's values as [B, H_kv, T, d]; pages outside the pool read as zeros."""
    if cache == "e5m2":
        v = dequantize_e5m2(x)
    elif cache == "u8":
        v = dequantize_u8(x, sz[..., 0], sz[..., 1])
    else:
        v = _f64(x)
    if table is None:
        return v
    n, h, ps, d = v.shape
    out = np.zeros((len(table), h, tokens, d), F64)
    for b, row in enumerate(table):
        for t in range(tokens):
            if t // ps < len(row) and 0 <= int(row[t // ps]) < n:
                out[b, :, t] = v[int(row[t // ps]), :, t % ps]
    return out


def verify_tree(target, draft, tokens, parents, nodes, u_accept, u_next):
    """target (and draft, or None) [B, n, vocab] probabilities. The walk as it
    is defined: the target's distribution is tried against each child, and
    after a rejection replaced by the normalised positive part of itself minus
    the draft's; without a draft's distribution a rejected token's probability
    is struck out and the rest measured against what is left of 1. (The first
    is for children drawn from draft independently of each other, the second for
    any.) Returns (num_kept [B], path [B, n], next_token [B], margin): margin is the smallest distance of a comparison from a tie, as a
    probability (a sum formed in another order may decide those closer than
    its own rounding otherwise)."""
    target = _f64(target)
    draft = None if draft is None else _f64(draft)
    B, n, vocab = target.shape
    kept, path, nxt = np.zeros(B, np.int64), np.full((B, n), -1, np.int64), np.full(B, -1, np.int64)
    margin = np.inf
    for b in range(B):
        if int(nodes[b]) == 0:
            continue
        cur, way = 0, [0]
        while True:
            dist, moved = target[b, cur].copy(), False  # the distribution the next token is to follow
            left = 1.0  # (no draft) what is left of 1
            for c in range(1, int(nodes[b])):
                x = int(tokens[b][c])
                if int(parents[b][c]) != cur or not 0 <= x < vocab or not 0 <= int(parents[b][c]) < c:
                    continue
                q = draft[b, cur] if draft is not None else None
                ask, have = float(u_accept[b][c]) * (left if q is None else q[x]), dist[x]
                margin = min(margin, abs(ask - have))
                if ask < have:
                    cur, moved = c, True
                    way.append(c)
                    break
                if q is None:
                    left -= dist[x]
                    dist[x] = 0.0
                    continue
                rest = np.maximum(dist - q, 0.0)
                dist = rest / rest.sum() if rest.sum() > 0 else np.zeros(vocab)
            if moved:
                continue
            if dist.sum() > 0:
                cum = np.cumsum(dist)
                goal = float(u_next[b]) * cum[-1]
                nxt[b] = int(np.searchsorted(cum, goal, side="right"))
                margin = min(margin, float(np.abs(cum - goal).min()))
            else:
                nxt[b] = int(target[b, cur].argmax())
            break
        kept[b] = len(way)
        path[b, :len(way)] = way
    return kept, path, nxt, margin


def keep_path(cache, pos, path, kept, table=None, page_size: int = 0):
    """A copy of one cache [B, H, T, ...] (or pool [pages, H, page_size, ...])
    with row pos + path[i] at row pos + i: every row read before any is written."""
    out = np.array(cache, copy=True)
    src = np.array(cache, copy=True)
    for b in range(len(pos)):
        for i in range(int(kept[b])):
            a, c = int(pos[b]) + int(path[b][i]), int(pos[b]) + i
            if table is None:
                out[b, :, c] = src[b, :, a]
            else:
                out[int(table[b][c // page_size]), :, c % page_size] = src[int(table[b][a // page_size]), :, a % page_size]
    return out
