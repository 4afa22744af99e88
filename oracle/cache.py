"""Oracle of the operators around a paged key/value cache, in float64 (test
infrastructure): the weights that cached keys receive, the cut of a cache to a
budget by them, and the attention of a tree of drafted tokens.

Only ``tests/`` and ``__graft_entry__.smoke()`` may call this module; the
product path never does.

The operators stand beside selected-page decode ("BF1: A Causal Dyadic
Sparse-Attention Retrofit for Efficient Long-Context Transformers", section 5)
and read its cache: page p holds the B consecutive slots of one logical block
for every key/value head, ``page_table[b][j]`` names the page of block j.

* The weight of a key is the sum, over the query rows that may read it, of the
  probability they give it, exp(s - lse).
* A cut keeps, for every key/value head by itself, the `recent` newest tokens
  and then those of largest weight (the lower slot at equal weights, a NaN as
  -inf).  Kept tokens below the new length stay; the i-th free slot below it
  takes the i-th kept token from behind.
* Drafted token i follows its parent (an earlier drafted token, or the cache
  for -1) at depth e, position t = length + e.  It reads the cached tokens and
  the tokens of its own path, itself included, that lie in the key blocks
  which block t // B of the layout keeps: what one decode step at position t
  would read, were the path in the cache.
"""
from __future__ import annotations

import numpy as np


def prompt_weights(q, k, lse, sets, B: int, scale: float):
    """[kv_heads, n]: column sums of exp(scale q k^T - lse) over allowed pairs."""
    heads, n, _ = q.shape
    kv_heads = k.shape[0]
    g = heads // kv_heads
    out = np.zeros((kv_heads, n))
    for f in range(heads):
        rows = sets[f % len(sets)]
        for i, kept in enumerate(rows):
            t = np.arange(i * B, min(n, (i + 1) * B))
            for j in kept:
                u = np.arange(j * B, min(n, (j + 1) * B))
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.exp(scale * (q[f, t] @ k[f // g, u].T) - lse[f, t][:, None])
                p = np.where(u[None, :] <= t[:, None], p, 0.0)
                p = np.where(np.isneginf(lse[f, t])[:, None], 0.0, p)
                out[f // g, u] += p.sum(0)
    return out


def step_weights(q, k_cache, page_table, positions, lse, sets, B: int, scale: float, n: int):
    """[batch * H_kv, n]: what one decode step adds to the weights, given its lse."""
    heads, _ = q.shape
    batch = len(positions)
    H, hkv = heads // batch, k_cache.shape[1]
    out = np.zeros((batch * hkv, n))
    for b in range(batch):
        t = int(positions[b])
        for h in range(H):
            f, kv = b * H + h, h // (H // hkv)
            if np.isneginf(lse[f]):
                continue
            for j in sorted(sets[f % len(sets)][t // B]):
                for x in range(B):
                    u = j * B + x
                    if u <= t:
                        s = scale * float(k_cache[page_table[b][j], kv, x] @ q[f])
                        out[b * hkv + kv, u] += np.exp(s - lse[f])
    return out


def evict(k_cache, v_cache, page_table, lengths, weights, tokens, n: int, budget: int, recent: int):
    """(k_cache, v_cache, weights, tokens, lengths) after the cut; weights and
    tokens are [batch * H_kv, n], tokens None for slot = token."""
    kc, vc = k_cache.copy(), v_cache.copy()
    hkv, B = kc.shape[1], kc.shape[2]
    w_out = np.zeros((len(weights), n), dtype=weights.dtype)
    t_out = np.zeros((len(weights), n), dtype=np.int64)
    for r in range(len(weights)):
        b, length = r // hkv, int(lengths[r // hkv])
        tok = [int(x) for x in (tokens[r][:length] if tokens is not None else range(length))]
        newest = max(tok) if length else -1
        kept = min(length, budget)
        w = [-np.inf if np.isnan(x) else float(x) for x in weights[r][:length]]
        order = sorted(range(length), key=lambda s: (tok[s] <= newest - recent, -w[s] if tok[s] <= newest - recent else 0.0, s))
        stay = set(order[:kept])
        behind = iter(sorted(s for s in stay if s >= kept))
        for s in range(kept):
            src = s if s in stay else next(behind)
            w_out[r, s], t_out[r, s] = weights[r][src], tok[src]
            if src != s:
                to, at = page_table[b][s // B], page_table[b][src // B]
                kc[to, r % hkv, s % B] = k_cache[at, r % hkv, src % B]
                vc[to, r % hkv, s % B] = v_cache[at, r % hkv, src % B]
        for s in range(kept, n):
            t_out[r, s] = newest + 1 + s - kept
    return kc, vc, w_out, t_out, np.minimum(np.asarray(lengths), budget)


def tree(q, k_tree, v_tree, k_cache, v_cache, page_table, lengths, parents, sets, B: int, scale: float):
    """(o [batch*H, T, d], lse [batch*H, T]); unused rows (parent -2) get o = 0, lse = nan."""
    heads, T, d = q.shape
    batch = len(lengths)
    H, hkv = heads // batch, k_cache.shape[1]
    g = H // hkv
    o = np.zeros((heads, T, d))
    lse = np.full((heads, T), np.nan)
    for b in range(batch):
        length = int(lengths[b])
        for i in range(T):
            if parents[b][i] == -2:
                continue
            path = [i]
            while parents[b][path[0]] != -1:
                path.insert(0, int(parents[b][path[0]]))
            blk = (length + len(path) - 1) // B
            for h in range(H):
                f, kv = b * H + h, h // g
                kept = sets[f % len(sets)][blk]
                keys, vals = [np.zeros((0, d))], [np.zeros((0, d))]
                for j in sorted(kept):
                    m = min(B, length - j * B)
                    if m > 0:
                        keys.append(k_cache[page_table[b][j], kv, :m])
                        vals.append(v_cache[page_table[b][j], kv, :m])
                for e, x in enumerate(path):
                    if (length + e) // B in kept:
                        keys.append(k_tree[b * hkv + kv, x][None])
                        vals.append(v_tree[b * hkv + kv, x][None])
                kf, vf = np.concatenate(keys), np.concatenate(vals)
                if not len(kf):
                    lse[f, i] = -np.inf
                    continue
                s = scale * (kf @ q[f, i])
                m = s.max()
                p = np.exp(s - m)
                lse[f, i] = m + np.log(p.sum())
                o[f, i] = (p / p.sum()) @ vf
    return o, lse
