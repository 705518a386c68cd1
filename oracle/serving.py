"""CPU oracle of the serving step: block tables and slot maps, the paged cache
write, and attention over a shared prefix and each request's own pages.

TEST INFRASTRUCTURE ONLY (see the package docstring).  fp64 numpy and plain
Python, one request after the other.

The attention is the packed forward's ("muse_spark.magi_cp" / "flint.magi"
pages: causal or sliding window counting the query's own token, repeat_kv head
mapping, sinks in the denominator only) over the sequence [prefix; own] of
every request, whose queries are its last n_q tokens.
"""
from __future__ import annotations

import numpy as np

from .sparse_mla import _f64


def _keys(cache, table, length, num_blocks, block):
    """Rows [0, length) of a page list: ([n, Hkv, D], their key positions);
    entries outside the cache contribute none."""
    pos = np.arange(length, dtype=np.int64)
    page = np.asarray(table, dtype=np.int64)[pos // block]
    pos, page = pos[(page >= 0) & (page < num_blocks)], page[(page >= 0) & (page < num_blocks)]
    return cache[page, pos % block], pos


def shared_prefix_attention(q, k_cache, v_cache, block_tables, kv_lens, prefix_table=None, prefix_len=0,
                            window: int = 0, scale: float = 1.0, sinks=None):
    """fp64 (out [B * n_q, Hq, D], lse [B * n_q, Hq], spread, reach): ``spread``
    is sum_j p_j |v_j| (what a relative error of the weights is multiplied by)
    and ``reach`` the largest scale * sum_d |q_d k_jd| of a row (what a relative
    error of the products is multiplied by).  Rows of vacant requests
    (kv_lens < 0) are NaN."""
    q, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    tables = np.asarray(block_tables.cpu() if hasattr(block_tables, "cpu") else block_tables)
    lens = np.asarray(kv_lens.cpu() if hasattr(kv_lens, "cpu") else kv_lens)
    T, Hq, D = q.shape
    nb, bs, Hkv, _ = kc.shape
    B = tables.shape[0]
    n_q, G = T // B, Hq // Hkv
    out, spread = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, reach = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    P, pt = 0, np.zeros(0, dtype=np.int32)
    if prefix_table is not None:
        pt = np.asarray(prefix_table.cpu() if hasattr(prefix_table, "cpu") else prefix_table)
        P = min(max(int(prefix_len), 0), pt.size * bs)
    pk, ppos = _keys(kc, pt, P, nb, bs)
    pv, _ = _keys(vc, pt, P, nb, bs)
    snk = _f64(sinks) if sinks is not None else None
    for b in range(B):
        n = int(lens[b])
        if n < 0:
            continue
        n = min(n, tables.shape[1] * bs)
        ok, opos = _keys(kc, tables[b], n, nb, bs)
        ov, _ = _keys(vc, tables[b], n, nb, bs)
        keys, vals = np.concatenate([pk, ok]), np.concatenate([pv, ov])
        at = np.concatenate([ppos, opos + P])
        for i in range(n_q):
            p, r = P + n - n_q + i, b * n_q + i
            see = at <= p
            if window > 0:
                see &= at > p - window
            for g in range(Hkv):
                kk, vv = keys[see, g], vals[see, g]
                qq = q[r, g * G:(g + 1) * G]
                s = scale * (qq @ kk.T)                            # [G, keys]
                far = scale * (np.abs(qq) @ np.abs(kk).T)
                for x in range(G):
                    h = g * G + x
                    z = s[x] if snk is None else np.append(s[x], snk[h])
                    top = z.max() if z.size else -np.inf
                    if top == -np.inf:
                        out[r, h], spread[r, h], lse[r, h] = 0.0, 0.0, -np.inf
                        continue
                    e = np.exp(s[x] - top)
                    Z = np.exp(z - top).sum()
                    out[r, h], spread[r, h] = e @ vv / Z, e @ np.abs(vv) / Z
                    lse[r, h] = top + np.log(Z)
                    reach[r, h] = far[x].max(initial=0.0)
    return out, lse, spread, reach


def block_tables(seq_lens, new_lens, table, free_blocks, free_count, block, n_rows, first_position=0):
    """One request after the other.  Returns a dict of the step's outputs; the
    arguments stay as they are."""
    table, free = np.array(table, dtype=np.int64), np.array(free_blocks, dtype=np.int64)
    M, cap = table.shape[1], free.size
    stack = list(free[:min(max(int(free_count), 0), cap)])
    for n, m, row in zip(seq_lens, new_lens, table):
        if n >= 0 and m < 0:
            for page in row[:min(-(-int(n) // block), M)]:
                if len(stack) < cap:
                    stack.append(page)
    free[:len(stack)] = stack
    top, wanted, popped = len(stack), 0, 0
    seq_out, cu, slots, positions, refused = [], [0], [], [], 0
    for b, (n, m) in enumerate(zip(map(int, seq_lens), map(int, new_lens))):
        if n < 0 or m < 0:
            seq_out.append(-1)
            cu.append(cu[-1])
            continue
        cu.append(cu[-1] + m)
        held, total = -(-n // block), -(-(n + m) // block)
        no = m > 0 and (total > M or cu[-1] > n_rows)
        if not no and m > 0:
            need = total - held
            no = need > 0 and wanted + need > top
            if not no:
                for j in range(need):
                    table[b, held + j] = stack[top - 1 - wanted - j]
                popped += need
            wanted += need
        refused += no
        seq_out.append(n if no else n + m)
        for x in range(n, n + min(m, n_rows - len(slots))):     # (rows behind the call's are not given)
            slots.append(-1 if no else int(table[b, x // block]) * block + x % block)
            positions.append(first_position + x)
    pad = max(0, n_rows - len(slots))
    return dict(seq_lens=np.array(seq_out), free_count=top - popped, cu=np.array(cu), table=table, free=free,
                slots=np.array((slots + [-1] * pad)[:n_rows], dtype=np.int64),
                positions=np.array((positions + [0] * pad)[:n_rows], dtype=np.int64), refused=refused)


def kv_write(rows, slots, cache):
    """The cache [blocks, block, Hkv, D] (numpy copy) with row r at slots[r]."""
    cache = np.array(cache)
    flat = cache.reshape((-1,) + cache.shape[2:])
    for r, s in enumerate(np.asarray(slots)):
        if 0 <= s < flat.shape[0]:
            flat[s] = rows[r]
    return cache
