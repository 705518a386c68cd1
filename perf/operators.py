"""Workloads of the serving operators: one step of a batch that shares a prefix.

A batch of requests continues the same long prompt.  The prompt's keys and
values sit once in a paged cache; every request owns further pages for its own
tokens.  One step of such a server is three operators:

* ``tables``: from the requests' lengths, the pages they take or give back,
  their block tables, and the cache slot and the position of every new token;
* ``write``: the new tokens' keys and values into their slots;
* ``attend``: attention of the new tokens over the shared prefix and the
  request's own pages, causal or with a sliding window, with optional sinks.

``run`` computes each either in its plain form (elementary torch operations,
fp32, one rounding at the end) or, with ``own`` set, through the package.
"""
import math

import numpy as np
import torch

own = False

# (query heads, kv heads, head dim) of the packed workloads, and the standard
# deviation of their q / k / v
HEADS = ((4, 2, 64), (32, 8, 64), (32, 8, 128), (64, 8, 128), (16, 1, 256))


def listed():
    return [
        # four chats over a short system prompt: the latency of one step
        dict(name="attend_b4_p1000", op="attend", batch=4, n_q=1, Hq=32, Hkv=8, D=128, prefix=1000,
             own_lo=1, own_hi=200, block=16, window=0, sinks=False, layout="thd"),
        # an ordinary server batch over a document of some pages, with sinks
        dict(name="attend_b64_p8191_sink", op="attend", batch=64, n_q=1, Hq=64, Hkv=8, D=128, prefix=8191,
             own_lo=64, own_hi=4096, block=16, window=0, sinks=True, layout="thd"),
        # the largest batch over a long document
        dict(name="attend_b256_p32768", op="attend", batch=256, n_q=1, Hq=64, Hkv=8, D=128, prefix=32768,
             own_lo=64, own_hi=4096, block=32, window=0, sinks=False, layout="thd"),
        # four drafted tokens per request are checked in one step; sliding window, heads outermost in a page
        dict(name="attend_b32_q4_w4096", op="attend", batch=32, n_q=4, Hq=32, Hkv=8, D=128, prefix=16001,
             own_lo=16, own_hi=2048, block=64, window=4096, sinks=False, layout="htd"),
        # multi-query attention with the widest heads, sliding window and sinks
        dict(name="attend_b48_mqa_d256_w8192", op="attend", batch=48, n_q=1, Hq=16, Hkv=1, D=256, prefix=65536,
             own_lo=64, own_hi=8192, block=128, window=8192, sinks=True, layout="thd"),
        # no shared prefix: plain decoding from the paged cache, narrow heads
        dict(name="attend_b128_d64_alone", op="attend", batch=128, n_q=1, Hq=32, Hkv=8, D=64, prefix=0,
             own_lo=16, own_hi=8192, block=16, window=0, sinks=False, layout="thd"),
        # one decoding step: one token for each request
        dict(name="tables_b256_step", op="tables", batch=256, block=16, max_blocks=512, kind="step", rows=256),
        # prompts of a whole pack are admitted at once
        dict(name="tables_b64_admit64k", op="tables", batch=64, block=16, max_blocks=512, kind="admit", rows=65536),
        # a large pool: some requests decode, some end, some begin
        dict(name="tables_b4096_mixed", op="tables", batch=4096, block=32, max_blocks=256, kind="mixed", rows=131072),
        # the new tokens of one decoding step, from a fused projection's output
        dict(name="write_t64_fused", op="write", rows=64, Hq=64, Hkv=8, D=128, block=16, fused=True, layout="thd"),
        # a prompt of the 8k pack, odd row count, heads outermost in a page
        dict(name="write_t8191_d64", op="write", rows=8191, Hq=32, Hkv=8, D=64, block=64, fused=False, layout="htd"),
        # the prompts of the 64k pack
        dict(name="write_t65536_fused", op="write", rows=65536, Hq=64, Hkv=8, D=128, block=16, fused=True,
             layout="thd"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "tables", "write"))
    if op == "attend":
        top = max(_attend_cost(c) for c in listed() if c["op"] == "attend")
        while True:
            Hq, Hkv, D = rng.choice(HEADS)
            own_hi = _log_int(rng, 32, 8192)
            case = dict(op=op, batch=_log_int(rng, 1, 256), n_q=rng.choice((1, 1, 1, 2, 3, 4, 8)), Hq=Hq, Hkv=Hkv,
                        D=D, prefix=rng.choice((0, _log_int(rng, 16, 65536), _log_int(rng, 16, 65536))),
                        own_lo=max(1, own_hi // rng.choice((1, 4, 64))), own_hi=own_hi,
                        block=rng.choice((16, 32, 64, 128)),
                        window=rng.choice((0, 0, _log_int(rng, 64, 8192))), sinks=rng.random() < 0.5,
                        layout=rng.choice(("thd", "thd", "htd")))
            case["own_lo"] = max(case["own_lo"], case["n_q"])
            if _attend_cost(case) <= top:
                return case
    if op == "tables":
        kind = rng.choice(("step", "admit", "mixed"))
        batch = _log_int(rng, 1, 4096)
        block = rng.choice((16, 32, 64, 128))
        rows = batch if kind == "step" else max(batch, _log_int(rng, 256, 131072))
        return dict(op=op, batch=batch, block=block, max_blocks=8192 // block, kind=kind, rows=rows)
    Hq, Hkv, D = rng.choice(HEADS)
    rows = _log_int(rng, 1, 65536)
    while rows * Hkv * D > 65536 * 8 * 128:
        rows //= 2
    return dict(op=op, rows=rows, Hq=Hq, Hkv=Hkv, D=D, block=rng.choice((16, 32, 64, 128)),
                fused=rng.random() < 0.5, layout=rng.choice(("thd", "htd")))


# ------------------------------------------------------------------- inputs

def _own_lens(case):
    """Log-uniform lengths of the requests' own tokens, the same for every seed."""
    rng = np.random.default_rng([case["batch"], case["own_lo"], case["own_hi"], case["prefix"]])
    u = rng.uniform(math.log(case["own_lo"]), math.log(case["own_hi"]) + 1e-9, size=case["batch"])
    return np.clip(np.rint(np.exp(u)), case["own_lo"], case["own_hi"]).astype(np.int64)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    x.normal_(0.0, std, generator=g)
    return x


def _cache(g, n_blocks, block, Hkv, D, layout, std=1.0):
    """A paged cache seen as [blocks, tokens of a block, kv heads, head dim];
    layout "htd" keeps the heads outermost inside a page."""
    if layout == "htd":
        return _randn(g, (n_blocks, Hkv, block, D), std).transpose(1, 2)
    return _randn(g, (n_blocks, block, Hkv, D), std)


def _prepare_attend(case, seed):
    g = _gen(seed)
    B, n_q, block, P = case["batch"], case["n_q"], case["block"], case["prefix"]
    std = 0.5 if case["D"] == 256 else 1.0
    lens = _own_lens(case)
    n_own = -(-lens // block)
    n_pre = -(-P // block)
    n_blocks = int(n_own.sum() + n_pre) + 3
    perm = torch.randperm(n_blocks, generator=torch.Generator().manual_seed(seed)).to(torch.int32).numpy()
    tables = np.full((B, int(n_own.max())), -1, dtype=np.int32)
    at = n_pre
    for b in range(B):
        tables[b, : n_own[b]] = perm[at : at + n_own[b]]
        at += int(n_own[b])
    state = dict(op="attend", n_q=n_q, window=case["window"], scale=case["D"] ** -0.5)
    state["q"] = _randn(g, (B * n_q, case["Hq"], case["D"]), std)
    state["k_cache"] = _cache(g, n_blocks, block, case["Hkv"], case["D"], case["layout"], std)
    state["v_cache"] = _cache(g, n_blocks, block, case["Hkv"], case["D"], case["layout"], std)
    state["block_tables"] = torch.from_numpy(tables).cuda()
    state["kv_lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    state["prefix_table"] = torch.from_numpy(perm[:n_pre].copy()).cuda() if P else None
    state["prefix_len"] = torch.tensor([P], dtype=torch.int32, device="cuda") if P else None
    state["sinks"] = torch.randn((case["Hq"],), generator=g, device="cuda") if case["sinks"] else None
    if own:
        import sliding_window_gqa_cu_b200 as swa

        # a server allocates the scratch once, for its largest batch
        n = swa.thd_attn_shared_prefix_workspace_bytes(B, n_q, case["Hq"], case["Hkv"], case["D"])
        state["workspace"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
    return state


def _table_lens(case, seed):
    """Cached tokens (-1: vacant entry) and new tokens (-1: the request ends).
    Every seed has the same requests in another order, so the pool's size stays."""
    rng = np.random.default_rng([case["batch"], case["rows"], case["block"]])
    B, cap = case["batch"], case["max_blocks"] * case["block"]
    old = np.rint(np.exp(rng.uniform(math.log(16), math.log(cap - 1), size=B))).astype(np.int64)
    new = np.ones(B, dtype=np.int64)
    if case["kind"] == "admit":
        old[:] = 0
    if case["kind"] == "mixed":
        part = rng.uniform(size=B)
        new[part < 0.1] = -1                                     # ended
        old[(part >= 0.1) & (part < 0.3)] = 0                    # begins
        old[(part >= 0.3) & (part < 0.35)] = -1                  # vacant
    starts = np.flatnonzero(old == 0)
    room = case["rows"] - B
    if len(starts) and room > 0:
        w = rng.uniform(0.2, 1.0, size=len(starts))
        new[starts] += np.minimum((w / w.sum() * room).astype(np.int64), cap - 1)
    order = np.random.default_rng(seed).permutation(B)
    return old[order], new[order]


def _prepare_tables(case, seed):
    old, new = _table_lens(case, seed)
    B, block, M = case["batch"], case["block"], case["max_blocks"]
    held = np.where(old > 0, -(-old // block), 0)
    want = np.where((old >= 0) & (new > 0), -(-(old + new) // block), held) - held
    n_blocks = int(held.sum() + want.sum()) + 64
    perm = np.random.default_rng([seed, 1]).permutation(n_blocks).astype(np.int32)
    tables = np.full((B, M), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        tables[b, : held[b]] = perm[at : at + held[b]]
        at += int(held[b])
    free = np.full((n_blocks,), -1, dtype=np.int32)
    free[: n_blocks - at] = perm[at:]
    dev = "cuda"
    return dict(op="tables", block=block, rows=case["rows"],
                seq_lens=torch.from_numpy(old.astype(np.int32)).to(dev),
                new_lens=torch.from_numpy(new.astype(np.int32)).to(dev),
                block_tables=torch.from_numpy(tables).to(dev), free_blocks=torch.from_numpy(free).to(dev),
                free_count=torch.tensor([n_blocks - at], dtype=torch.int32, device=dev),
                first_position=torch.tensor([1000], dtype=torch.int32, device=dev))


def _prepare_write(case, seed):
    g = _gen(seed)
    T, Hq, Hkv, D, block = (case[n] for n in ("rows", "Hq", "Hkv", "D", "block"))
    n_blocks = -(-T // block) + 8
    if case["fused"]:
        qkv = _randn(g, (T, Hq + 2 * Hkv, D))
        k, v = qkv[:, Hq : Hq + Hkv], qkv[:, Hq + Hkv :]
    else:
        k, v = _randn(g, (T, Hkv, D)), _randn(g, (T, Hkv, D))
    # each request's tokens fill pages of its own in order; the rows behind
    # the last token of a padded batch carry -1
    perm = torch.randperm(n_blocks, generator=torch.Generator().manual_seed(seed))
    t = torch.arange(T)
    slots = perm[t // block] * block + t % block
    slots[T - T // 16 :] = -1
    return dict(op="write", k=k, v=v, slots=slots.to(torch.int32).cuda(),
                k_cache=_cache(g, n_blocks, block, Hkv, D, case["layout"]),
                v_cache=_cache(g, n_blocks, block, Hkv, D, case["layout"]))


def prepare(case, seed):
    return {"attend": _prepare_attend, "tables": _prepare_tables, "write": _prepare_write}[case["op"]](case, seed)


# --------------------------------------------------------------- plain forms

def _part(q, k, v, pos, key_pos, n_keys, window, scale):
    """One softmax part: q [..., rows, D], k / v [..., keys, D], positions of
    the rows and keys, the number of keys that exist.  Returns the row
    maximum, the sum and the weighted values (not divided)."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    see = (key_pos[..., None, :] <= pos[..., :, None]) & (
        torch.arange(k.shape[-2], device=k.device) < n_keys[..., None])[..., None, :]
    if window > 0:
        see = see & (key_pos[..., None, :] > pos[..., :, None] - window)
    s = s.masked_fill(~see, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return m, p.sum(dim=-1, keepdim=True), torch.matmul(p, v)


def _merge(a, b):
    if a is None:
        return b
    m = torch.maximum(a[0], b[0])
    z = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    wa, wb = torch.exp(a[0] - z), torch.exp(b[0] - z)
    return m, a[1] * wa + b[1] * wb, a[2] * wa + b[2] * wb


def _plain_attend(s):
    q, kc, vc, tables, lens = s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["kv_lens"].long()
    B, n_q, W, scale = tables.shape[0], s["n_q"], s["window"], s["scale"]
    (_, block, Hkv, D), Hq = kc.shape, q.shape[1]
    G = Hq // Hkv
    dev = q.device
    P = s["prefix_len"].long()[0] if s["prefix_len"] is not None else torch.zeros((), dtype=torch.long, device=dev)
    pos = P + lens[:, None] - n_q + torch.arange(n_q, device=dev)             # [B, n_q]
    pos = pos[:, :, None].expand(B, n_q, G).reshape(B, n_q * G)
    # [Hkv, B, n_q * G, D]: the rows that share a kv head
    qf = q.float().view(B, n_q, Hkv, G, D).permute(2, 0, 1, 3, 4).reshape(Hkv, B, n_q * G, D)
    m = torch.empty((Hkv, B, n_q * G, 1), device=dev)
    l = torch.empty_like(m)
    acc = torch.empty((Hkv, B, n_q * G, D), device=dev)
    pre = [None] * Hkv
    if s["prefix_table"] is not None:
        pt = s["prefix_table"].long()
        for j0 in range(0, pt.shape[0] * block, 8192):                        # the prefix, once for all rows
            pages = pt[j0 // block : (j0 + 8192) // block]
            n = pages.shape[0] * block
            kf, vf = kc[pages].reshape(n, Hkv, D), vc[pages].reshape(n, Hkv, D)
            key = torch.arange(j0, j0 + n, device=dev)
            for h in range(Hkv):
                part = _part(qf[h].reshape(B * n_q * G, D), kf[:, h].float(), vf[:, h].float(),
                             pos.reshape(-1), key, P - j0, W, scale)
                pre[h] = _merge(pre[h], part)
    keys = tables.shape[1] * block
    step = max(1, min(B, (1 << 27) // (keys * Hkv * D)))
    for b0 in range(0, B, step):                                              # own pages, some requests at a time
        b1 = min(B, b0 + step)
        pages = tables[b0:b1].long().clamp(min=0)
        kf = kc[pages].reshape(b1 - b0, keys, Hkv, D).permute(2, 0, 1, 3).float()
        vf = vc[pages].reshape(b1 - b0, keys, Hkv, D).permute(2, 0, 1, 3).float()
        m[:, b0:b1], l[:, b0:b1], acc[:, b0:b1] = _part(
            qf[:, b0:b1], kf, vf, pos[b0:b1], (P + torch.arange(keys, device=dev)).expand(b1 - b0, keys),
            lens[b0:b1], W, scale)
    own_part = (m, l, acc)
    if pre[0] is not None:
        own_part = _merge(tuple(torch.stack([p[i].view(B, n_q * G, -1) for p in pre]) for i in range(3)), own_part)
    if s["sinks"] is not None:
        sink = s["sinks"].view(Hkv, 1, 1, G).expand(Hkv, B, n_q, G).reshape(Hkv, B, n_q * G, 1)
        own_part = _merge(own_part, (sink, torch.ones_like(sink), torch.zeros_like(own_part[2])))
    m, l, acc = own_part
    out = (acc / l).view(Hkv, B, n_q, G, D).permute(1, 2, 0, 3, 4).reshape(B * n_q, Hq, D)
    lse = (m + torch.log(l)).view(Hkv, B, n_q, G).permute(1, 2, 0, 3).reshape(B * n_q, Hq)
    return [out.to(torch.bfloat16), lse.contiguous()]


def _plain_tables(s):
    seq, new, table, free = s["seq_lens"].long(), s["new_lens"].long(), s["block_tables"], s["free_blocks"]
    block, rows = s["block"], s["rows"]
    B, M = table.shape
    F = free.shape[0]
    dev = seq.device
    live = seq >= 0
    ends = live & (new < 0)
    grow = live & ~ends
    add = torch.where(grow, new, torch.zeros_like(new))
    held = torch.where(live, (seq + block - 1) // block, torch.zeros_like(seq))
    back = torch.where(ends, held.clamp(max=M), torch.zeros_like(seq))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(add, 0)])
    total = torch.where(grow, (seq + add + block - 1) // block, held)
    refused = grow & (add > 0) & ((total > M) | (cu[1:] > rows))
    need = torch.where(grow & ~refused, total - held, torch.zeros_like(seq))
    off = torch.cumsum(need, 0) - need
    n_free = s["free_count"].long()[0]
    top = (n_free + back.sum()).clamp(max=F)
    refused = refused | ((need > 0) & (off + need > top))
    taken = torch.where(refused, torch.zeros_like(off), torch.where(need > 0, off + need, torch.zeros_like(off))).amax()
    j = torch.arange(M, device=dev)
    give = j < back[:, None]                                                  # pages given back, in request order
    to = torch.where(give, n_free + (torch.cumsum(back, 0) - back)[:, None] + j, torch.full_like(j, F)).clamp(max=F)
    wide = torch.cat([free, free[:1]])
    wide[to.reshape(-1)] = table.reshape(-1)
    free.copy_(wide[:F])
    get = (j >= held[:, None]) & (j < total[:, None]) & ~refused[:, None] & (need > 0)[:, None]
    src = (top - 1 - (off[:, None] + j - held[:, None])).clamp(0, F - 1)
    table.copy_(torch.where(get, free[src], table))
    t = torch.arange(rows, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    at = seq[b] + t - cu[b]
    inside = t < cu[B]
    page = table[b, (at // block).clamp(0, M - 1)].long()
    slots = torch.where(inside & ~refused[b], page * block + at % block, torch.full_like(t, -1))
    positions = torch.where(inside, s["first_position"].long() + at, torch.zeros_like(t))
    seq_out = torch.where(ends, torch.full_like(seq, -1), torch.where(refused, seq, seq + add))
    i32 = torch.int32
    return [seq_out.to(i32), (top - taken).to(i32).view(1), cu.to(i32), slots.to(i32), positions.to(i32),
            refused.sum().to(i32).view(1), table, free]


def _plain_write(s):
    slots, block = s["slots"].long(), s["k_cache"].shape[1]
    ok = slots >= 0
    first = torch.argmax(ok.to(torch.int32)).view(1)          # rows without a slot repeat the first one that has
    row = torch.where(ok, torch.arange(slots.shape[0], device=slots.device), first)
    at = slots[row]
    s["k_cache"][at // block, at % block] = s["k"][row]
    s["v_cache"][at // block, at % block] = s["v"][row]
    return [s["k_cache"], s["v_cache"]]


# ------------------------------------------------------------------ the pass

def run(state):
    if not own:
        return {"attend": _plain_attend, "tables": _plain_tables, "write": _plain_write}[state["op"]](state)
    import sliding_window_gqa_cu_b200 as swa

    s = state
    if s["op"] == "attend":
        return list(swa.thd_attn_shared_prefix(
            s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["kv_lens"], s["prefix_table"],
            s["prefix_len"], window=s["window"], scale=s["scale"], sinks=s["sinks"], workspace=s["workspace"]))
    if s["op"] == "tables":
        seq_lens, free_count, cu_new, slots, positions, refused = swa.thd_kv_block_tables(
            s["seq_lens"], s["new_lens"], s["block_tables"], s["free_blocks"], s["free_count"], s["block"],
            s["rows"], first_position=s["first_position"])
        return [seq_lens, free_count, cu_new, slots, positions, refused, s["block_tables"], s["free_blocks"]]
    return list(swa.thd_kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"]))


# ---------------------------------------------------------------------- work

def _seen_pairs(case):
    """(query row, key) pairs the mask leaves, and the keys that some query of
    the batch sees in the prefix and in the requests' own pages."""
    lens, P, W, n_q = _own_lens(case), case["prefix"], case["window"], case["n_q"]
    pos = P + lens[:, None] - n_q + np.arange(n_q)
    lo = np.maximum(0, pos - W + 1) if W else np.zeros_like(pos)
    pairs = np.maximum(pos + 1 - lo, 0).sum()
    first = lo.min(axis=1)
    pre = P - min(P, int(first.min()))
    own_keys = int((lens - np.clip(first - P, 0, lens)).sum())
    return int(pairs), pre, own_keys


def _attend_cost(case):
    pairs, pre, own_keys = _seen_pairs(case)
    return max(4.0 * pairs * case["Hq"] * case["D"] / 1.6e15, 4.0 * (pre + own_keys) * case["Hkv"] * case["D"] / 6.5e12)


def work(case):
    if case["op"] == "attend":
        pairs, pre, own_keys = _seen_pairs(case)
        rows = case["batch"] * case["n_q"] * case["Hq"]
        return {"bytes": 4 * (pre + own_keys) * case["Hkv"] * case["D"] + rows * (4 * case["D"] + 4),
                "flops": 4 * pairs * case["Hq"] * case["D"]}
    if case["op"] == "tables":
        old, new = _table_lens(case, 0)
        block = case["block"]
        held = np.where(old > 0, -(-old // block), 0)
        live = (old >= 0) & (new > 0)
        need = int(np.where(live, -(-(old + new) // block) - held, 0).sum())
        back = int(held[(old >= 0) & (new < 0)].sum())
        # lengths in, lengths and row offsets out, pages moved, one page entry
        # read for each page that holds a new token, slot and position out
        tokens = int(new[live].sum())
        return {"bytes": 16 * case["batch"] + 8 * (need + back) + 4 * (tokens // block) + 8 * case["rows"], "flops": 0}
    T = case["rows"]
    return {"bytes": (T - T // 16) * case["Hkv"] * case["D"] * 8 + 4 * T, "flops": 0}


# --------------------------------------------------- definition, in 64 bits

def _exact_attend(case, seed):
    s = _prepare_attend(case, seed)
    Hq, Hkv, D, n_q, W = case["Hq"], case["Hkv"], case["D"], case["n_q"], case["window"]
    G, P, block = Hq // Hkv, case["prefix"], case["block"]
    lens = s["kv_lens"].tolist()
    tables = s["block_tables"].long()
    out = torch.empty((len(lens) * n_q, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((len(lens) * n_q, Hq), dtype=torch.float64, device="cuda")

    def rows_of(cache, h, pages, first, end):
        return cache[:, :, h][pages[first // block : (end + block - 1) // block]].reshape(-1, D)[
            first % block : first % block + end - first].double()

    for h in range(Hkv):
        heads = slice(h * G, (h + 1) * G)
        if P:
            k0, v0 = (rows_of(s[c], h, s["prefix_table"].long(), 0, P) for c in ("k_cache", "v_cache"))
        for b, n in enumerate(lens):
            k1, v1 = (rows_of(s[c], h, tables[b], 0, n) for c in ("k_cache", "v_cache"))
            for i in range(n_q):
                p = P + n - n_q + i
                lo = max(0, p - W + 1) if W else 0
                kk = ([k0[lo:p + 1]] if P else []) + [k1[max(0, lo - P):p + 1 - P]]
                vv = ([v0[lo:p + 1]] if P else []) + [v1[max(0, lo - P):p + 1 - P]]
                x = s["q"][b * n_q + i, heads].double()
                z = torch.cat([x @ part.T for part in kk], dim=1) * s["scale"]
                if s["sinks"] is not None:
                    z = torch.cat([z, s["sinks"][heads].double()[:, None]], dim=1)
                norm = torch.logsumexp(z, dim=1)
                w = torch.exp(z - norm[:, None])
                at, total = 0, 0
                for part in vv:
                    total = total + w[:, at : at + part.shape[0]] @ part
                    at += part.shape[0]
                out[b * n_q + i, heads] = total
                lse[b * n_q + i, heads] = norm
    return [out, lse]


def _exact_tables(case, seed):
    s = _prepare_tables(case, seed)
    seq, new = s["seq_lens"].tolist(), s["new_lens"].tolist()
    table, free = s["block_tables"].cpu().numpy(), s["free_blocks"].cpu().numpy()
    block, rows, first = case["block"], case["rows"], int(s["first_position"])
    M, stack = case["max_blocks"], free[: int(s["free_count"])].tolist()
    for b, (have, n) in enumerate(zip(seq, new)):
        if have >= 0 and n < 0:
            stack += table[b, : -(-have // block)].tolist()
    free[: len(stack)] = stack
    slots, positions, cu = [], [], [0]
    seq_out, n_refused, taken, top = [], 0, 0, len(stack)
    for b, (have, n) in enumerate(zip(seq, new)):
        grows = have >= 0 and n >= 0
        n_new = n if grows else 0
        cu.append(cu[-1] + n_new)
        if not grows:
            seq_out.append(-1)
            continue
        want = -(-(have + n_new) // block) - -(-have // block)
        fits = -(-(have + n_new) // block) <= M and cu[-1] <= rows and taken + want <= top
        if not fits:     # (the pools of these cases hold every request)
            n_refused += 1
            want = 0
        for j in range(want):
            table[b, -(-have // block) + j] = stack[top - 1 - taken - j]
        taken += want
        at = range(have, have + n_new)
        slots += [int(table[b, x // block]) * block + x % block for x in at] if fits else [-1] * n_new
        positions += [first + x for x in at]
        seq_out.append(have + n_new if fits else have)
    slots += [-1] * (rows - len(slots))
    positions += [0] * (rows - len(positions))
    as_i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return [as_i32(seq_out), as_i32([top - taken]), as_i32(cu), as_i32(slots), as_i32(positions), as_i32([n_refused]),
            torch.from_numpy(table).cuda(), torch.from_numpy(free).cuda()]


def _exact_write(case, seed):
    s = _prepare_write(case, seed)
    slots = s["slots"].cpu().numpy()
    block = case["block"]
    rows = torch.from_numpy(np.flatnonzero(slots >= 0)).cuda()
    to = s["slots"].long()[rows]
    result = []
    for cache, x in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        flat = cache.double().reshape(-1, case["Hkv"], case["D"])
        flat.index_copy_(0, to, x.double()[rows])
        result.append(flat.view(-1, block, case["Hkv"], case["D"]))
    return result


def exact(case, seed):
    return {"attend": _exact_attend, "tables": _exact_tables, "write": _exact_write}[case["op"]](case, seed)
