"""The serving step as a server runs it: steps without requests, steps replayed
from a captured graph, block tables of every size class."""
import os
import re
import textwrap

import numpy as np
import pytest
import torch

from oracle import prologue as OP
from oracle import serving as OS
import sliding_window_gqa_cu_b200 as swa
from sliding_window_gqa_cu_b200 import build, workloads
from test_serving_gpu import compare

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    swa.load_library()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


TABLE_OUTPUTS = ("seq_lens", "free_count", "cu", "slots", "positions", "refused")


def check_outputs(got, want):
    for name, x in zip(TABLE_OUTPUTS, got):
        assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(want[name]).reshape(-1)), name


# ------------------------------------------------------- a step of no requests

@pytest.mark.parametrize("count,n_rows", [(5, 0), (5, 7), (0, 3), (-4, 3), (99, 4)])
@pytest.mark.parametrize("how", ["new", "given", "in place"])
def test_tables_of_no_requests(count, n_rows, how):
    # an idle step of a server: the pool stays as it is and padded rows have no slot
    free = i32([3, 1, 4, 0, 2, 6])
    n = i32([count])
    seq, table = i32([]), torch.empty((0, 4), dtype=torch.int32, device=DEV)
    want = OS.block_tables([], [], np.zeros((0, 4)), free.tolist(), count, 16, n_rows, 100)
    kw = {}
    if how != "new":
        kw = dict(slots=torch.full((n_rows,), 9, dtype=torch.int32, device=DEV), cu_new=i32([7]), refused=i32([7]),
                  positions=torch.full((n_rows,), 9, dtype=torch.int32, device=DEV))
        kw["free_count_out"] = n if how == "in place" else i32([77])
    # what the allocator hands out next is not zero
    dirt = [torch.full((k,), 0x01010101, dtype=torch.int32, device=DEV) for k in (1, 2, 8, 16, 32, 64)]
    del dirt
    got = swa.thd_kv_block_tables(seq, i32([]), table, free, n, 16, n_rows, first_position=i32([100]), **kw)
    check_outputs(got, want)
    assert free.tolist() == [3, 1, 4, 0, 2, 6]
    if how == "in place":
        assert got[1] is n


def test_tables_of_no_requests_on_a_stream_and_captured():
    side = torch.cuda.Stream()
    free, n, seq = i32([3, 1, 4]), i32([2]), i32([])
    table = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    want = OS.block_tables([], [], np.zeros((0, 4)), [3, 1, 4], 2, 16, 5)
    torch.cuda.synchronize()
    got = swa.thd_kv_block_tables(seq, seq, table, free, n, 16, 5, stream=side)
    side.synchronize()
    check_outputs(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = swa.thd_kv_block_tables(seq, seq, table, free, n, 16, 5)
    for x in got:
        x.fill_(55)
    g.replay()
    torch.cuda.synchronize()
    check_outputs(got, want)


def test_idle_step_then_tokens():
    # the count that an idle step returns serves the next step
    free = i32([5, 6, 7, 8])
    _, count, _, slots, _, _ = swa.thd_kv_block_tables(i32([]), i32([]), torch.empty((0, 2), dtype=torch.int32, device=DEV),
                                                       free, i32([4]), 4, 3)
    assert slots.tolist() == [-1, -1, -1]
    table = i32([[-1, -1]])
    lens, count, _, slots, _, refused = swa.thd_kv_block_tables(i32([0]), i32([5]), table, free, count, 4, 6)
    assert refused.item() == 0 and count.item() == 2 and lens.tolist() == [5] and table.tolist() == [[8, 7]]
    assert slots.tolist() == [32, 33, 34, 35, 28, -1]


# -------------------------------------------------- a captured step, replayed

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def documented_step():
    """The code of the step that users are shown."""
    text = open(README).read()
    block = re.search(r"## A serving step\n(.*?)\n## ", text, flags=re.S).group(1)
    return textwrap.dedent("\n".join(line for line in block.split("\n") if line.startswith("    ")))


@pytest.mark.parametrize("window,with_sinks", [(0, False), (50, True)])
def test_the_documented_step_replays_from_a_graph(window, with_sinks):
    """The documented step is captured once; every replay takes the step after the
    one before: new pages, slots and positions, nothing of the step before written
    over, and the attention over all tokens so far, against the oracle's own state."""
    B, block, M, Hq, Hkv, D, P = 6, 16, 6, 8, 2, 64, 37
    rng = np.random.default_rng(3)
    n_rows, pool, pages = B + 2, 40, -(-P // block)
    perm = rng.permutation(pool).astype(np.int64)
    # the oracle's state; requests of 0, 15, 16, 31 and 33 tokens and a vacant entry
    seq, table = np.array([0, 15, 16, -1, 31, 33]), np.full((B, M), -1, dtype=np.int64)
    at = pages
    for b in range(B):
        held = -(-max(seq[b], 0) // block)
        table[b, :held] = perm[at:at + held]
        at += held
    free, count = np.full(pool, -1, dtype=np.int64), pool - at
    free[:count] = perm[at:]
    cache = [workloads.random_bf16(rng, (pool, block, Hkv, D)) for _ in range(2)]
    sinks = torch.from_numpy(rng.standard_normal(Hq).astype(np.float32)) if with_sinks else None
    rows = lambda h: workloads.random_bf16(rng, (n_rows, h, D))

    q, k, v = (torch.zeros((n_rows, h, D), dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    ns = dict(lens=i32(seq), new_lens=i32([1] * B), block_tables=i32(table), free_blocks=i32(free), n_free=i32([count]),
              block_size=block, n_rows=n_rows, prefix_len=i32([P]), q=q, k=k, v=v, k_cache=cache[0].to(DEV),
              v_cache=cache[1].to(DEV), q_last=torch.zeros((B, Hq, D), dtype=torch.bfloat16, device=DEV),
              prefix_table=i32(perm[:pages]), window=window, sinks=sinks.to(DEV) if with_sinks else None,
              workspace=torch.empty((swa.thd_attn_shared_prefix_workspace_bytes(B, 1, Hq, Hkv, D),), dtype=torch.uint8,
                                    device=DEV))
    state = {n: ns[n] for n in ("lens", "n_free", "block_tables", "free_blocks", "k_cache", "v_cache")}
    before = {n: t.clone() for n, t in state.items()}
    code = compile(documented_step(), "documented step", "exec")
    exec(code, dict(ns))                                   # (a first, eager call; its state is put back)
    for n, t in state.items():
        t.copy_(before[n])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        exec(code, ns)
    for step in range(36):
        new = np.ones(B, dtype=np.int64)
        if step == 5:
            new[1] = -1                                    # a request ends,
        if step == 9:
            seq[1] = 0                                     # and another takes its entry
            state["lens"][1] = 0
        if step == 20:
            new[2] = 0                                     # a request pauses
        qh, kh, vh = rows(Hq), rows(Hkv), rows(Hkv)
        for t, x in ((q, qh), (k, kh), (v, vh)):
            t.copy_(x)
        ns["q_last"].copy_(qh[:B])
        ns["new_lens"].copy_(torch.from_numpy(new))
        g.replay()
        torch.cuda.synchronize()
        want = OS.block_tables(seq, new, table, free, count, block, n_rows, P)
        check_outputs((state["lens"], state["n_free"], ns["cu"], ns["slots"], ns["positions"], ns["refused"]), want)
        seq, count, table, free = want["seq_lens"], want["free_count"], want["table"], want["free"]
        assert want["refused"] == 0
        assert np.array_equal(state["block_tables"].cpu().numpy(), table) and \
            np.array_equal(state["free_blocks"].cpu().numpy(), free)
        # the rotated rows (rounded to bf16 once; angles below 2^7 in fp32 are off by at
        # most 2^-17, values are at most sqrt(D) = 8), and every row where it belongs
        kd, kr = k.cpu(), OP.qk_norm_rope(kh, None, positions=want["positions"])
        assert (np.abs(kd.double().numpy() - kr) <= 2.0 ** -8 * np.abs(kr) + 2.0 ** -13).all()
        for i, (x, dev) in enumerate(((kd, state["k_cache"]), (vh, state["v_cache"]))):
            for r, slot in enumerate(want["slots"]):
                if slot >= 0:
                    cache[i][slot // block, slot % block] = x[r]
            assert torch.equal(dev.cpu(), cache[i])
        ref = OS.shared_prefix_attention(ns["q_last"].cpu(), *cache, table, seq, perm[:pages], P, window,
                                         np.float32(D ** -0.5).item(), sinks)
        compare(ns["out"], ns["lse"], ref, D, f"step {step}")
    assert swa.thd_attn_shared_prefix_get_error() == 0


@pytest.mark.parametrize("B", [40, 300, 3001])
def test_tables_in_place_replay_from_a_graph(B):
    # one CTA, a cluster of CTAs
    rng = np.random.default_rng(B)
    block, M, n_rows = 4, 8, B + 5
    pool = B * M
    seq, table = np.zeros(B, dtype=np.int64), np.full((B, M), -1, dtype=np.int64)
    free, count = rng.permutation(pool).astype(np.int64), pool
    lens, new_d, tab, fr, n = i32(seq), i32(np.ones(B)), i32(table), i32(free), i32([count])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = swa.thd_kv_block_tables(lens, new_d, tab, fr, n, block, n_rows, seq_lens_out=lens, free_count_out=n)
    for step in range(12):
        new = rng.integers(0, 2, size=B)
        new[rng.uniform(size=B) < 0.05] = -1
        new_d.copy_(torch.from_numpy(new))
        seq = np.where((seq < 0) & (rng.uniform(size=B) < 0.5), 0, seq)     # entries are taken again
        lens.copy_(torch.from_numpy(seq))
        g.replay()
        want = OS.block_tables(seq, new, table, free, count, block, n_rows)
        check_outputs(got, want)
        seq, count, table, free = want["seq_lens"], want["free_count"], want["table"], want["free"]
        assert np.array_equal(tab.cpu().numpy(), table) and np.array_equal(fr.cpu().numpy(), free)


# ------------------------------------------------ positions close to 2^31

@pytest.mark.parametrize("rows", [8, 9])                  # the own pages' kernel takes the prefix; the prefix kernel does
def test_prefix_of_nearly_two_to_the_31_keys(rows):
    """A prefix table as long as the sizes allow, whose entries go through three
    pages: keys and values are zero, so every weight is the same and the output
    zero whatever the order of the sums; behind the last key there is NaN."""
    block, D, n = 16, 64, 5
    entries = 2 ** 27 - 2
    P = entries * block - 5
    assert (entries + 1) * block < 2 ** 31 and P + n < 2 ** 31
    kc, vc = (torch.zeros((5, block, 1, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for x in (kc, vc):
        x[3, block - 5:] = float("nan")                   # the prefix's last page
        x[4, n:] = float("nan")                           # the request's own
    pt = torch.arange(entries, dtype=torch.int32, device=DEV).remainder_(3)
    pt[-1] = 3
    q = torch.ones((1, rows, D), dtype=torch.bfloat16, device=DEV)
    out, lse = swa.thd_attn_shared_prefix(q, kc, vc, i32([[4]]), i32([n]), pt, torch.tensor([P], dtype=torch.int32, device=DEV))
    assert swa.thd_attn_shared_prefix_get_error() == 0
    assert (out == 0).all()
    want = np.log(P + n)
    assert np.abs(lse.cpu().numpy() - want).max() <= 2.0 ** -20 * (1 + want)


# -------------------------- tables of every number of requests a thread takes

def random_tables(B, block, M, seed):
    rng = np.random.default_rng([seed, B])
    seq, new = rng.integers(-1, M * block + 1, size=B), rng.integers(-1, 2 * block, size=B)
    new[rng.uniform(size=B) < 0.2] = 0
    held = np.where(seq > 0, -(-seq // block), 0)
    pool = int(held.sum()) + B // 2                       # (pages run out)
    perm = rng.permutation(pool).astype(np.int64)
    table, at = np.full((B, M), -1), 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(pool, -1)
    free[:pool - at] = perm[at:]
    rows = int(np.where((seq >= 0) & (new > 0), new, 0).sum()) + 3
    return seq, new, table, free, pool - at, rows


@pytest.mark.parametrize("B", [1024, 1025, 2047, 2048, 2049, 3001, 4095, 4096, 4097, 8191, 8192])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_of_many_requests(B, in_place):
    # one, two, four and eight requests a thread, the last thread's run cut or not
    block, M = 8, 4
    seq, new, table, free, count, rows = random_tables(B, block, M, 9)
    want = OS.block_tables(seq, new, table, free, count, block, rows, 11)
    assert 0 < want["refused"] < B
    s, t, f, n = i32(seq), i32(table), i32(free), i32([count])
    kw = dict(seq_lens_out=s, free_count_out=n) if in_place else {}
    got = swa.thd_kv_block_tables(s, i32(new), t, f, n, block, rows, first_position=i32([11]), **kw)
    check_outputs(got, want)
    assert np.array_equal(t.cpu().numpy(), want["table"]) and np.array_equal(f.cpu().numpy(), want["free"])


# ------------------------------------------------ the first tokens of an answer

def call_us(B, own, P=16384, Hq=64, Hkv=8, D=128, block=16):
    """Median time of a call for B requests of `own` tokens each after P."""
    per, pages = -(-own // block), P // block
    kc, vc = (torch.zeros((pages + B * per, block, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros((B, Hq, D), dtype=torch.bfloat16, device=DEV)
    tables = torch.arange(pages, pages + B * per, dtype=torch.int32, device=DEV).view(B, per)
    args = (q, kc, vc, tables, i32([own] * B), torch.arange(pages, dtype=torch.int32, device=DEV), i32([P]))
    ws = torch.empty((swa.thd_attn_shared_prefix_workspace_bytes(B, 1, Hq, Hkv, D),), dtype=torch.uint8, device=DEV)
    times = []
    for _ in range(8):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(10):
            swa.thd_attn_shared_prefix(*args, workspace=ws)
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 100)
    return sorted(times[1:])[3]


@pytest.mark.parametrize("B,P", [(64, 4096), (256, 16384)])
def test_few_own_tokens_cost_no_more_than_many(B, P):
    # reading 200 tokens a request is more work than reading one; the SMs were shared as
    # if items without keys to speak of took no time (135 against 43 us for 64 requests)
    assert call_us(B, 1, P) <= 1.3 * call_us(B, 200, P)


def test_fewer_own_tokens_cost_no_more_at_head_dim_256():
    kw = dict(P=65536, Hq=16, Hkv=1, D=256)
    assert call_us(256, 200, **kw) <= 1.1 * call_us(256, 1000, **kw)      # (490 against 410 us with too high a rate)


# --------------------------------------------------------- many calls in a row

@pytest.mark.parametrize("D,B,Hq,Hkv,P,own", [(256, 64, 16, 1, 32768, 700), (128, 64, 64, 8, 16384, 700), (64, 128, 32, 8, 32768, 700)])
def test_many_calls_without_a_stall_and_with_the_same_bits(D, B, Hq, Hkv, P, own):
    # both producers of the prefix's ring, with pages all over the cache and memory busy
    block = 16
    per, pages = -(-own // block), P // block
    g = torch.Generator(device=DEV).manual_seed(7)
    kc, vc, q = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in
                 ((pages + B * per, block, Hkv, D), (pages + B * per, block, Hkv, D), (B, Hq, D)))
    perm = torch.randperm(pages + B * per, generator=g, device=DEV).to(torch.int32)
    args = (q, kc, vc, perm[pages:].view(B, per).contiguous(), i32([own] * B), perm[:pages].contiguous(), i32([P]))
    ws = torch.empty((swa.thd_attn_shared_prefix_workspace_bytes(B, 1, Hq, Hkv, D),), dtype=torch.uint8, device=DEV)
    first = swa.thd_attn_shared_prefix(*args, workspace=ws)
    for i in range(3000):
        out = swa.thd_attn_shared_prefix(*args, workspace=ws)
        if i % 300 == 299:
            assert swa.thd_attn_shared_prefix_get_error() == 0
            assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
