"""GPU parity of the serving step (thd_kv_block_tables, thd_kv_write,
thd_attn_shared_prefix) against the fp64 oracle.

Tables and caches are compared bit for bit.

Attention tolerance, per element.  The kernel may round the weights p to bf16
for the second product (2^-8 relative each) and rounds the output once (2^-8).
A product of bf16 numbers is exact in fp32; a sum of D of them on the tensor
core is off by at most about D 2^-22 of the sum of magnitudes (each addition may
truncate instead of rounding), so a score by e = (D + 16) 2^-22 reach, with
reach = scale max_j sum_d |q_d k_jd|; a weight and the sum of weights by the
same relative amount plus 2^-20 for the exponential and the fp32 sums:
  |out - ref| <= 2^-8 |ref| + (2^-8 (1 + 2^-7) + 2 e + 2^-19) spread
with spread = sum_j p_j |v_j|, and |lse - ref| <= e + 2^-20 (1 + |ref|).
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import prologue as OP
from oracle import serving as OS
import sliding_window_gqa_cu_b200 as swa
from sliding_window_gqa_cu_b200 import build, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    swa.load_library()


# ------------------------------------------------------------------ attention

def make_case(seed, P, lens, n_q, Hq, Hkv, D, block, window=0, sinks=False, layout="thd", std=1.0, extra_pages=2,
              extra_cols=1):
    """CPU inputs.  Slots that no request owns hold NaN, table entries behind a
    request's pages hold nonsense."""
    rng = np.random.default_rng([seed, P, n_q, Hq, D])
    pages = lambda n: -(-max(n, 0) // block)
    n_blocks = pages(P) + sum(map(pages, lens)) + extra_pages
    perm = rng.permutation(n_blocks).astype(np.int32)
    M = max(map(pages, lens)) + extra_cols
    tables = rng.choice(np.array([-1, n_blocks, 2 ** 31 - 1, -2 ** 31], dtype=np.int32), size=(len(lens), M))
    pt, at = perm[:pages(P)], pages(P)
    used = np.zeros((n_blocks, block), dtype=bool)
    for j in range(P):
        used[pt[j // block], j % block] = True
    for b, n in enumerate(lens):
        tables[b, :pages(n)] = perm[at:at + pages(n)]
        at += pages(n)
        for j in range(max(n, 0)):
            used[tables[b, j // block], j % block] = True
    kv = workloads.random_bf16(rng, (2, n_blocks, block, Hkv, D), std)
    kv[:, torch.from_numpy(~used)] = float("nan")
    q = workloads.random_bf16(rng, (len(lens) * n_q, Hq, D), std)
    snk = torch.from_numpy(rng.standard_normal(Hq).astype(np.float32)) if sinks else None
    return dict(q=q, kc=kv[0], vc=kv[1], tables=torch.from_numpy(tables.astype(np.int32)),
                lens=torch.tensor(lens, dtype=torch.int32), pt=torch.from_numpy(pt) if P else None, P=P,
                window=window, scale=D ** -0.5, sinks=snk, layout=layout, n_q=n_q)


def cache_dev(x, layout):
    x = x.to(DEV)
    return x.transpose(1, 2).contiguous().transpose(1, 2) if layout == "htd" else x


def args_dev(c):
    d = lambda x: None if x is None else x.to(DEV)
    return dict(q=d(c["q"]), k_cache=cache_dev(c["kc"], c["layout"]), v_cache=cache_dev(c["vc"], c["layout"]),
                block_tables=d(c["tables"]), kv_lens=d(c["lens"]), prefix_table=d(c["pt"]),
                prefix_len=torch.tensor([c["P"]], dtype=torch.int32, device=DEV) if c["pt"] is not None else None,
                window=c["window"], scale=c["scale"], sinks=d(c["sinks"]))


def reference(c):
    kc, vc = torch.nan_to_num(c["kc"].double(), nan=0.0), torch.nan_to_num(c["vc"].double(), nan=0.0)
    return OS.shared_prefix_attention(c["q"], kc, vc, c["tables"], c["lens"], c["pt"], c["P"], c["window"],
                                      np.float32(c["scale"]).item(), c["sinks"])


def compare(out, lse, ref, D, what=""):
    ro, rl, spread, reach = ref
    o, l = out.cpu().double().numpy(), lse.cpu().double().numpy()
    live = ~np.isnan(rl)
    e = (D + 16) * 2.0 ** -22 * reach
    bound = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 * (1 + 2.0 ** -7) + 2 * e[..., None] + 2.0 ** -19) * spread
    assert np.isfinite(o[live]).all(), what
    worst = (np.abs(o - ro) - bound)[live].max()
    assert worst <= 0, f"{what}: out exceeds its bound by {worst:.3e}"
    none = live & (rl == -np.inf)
    assert (l[none] == -np.inf).all() and (o[none] == 0).all(), what
    some = live & ~none
    assert (np.abs(l - rl)[some] <= (e + 2.0 ** -20 * (1 + np.abs(rl)))[some]).all(), what


def run_and_compare(c, what=""):
    out, lse = swa.thd_attn_shared_prefix(**args_dev(c))
    assert swa.thd_attn_shared_prefix_get_error() == 0
    compare(out, lse, reference(c), c["q"].shape[2], what)
    return out, lse


CASES = [
    # one token everywhere; a prefix of one key; page borders on every side
    dict(P=0, lens=[1], n_q=1, Hq=4, Hkv=2, D=64, block=16),
    dict(P=1, lens=[1, 2], n_q=1, Hq=4, Hkv=2, D=64, block=16),
    dict(P=16, lens=[16, 15, 17], n_q=1, Hq=8, Hkv=2, D=128, block=16),
    dict(P=127, lens=[127, 128, 129, 1], n_q=1, Hq=8, Hkv=2, D=128, block=32),
    dict(P=128, lens=[63, 64, 65], n_q=1, Hq=16, Hkv=1, D=256, block=64, sinks=True),
    dict(P=129, lens=[255, 256, 257], n_q=1, Hq=32, Hkv=8, D=64, block=128, sinks=True),
    dict(P=300, lens=[5, 300, 77], n_q=1, Hq=8, Hkv=8, D=128, block=256),
    # several queries per request, more than there are own tokens among them
    dict(P=40, lens=[1, 3, 20], n_q=3, Hq=8, Hkv=2, D=128, block=16),
    dict(P=2, lens=[1, 0, 20], n_q=5, Hq=8, Hkv=2, D=64, block=16),
    dict(P=0, lens=[1, 0, 2], n_q=4, Hq=8, Hkv=2, D=64, block=16, sinks=True),
    # a group that does not divide 128, and groups of 1, 32 and 128
    dict(P=150, lens=[30, 200], n_q=7, Hq=12, Hkv=2, D=128, block=16),
    dict(P=150, lens=[30, 200], n_q=40, Hq=10, Hkv=2, D=64, block=16),
    dict(P=70, lens=[130, 1, 9], n_q=9, Hq=32, Hkv=1, D=128, block=32),
    dict(P=70, lens=[130, 4], n_q=3, Hq=128, Hkv=1, D=64, block=32),
    dict(P=70, lens=[130, 140], n_q=150, Hq=2, Hkv=2, D=128, block=32),
    # windows: inside the own tokens, across the border, longer than everything, of one token
    dict(P=200, lens=[300, 50, 120], n_q=2, Hq=8, Hkv=2, D=128, block=16, window=100),
    dict(P=700, lens=[10, 200, 64], n_q=1, Hq=8, Hkv=2, D=128, block=16, window=150, sinks=True),
    dict(P=100, lens=[10, 20], n_q=3, Hq=8, Hkv=2, D=128, block=64, window=5000),
    dict(P=33, lens=[1, 20], n_q=2, Hq=8, Hkv=2, D=256, block=16, window=1),
    dict(P=600, lens=[0, 400], n_q=2, Hq=16, Hkv=1, D=256, block=16, window=130, sinks=True),
    # heads outermost in a page
    dict(P=333, lens=[100, 7, 260], n_q=2, Hq=8, Hkv=4, D=128, block=16, layout="htd"),
    dict(P=333, lens=[100, 7], n_q=1, Hq=16, Hkv=2, D=256, block=64, layout="htd", sinks=True),
    # many rows share the prefix (several row tiles per kv head), no own token for some
    dict(P=520, lens=[3] * 40, n_q=1, Hq=16, Hkv=2, D=128, block=16),
    dict(P=520, lens=[0, 9, 2] * 30, n_q=1, Hq=16, Hkv=2, D=64, block=16),
    dict(P=260, lens=[4, 9] * 16, n_q=2, Hq=16, Hkv=1, D=256, block=32, sinks=True),
    # many short requests: several per processor
    dict(P=0, lens=list(range(1, 201)), n_q=1, Hq=8, Hkv=8, D=64, block=16),
    dict(P=17, lens=[1, 40] * 100, n_q=1, Hq=8, Hkv=4, D=128, block=16, sinks=True),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join(
    f"{n}{v if not isinstance(v, list) else len(v)}" for n, v in k.items()))
def test_attention_parity(kw):
    run_and_compare(make_case(1, **kw), str(kw))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 8, 2), (256, 8, 1)])
def test_long_sequences(D, Hq, Hkv):
    run_and_compare(make_case(2, P=9001, lens=[5003, 1, 2048], n_q=1, Hq=Hq, Hkv=Hkv, D=D, block=16, sinks=True))


def test_pages_outside_the_cache_contribute_no_keys():
    c = make_case(3, P=300, lens=[100, 200, 300], n_q=2, Hq=8, Hkv=2, D=128, block=16)
    c["tables"][0, 2] = -1
    c["tables"][1, 12] = c["kc"].shape[0]
    c["tables"][2, :19] = 2 ** 31 - 1                       # nothing of its own is left
    c["pt"][3:11] = -7
    run_and_compare(c)


def test_a_request_whose_pages_are_all_outside_has_empty_rows():
    c = make_case(4, P=0, lens=[33, 200], n_q=1, Hq=8, Hkv=2, D=128, block=16)
    c["tables"][1] = -1
    out, lse = run_and_compare(c)
    assert (out[1] == 0).all() and (lse[1] == float("-inf")).all()


def test_lengths_beyond_the_tables_are_cut():
    c = make_case(5, P=64, lens=[48, 64], n_q=1, Hq=8, Hkv=2, D=64, block=16, extra_cols=0)
    want = reference(c)
    a = args_dev(c)
    # request 1 holds its whole table, so a longer length means the same;
    # the prefix fills its table too
    a["kv_lens"] = torch.tensor([48, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    a["prefix_len"] = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out, lse = swa.thd_attn_shared_prefix(**a)
    compare(out, lse, want, 64)
    a["prefix_len"].fill_(-5)                               # negative: no prefix
    out, lse = swa.thd_attn_shared_prefix(**a)
    c.update(pt=None, P=0)
    compare(out, lse, reference(c), 64)


def test_vacant_requests_keep_their_rows():
    c = make_case(6, P=100, lens=[20, -1, 30, -9], n_q=2, Hq=8, Hkv=2, D=128, block=16)
    a = args_dev(c)
    out = torch.full((8, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((8, 8), 5.0, device=DEV)
    swa.thd_attn_shared_prefix(**a, out=out, lse=lse)
    compare(out, lse, reference(c), 128)
    for b in (1, 3):
        assert (out[2 * b:2 * b + 2] == 3).all() and (lse[2 * b:2 * b + 2] == 5).all()
    # no request at all
    a["kv_lens"].fill_(-1)
    out.fill_(3.0)
    swa.thd_attn_shared_prefix(**a, out=out, lse=lse)
    assert (out == 3).all() and swa.thd_attn_shared_prefix_get_error() == 0


def test_no_requests_and_no_lse():
    c = make_case(7, P=30, lens=[20, 3], n_q=1, Hq=8, Hkv=2, D=64, block=16)
    a = args_dev(c)
    o1, l1 = swa.thd_attn_shared_prefix(**a, return_lse=False)
    o2, _ = swa.thd_attn_shared_prefix(**a)
    assert l1 is None and torch.equal(o1, o2)
    for n in ("q", "block_tables", "kv_lens"):
        a[n] = a[n][:0]
    o, l = swa.thd_attn_shared_prefix(**a)
    assert o.shape == (0, 8, 64) and l.shape == (0, 8)


def test_sink_of_minus_infinity_is_no_sink():
    c = make_case(8, P=50, lens=[20, 0], n_q=1, Hq=8, Hkv=2, D=64, block=16)
    a = args_dev(c)
    want = swa.thd_attn_shared_prefix(**a)
    a["sinks"] = torch.full((8,), float("-inf"), device=DEV)
    got = swa.thd_attn_shared_prefix(**a)
    compare(*got, reference(c), 64)
    assert torch.equal(got[0], want[0])


def test_same_result_every_time_and_with_a_used_workspace():
    c = make_case(9, P=3000, lens=[700, 40, 1300] * 6, n_q=1, Hq=16, Hkv=2, D=128, block=16)
    a = args_dev(c)
    n = swa.thd_attn_shared_prefix_workspace_bytes(18, 1, 16, 2, 128)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)        # NaN everywhere
    first = swa.thd_attn_shared_prefix(**a, workspace=ws)
    compare(*first, reference(c), 128)
    for _ in range(5):
        again = swa.thd_attn_shared_prefix(**a, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    with pytest.raises(swa.ThdAttnError):
        swa.thd_attn_shared_prefix(**a, workspace=ws[: n - 16])


def test_two_streams_at_once():
    cases = [make_case(10 + i, P=2000, lens=[900, 30, 500, 64], n_q=1, Hq=16, Hkv=2, D=128, block=16) for i in range(2)]
    args = [args_dev(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [[], []]
    for _ in range(10):
        for i in (0, 1):
            res[i].append(swa.thd_attn_shared_prefix(**args[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        compare(*res[i][0], reference(cases[i]), 128)
        assert all(torch.equal(res[i][0][0], r[0]) for r in res[i])


def test_captured_graph_follows_lengths_and_tables():
    c = make_case(12, P=260, lens=[300, 200, 100], n_q=1, Hq=8, Hkv=2, D=128, block=16)
    short = dict(c, lens=torch.tensor([17, 200, -1], dtype=torch.int32), P=100)
    a = args_dev(c)
    n = swa.thd_attn_shared_prefix_workspace_bytes(3, 1, 8, 2, 128)
    ws = torch.empty((n,), dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((3, 8), device=DEV)
    swa.thd_attn_shared_prefix(**a, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        swa.thd_attn_shared_prefix(**a, out=out, lse=lse, workspace=ws)
    for case in (short, c, short):
        a["kv_lens"].copy_(case["lens"])
        a["prefix_len"].fill_(case["P"])
        g.replay()
        torch.cuda.synchronize()
        compare(out, lse, reference(case), 128)


def test_interleaved_caches_and_offsets_past_32_bits():
    # k and v of a page side by side in one pool whose last pages lie past 2^32 bytes
    block, Hkv, D = 16, 8, 128
    pages = (5 << 30) // (2 * block * Hkv * D * 2)
    pool = torch.zeros((pages, 2, block, Hkv, D), dtype=torch.bfloat16, device=DEV)
    kc, vc = pool[:, 0], pool[:, 1]
    c = make_case(13, P=40, lens=[100, 33], n_q=1, Hq=16, Hkv=Hkv, D=D, block=block)
    n = c["kc"].shape[0]
    kc[pages - n:] = c["kc"].to(DEV)
    vc[pages - n:] = c["vc"].to(DEV)
    a = args_dev(c)
    ok = (c["tables"] >= 0) & (c["tables"] < n)
    a.update(k_cache=kc, v_cache=vc, prefix_table=a["prefix_table"] + (pages - n),
             block_tables=torch.where(ok, c["tables"] + (pages - n), torch.tensor(-1, dtype=torch.int32)).to(DEV))
    out, lse = swa.thd_attn_shared_prefix(**a)
    compare(out, lse, reference(c), D)
    # and the write reaches them
    slots = torch.tensor([(pages - 1) * block + 3, 5], dtype=torch.int32, device=DEV)
    k = torch.randn((2, Hkv, D), device=DEV).to(torch.bfloat16)
    swa.thd_kv_write(k, -k, slots, kc, vc)
    assert torch.equal(kc[pages - 1, 3], k[0]) and torch.equal(vc[pages - 1, 3], -k[0])
    assert torch.equal(kc[0, 5], k[1]) and torch.equal(vc[0, 5], -k[1])


def test_attention_refuses():
    c = make_case(14, P=30, lens=[20, 3], n_q=1, Hq=8, Hkv=2, D=64, block=16)
    a = args_dev(c)
    for bad in (dict(q=a["q"][:, :, :32]), dict(q=a["q"].float()), dict(q=a["q"][:1]), dict(kv_lens=a["kv_lens"].long()),
                dict(kv_lens=a["kv_lens"][:1]), dict(prefix_table=None), dict(prefix_len=None),
                dict(prefix_len=a["prefix_len"].cpu()), dict(sinks=torch.zeros(4, device=DEV)),
                dict(block_tables=a["block_tables"][:, ::2]), dict(k_cache=a["k_cache"].float()),
                dict(out=torch.empty((2, 8, 64), device=DEV)), dict(lse=torch.empty((2, 4), device=DEV))):
        with pytest.raises(ValueError):
            swa.thd_attn_shared_prefix(**{**a, **bad})


# --------------------------------------------------------------- block tables

def run_tables(seq, new, table, free, count, block, rows, first=None, **kw):
    d = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)
    t, f = d(table), d(free)
    got = swa.thd_kv_block_tables(d(seq), d(new), t, f, d([count]), block, rows,
                                  first_position=None if first is None else d([first]), **kw)
    names = ("seq_lens", "free_count", "cu", "slots", "positions", "refused")
    r = {n: x.cpu().numpy().astype(np.int64) for n, x in zip(names, got)}
    r.update(table=t.cpu().numpy(), free=f.cpu().numpy())
    return r


def check_tables(seq, new, table, free, count, block, rows, first=None):
    got = run_tables(seq, new, table, free, count, block, rows, first)
    want = OS.block_tables(seq, new, table, free, count, block, rows, first or 0)
    for n in ("seq_lens", "cu", "slots", "positions", "table", "free"):
        assert np.array_equal(got[n], want[n]), n
    assert got["free_count"][0] == want["free_count"] and got["refused"][0] == want["refused"]
    return want


@pytest.mark.parametrize("B,block,M,seed", [(1, 16, 4, 0), (7, 1, 9, 1), (31, 16, 8, 2), (33, 3, 20, 3), (300, 32, 6, 4),
                                            (1024, 16, 5, 5), (1025, 16, 5, 6), (8192, 64, 3, 7)])
@pytest.mark.parametrize("scarce", [False, True])
def test_block_tables_random(B, block, M, seed, scarce):
    rng = np.random.default_rng([seed, scarce])
    cap = M * block
    seq = rng.integers(0, cap + 1, size=B)
    seq[rng.uniform(size=B) < 0.15] = -1
    new = rng.integers(0, 3 * block + 2, size=B)
    new[rng.uniform(size=B) < 0.2] = -1
    new[rng.uniform(size=B) < 0.2] = 0
    held = np.where(seq > 0, -(-seq // block), 0)
    pool = int(held.sum()) + (max(1, B // 3) if scarce else B * M)
    perm = rng.permutation(pool).astype(np.int64)
    table, at = np.full((B, M), -1), 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(pool, -1)
    free[:pool - at] = perm[at:]
    grow = np.where((seq >= 0) & (new > 0), new, 0)
    rows = int(grow.sum() * (0.8 if scarce else 1.0)) + (0 if scarce else 5)
    want = check_tables(seq, new, table, free, pool - at, block, rows, 77)
    assert scarce == (want["refused"] > 0) or not scarce
    live = want["slots"][want["slots"] >= 0]
    assert np.unique(live).size == live.size                # no slot is given twice


def test_block_tables_edges():
    check_tables([0], [0], [[-1]], [4], 1, 16, 0)                         # nothing to do, no rows
    check_tables([0], [0], [[-1]], [], 0, 16, 3)                          # an empty pool
    check_tables([-1, -5], [3, -1], [[1], [2]], [0], 1, 16, 4)            # vacant entries only
    check_tables([16], [1], [[1]], [5], 1, 16, 1)                         # no room in the table
    check_tables([5], [-1], [[1, 2]], [9, 9], 2, 4, 0)                    # the stack is full: nothing is pushed
    check_tables([0, 0], [70000, 2], [[-1] * 5000] * 2, list(range(5000)), 5000, 16, 70002, 1 << 20)
    check_tables([3], [2 ** 31 - 1], [[1, 2]], [9, 8], 2, 4, 10)          # a length past 2^31
    check_tables([100, 2], [-1, 2], [[1, 2], [3, -1]], [9, 8, 7], 1, 4, 4)  # a length past its table


def test_block_tables_in_place_and_into_buffers():
    d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    seq, new, count = d([4, 7, 0, -1, 2]), d([1, -1, 5, 9, 1]), d([2])
    table = d([[3, -1, -1], [5, 6, -1], [-1, -1, -1], [-1, -1, -1], [8, -1, -1]])
    free, slots = d([9, 2, 0, 0]), d([7] * 9)
    r = swa.thd_kv_block_tables(seq, new, table, free, count, 4, 9, first_position=d([100]), seq_lens_out=seq,
                                free_count_out=count, slots=slots)
    assert r[0] is seq and r[1] is count and r[3] is slots
    assert seq.tolist() == [5, -1, 5, -1, 3] and count.tolist() == [1]
    assert slots.tolist() == [24, 20, 21, 22, 23, 8, 34, -1, -1]
    assert table.tolist() == [[3, 6, -1], [5, 6, -1], [5, 2, -1], [-1] * 3, [8, -1, -1]]


def test_block_tables_unaligned_outputs():
    d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    buf = torch.full((2, 40), 9, dtype=torch.int32, device=DEV)
    r = swa.thd_kv_block_tables(d([0, 0]), d([20, 11]), d([[-1] * 2] * 2), d([0, 1, 2, 3]), d([4]), 16, 31,
                                slots=buf[0, 1:32], positions=buf[1, 3:34])
    assert r[4].tolist() == list(range(20)) + list(range(11))
    assert r[3].tolist() == list(range(48, 64)) + list(range(32, 36)) + list(range(16, 27))
    assert buf[0, 0] == 9 and (buf[0, 32:] == 9).all() and (buf[1, :3] == 9).all() and (buf[1, 34:] == 9).all()


# -------------------------------------------------------------------- kv write

@pytest.mark.parametrize("T,Hq,Hkv,D,block,fused,layout", [
    (1, 4, 2, 64, 16, False, "thd"), (7, 4, 2, 64, 1, True, "thd"), (130, 8, 1, 256, 16, True, "htd"),
    (1000, 16, 8, 128, 48, True, "thd"), (777, 5, 5, 128, 64, False, "htd"), (5000, 32, 8, 64, 32, True, "htd"),
])
def test_kv_write_parity(T, Hq, Hkv, D, block, fused, layout):
    rng = np.random.default_rng([T, D])
    nb = -(-T // block) + 3
    qkv = workloads.random_bf16(rng, (T, Hq + 2 * Hkv, D))
    slots = rng.permutation(nb * block)[:T].astype(np.int32)
    slots[rng.uniform(size=T) < 0.1] = -1
    if T > 5:
        slots[[2, 4, 5]] = [nb * block, 2 ** 31 - 1, -2 ** 31]
    kc, vc = (workloads.random_bf16(rng, (nb, block, Hkv, D)) for _ in range(2))
    g = qkv.to(DEV)
    k, v = g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    kd, vd = cache_dev(kc, layout), cache_dev(vc, layout)
    r = swa.thd_kv_write(k, v, torch.from_numpy(slots).to(DEV), kd, vd)
    assert r[0] is kd and r[1] is vd
    bits = workloads.bf16_bits
    assert np.array_equal(bits(kd.cpu()), OS.kv_write(bits(qkv[:, Hq:Hq + Hkv]), slots, bits(kc)))
    assert np.array_equal(bits(vd.cpu()), OS.kv_write(bits(qkv[:, Hq + Hkv:]), slots, bits(vc)))


def test_kv_write_refuses():
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    c = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad in (dict(k=k.float()), dict(k=k[:2]), dict(v=k[:, :, :32]), dict(slots=s.long()), dict(slots=s.cpu()),
                dict(k_cache=c.float()), dict(v_cache=c[:1]), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            swa.thd_kv_write(**{**dict(k=k, v=k, slots=s, k_cache=c, v_cache=c), **bad})
    with pytest.raises(swa.ThdAttnError):                       # rows that repeat
        swa.thd_kv_write(k[:1].expand(3, 2, 64), k, s, c, c)


# ------------------------------------------------------------ the step as a run

@pytest.mark.parametrize("window,sinks", [(0, False), (90, True)])
def test_prompt_then_answers_match_the_packed_oracle(window, sinks):
    """A shared prompt through the packed forward into the cache, the requests'
    own prompts, then decoding with two drafted tokens a step, one request
    ending and another taking its pages; every step against the packed oracle on
    the whole sequences."""
    Hq, Hkv, D, block, B, M = 8, 2, 64, 16, 4, 8
    P, scale = 75, 64 ** -0.5
    rng = np.random.default_rng(5)
    dev = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)
    nb = 40
    kc, vc = (torch.full((nb, block, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    free, count = dev(rng.permutation(nb)), dev([nb])
    snk = torch.from_numpy(rng.standard_normal(Hq).astype(np.float32)) if sinks else None
    snk_d = snk.to(DEV) if sinks else None
    tok = lambda n: tuple(workloads.random_bf16(rng, (n, h, D)) for h in (Hq, Hkv, Hkv))

    def prologue(q, k, pos):
        f = lambda x: torch.from_numpy(OP.qk_norm_rope(x, None, positions=pos)).to(torch.bfloat16)
        return f(q), f(k)

    # the shared prompt: a request of its own in a table of its own
    q, k, v = tok(P)
    pt = dev(np.full((1, 5), -1))
    plen, count, _, slots, positions, refused = swa.thd_kv_block_tables(dev([0]), dev([P]), pt, free, count, block, P)
    assert refused.item() == 0 and positions.tolist() == list(range(P))
    qd, kd, vd = (x.to(DEV) for x in (q, k, v))
    swa.thd_qk_norm_rope(qd, kd, [0, P], positions=positions)
    swa.thd_kv_write(kd, vd, slots, kc, vc)
    swa.thd_attn_fwd(qd, kd, vd, [0, P], window, scale, snk_d)
    hist = {"prefix": (kd.cpu(), v)}
    own = [None] * B
    seq, table = dev([0, 0, -1, 0]), dev(np.full((B, M), -1))

    def step(new, n_q):
        nonlocal seq, count
        total = int(sum(max(m, 0) for m, n in zip(new, seq.tolist()) if n >= 0))
        rows = total + 3                                   # a padded batch
        seq, count, cu, slots, positions, refused = swa.thd_kv_block_tables(
            seq, dev(new), table, free, count, block, rows, first_position=plen)
        assert refused.item() == 0
        q, k, v = tok(rows)
        qd, kd, vd = (x.to(DEV) for x in (q, k, v))
        swa.thd_qk_norm_rope(qd, kd, [0, rows], positions=positions)
        swa.thd_kv_write(kd, vd, slots, kc, vc)
        cu = cu.tolist()
        pick, kh = [], kd.cpu()
        for b in range(B):
            if new[b] < 0:
                own[b] = None
            if cu[b + 1] > cu[b]:
                part = (kh[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]])
                own[b] = part if own[b] is None else tuple(torch.cat(x) for x in zip(own[b], part))
            pick += [max(0, cu[b + 1] - n_q + i) for i in range(n_q)]
        qq = qd[torch.tensor(pick, device=DEV)].contiguous()
        out, lse = swa.thd_attn_shared_prefix(qq, kc, vc, table, seq, pt[0], plen, window, scale, snk_d)
        assert swa.thd_attn_shared_prefix_get_error() == 0
        for b in range(B):
            if own[b] is None:
                continue
            ks, vs = (torch.cat([hist["prefix"][i], own[b][i]]) for i in (0, 1))
            L = ks.shape[0]
            assert L == P + int(seq[b])
            full = torch.zeros((L, Hq, D), dtype=torch.bfloat16)
            full[L - n_q:] = qq[b * n_q:(b + 1) * n_q].cpu()
            ro, rl = oracle.attention(full, ks, vs, [0, L], window, scale, snk)
            err = np.abs(out[b * n_q:(b + 1) * n_q].cpu().double().numpy() - ro[L - n_q:])
            assert err.max() <= 2e-2 and err.mean() <= 2e-3
            assert np.abs(lse[b * n_q:(b + 1) * n_q].cpu().double().numpy() - rl[L - n_q:]).max() <= 1e-3

    step([20, 3, 0, 33], 2)                                # the requests' own prompts
    for _ in range(3):
        step([2, 2, 0, 2], 2)
    step([2, -1, 0, 2], 2)                                 # request 1 ends
    seq[1] = 0
    step([2, 40, 0, 2], 2)                                 # its pages serve another
    step([1, 1, 0, 1], 1)


# --------------------------------- many rows: the prefix on the tensor cores

MANY = [
    # several row groups and bundles of a kv head; groups that end inside a tile
    dict(P=700, lens=[1] * 300, n_q=1, Hq=8, Hkv=1, D=64, block=16),
    dict(P=131, lens=[7, 40] * 65, n_q=2, Hq=10, Hkv=1, D=128, block=32),
    dict(P=1000, lens=[5] * 33, n_q=1, Hq=16, Hkv=2, D=256, block=16),
    # long prefixes: every item in many pieces
    dict(P=9001, lens=[33, 700, 1] * 4, n_q=1, Hq=16, Hkv=2, D=128, block=16, sinks=True),
    dict(P=9001, lens=[33, 700] * 3, n_q=2, Hq=8, Hkv=1, D=64, block=128),
    dict(P=6000, lens=[600, 4] * 3, n_q=1, Hq=16, Hkv=2, D=256, block=64, sinks=True),
    # windows that begin in the prefix of some and behind it for others
    dict(P=3000, lens=[1, 500, 40, 130] * 5, n_q=3, Hq=8, Hkv=2, D=128, block=16, window=400),
    dict(P=2000, lens=[900, 10] * 10, n_q=1, Hq=16, Hkv=2, D=256, block=32, window=300, sinks=True),
    dict(P=513, lens=[600] * 20, n_q=2, Hq=8, Hkv=2, D=64, block=16, window=64),
    # queries inside the prefix (fewer own tokens than queries), and vacant requests
    dict(P=300, lens=[0, 2, -1, 20, -1, -1] * 4, n_q=6, Hq=8, Hkv=2, D=128, block=16),
    dict(P=260, lens=[-1] * 70 + [3] * 9, n_q=1, Hq=8, Hkv=1, D=128, block=16, sinks=True),
    # page sizes from one to two tiles; heads outermost
    dict(P=777, lens=[100, 7] * 9, n_q=1, Hq=16, Hkv=4, D=128, block=256),
    dict(P=777, lens=[100, 7] * 9, n_q=1, Hq=16, Hkv=4, D=128, block=128, layout="htd"),
    dict(P=777, lens=[100, 7] * 9, n_q=1, Hq=16, Hkv=4, D=64, block=32, layout="htd"),
    # large groups: several row tiles of a request in the paged kernel too
    dict(P=200, lens=[150, 90, 31], n_q=9, Hq=32, Hkv=1, D=256, block=32),
    dict(P=200, lens=[150, 90, 31], n_q=5, Hq=128, Hkv=1, D=128, block=16, sinks=True),
]


@pytest.mark.parametrize("kw", MANY, ids=lambda k: "-".join(
    f"{n}{v if not isinstance(v, list) else len(v)}" for n, v in k.items()))
def test_many_rows(kw):
    run_and_compare(make_case(21, **kw), str(kw))


def test_many_rows_with_pages_outside_the_cache():
    c = make_case(22, P=900, lens=[100, 30] * 12, n_q=2, Hq=8, Hkv=2, D=128, block=16)
    c["pt"][5:9] = c["kc"].shape[0]
    c["pt"][20:37] = -2 ** 31                        # whole tiles among them
    c["tables"][3] = -1
    run_and_compare(c)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_blocks_any_distance_apart(D):
    # block, token and head strides with no common divisor but 8 elements
    c = make_case(23, P=300, lens=[70, 20] * 11, n_q=1, Hq=16, Hkv=2, D=D, block=16)
    nb, bs, H, _ = c["kc"].shape
    st, sh = H * (D + 8) + 8, D + 8
    sb = bs * st + 24
    a = args_dev(c)
    for n in ("kc", "vc"):
        t = torch.full((nb * sb,), float("nan"), dtype=torch.bfloat16, device=DEV).as_strided((nb, bs, H, D), (sb, st, sh, 1))
        t.copy_(c[n])
        a["k_cache" if n == "kc" else "v_cache"] = t
    out, lse = swa.thd_attn_shared_prefix(**a)
    compare(out, lse, reference(c), D)


def test_many_rows_captured_follow_lengths():
    c = make_case(24, P=1500, lens=[300, 200, 100, 50] * 4, n_q=1, Hq=16, Hkv=2, D=128, block=16, window=0)
    short = dict(c, lens=torch.tensor([17, 200, -1, 0] * 4, dtype=torch.int32), P=129)
    none = dict(c, pt=None, P=0)
    a = args_dev(c)
    n = swa.thd_attn_shared_prefix_workspace_bytes(16, 1, 16, 2, 128)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros((16, 16, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((16, 16), device=DEV)
    swa.thd_attn_shared_prefix(**a, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        swa.thd_attn_shared_prefix(**a, out=out, lse=lse, workspace=ws)
    for case in (short, c, none, short):
        a["kv_lens"].copy_(case["lens"])
        a["prefix_len"].fill_(case["P"])
        g.replay()
        g.replay()                                          # nothing waits between two steps
        torch.cuda.synchronize()
        compare(out, lse, reference(case), 128)
    assert swa.thd_attn_shared_prefix_get_error() == 0


def test_many_rows_on_two_streams_at_once():
    cases = [make_case(25 + i, P=2500, lens=[900, 30, 500, 64] * 3, n_q=1, Hq=16, Hkv=2, D=128, block=16) for i in range(2)]
    args = [args_dev(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [[], []]
    for _ in range(8):
        for i in (0, 1):
            res[i].append(swa.thd_attn_shared_prefix(**args[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        compare(*res[i][0], reference(cases[i]), 128)
        assert all(torch.equal(res[i][0][j], r[j]) for r in res[i] for j in (0, 1))


def test_large_scores_and_masked_infinities():
    # scores of some hundreds, keys behind the window at the type's largest value
    c = make_case(27, P=600, lens=[40, 9] * 10, n_q=1, Hq=8, Hkv=2, D=128, block=16, window=500, std=6.0)
    kc, vc = c["kc"], c["vc"]
    for j in range(0, 90):                                  # (the furthest window begins at 600 + 9 - 500)
        kc[c["pt"][j // 16], j % 16] = float("inf") if j % 2 else float("-inf")
        vc[c["pt"][j // 16], j % 16] = 3.3e38 if j % 2 else float("-inf")
    ref = reference(dict(c, kc=torch.nan_to_num(kc, posinf=0.0, neginf=0.0), vc=torch.nan_to_num(vc, posinf=0.0, neginf=0.0)))
    out, lse = swa.thd_attn_shared_prefix(**args_dev(c))
    compare(out, lse, ref, 128)


@pytest.mark.parametrize("B", [257, 1025, 8192])
def test_block_tables_in_place_many(B):
    rng = np.random.default_rng(B)
    block, M = 16, 4
    seq, new = rng.integers(-1, 50, size=B), rng.integers(-1, 20, size=B)
    held = np.where(seq > 0, -(-seq // block), 0)
    pool = int(held.sum()) + B // 2
    perm = rng.permutation(pool).astype(np.int64)
    table, at = np.full((B, M), -1), 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(pool, -1)
    free[:pool - at] = perm[at:]
    rows = int(np.where((seq >= 0) & (new > 0), new, 0).sum()) + 3
    want = OS.block_tables(seq, new, table, free, pool - at, block, rows, 0)
    d = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)
    s, t, f, n = d(seq), d(table), d(free), d([pool - at])
    r = swa.thd_kv_block_tables(s, d(new), t, f, n, block, rows, seq_lens_out=s, free_count_out=n)
    got = dict(seq_lens=r[0], cu=r[2], slots=r[3], positions=r[4], table=t, free=f)
    for name, x in got.items():
        assert np.array_equal(x.cpu().numpy(), want[name]), name
    assert n.item() == want["free_count"] and r[5].item() == want["refused"]


def test_step_on_another_stream_than_the_current_one():
    # tables, write and attention on one side stream, nothing on the current one
    side = torch.cuda.Stream()
    B, block, M, Hq, Hkv, D = 40, 16, 3, 8, 2, 64
    d = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)
    rng = np.random.default_rng(7)
    kc, vc = (torch.zeros((B * M, block, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    seq, new = d([0] * B), d(rng.integers(1, 30, size=B))
    table, free, count = d(np.full((B, M), -1)), d(np.arange(B * M)), d([B * M])
    k, v, q = (workloads.random_bf16(rng, s).to(DEV) for s in ((B * 30, Hkv, D), (B * 30, Hkv, D), (B, Hq, D)))
    torch.cuda.synchronize()
    lens, _, cu, slots, _, refused = swa.thd_kv_block_tables(seq, new, table, free, count, block, B * 30, stream=side)
    swa.thd_kv_write(k, v, slots, kc, vc, stream=side)
    out, lse = swa.thd_attn_shared_prefix(q, kc, vc, table, lens, stream=side)
    side.synchronize()
    assert refused.item() == 0
    ref = OS.shared_prefix_attention(q.cpu(), kc.cpu(), vc.cpu(), table, lens, None, 0, 0, np.float32(D ** -0.5).item(), None)
    compare(out, lse, ref, D)
    host = k.cpu()
    for b in (0, 17, B - 1):
        n, first = int(new[b]), int(cu[b])
        pages = table[b].cpu()
        for j in (0, n - 1):
            assert torch.equal(kc[pages[j // block], j % block].cpu(), host[first + j])


# The same with a prefix table that could hold a long prefix: which kernel takes
# the prefix goes by what the table holds (above 8 rows the prefix kernel takes
# 32,768 keys, and below them the paged kernel).

WIDE = [kw for kw in CASES + MANY if kw["P"] > 0]


@pytest.mark.parametrize("kw", WIDE, ids=lambda k: "-".join(
    f"{n}{v if not isinstance(v, list) else len(v)}" for n, v in k.items()))
def test_wide_prefix_tables(kw):
    c = make_case(31, **kw)
    wide = torch.full((32768 // kw["block"],), -1, dtype=torch.int32)
    wide[:len(c["pt"])] = c["pt"]
    a = args_dev(dict(c, pt=wide))
    out, lse = swa.thd_attn_shared_prefix(**a)
    assert swa.thd_attn_shared_prefix_get_error() == 0
    compare(out, lse, reference(c), kw["D"], str(kw))


@pytest.mark.parametrize("D,Hq,Hkv,lens,n_q", [(128, 8, 2, [40, 3], 1), (64, 4, 4, [200], 5), (128, 8, 1, [700, 1, -1, 90], 1),
                                               (256, 8, 1, [20] * 3, 1), (128, 8, 2, [0, 33] * 8, 4)])
def test_wide_prefix_tables_captured_follow_the_prefix(D, Hq, Hkv, lens, n_q):
    c = make_case(32, P=32768, lens=lens, n_q=n_q, Hq=Hq, Hkv=Hkv, D=D, block=64, sinks=True)
    a = args_dev(c)
    T = len(lens) * n_q
    out, lse = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV), torch.zeros((T, Hq), device=DEV)
    swa.thd_attn_shared_prefix(**a, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        swa.thd_attn_shared_prefix(**a, out=out, lse=lse)
    for P in (2500, 0, 65, 2500):
        a["prefix_len"].fill_(P)
        g.replay()
        torch.cuda.synchronize()
        # (slots of the table's pages behind P are not seen)
        compare(out, lse, reference(dict(c, P=P)), D, f"P={P}")
    assert swa.thd_attn_shared_prefix_get_error() == 0


def test_blocks_far_apart_with_few_rows():
    # 2^31 places for the prefix kernel's map (strides share 8 elements): with few rows
    # the paged kernel takes a long table too
    D, Hq, Hkv, block, nb = 64, 8, 2, 16, (1 << 20) + 1
    sb, st, sh = (1 << 14) + 16, Hkv * (D + 8), D + 8
    c = make_case(33, P=700, lens=[40, 9], n_q=2, Hq=Hq, Hkv=Hkv, D=D, block=block)
    n = c["kc"].shape[0]
    far = lambda t: torch.where((t >= 0) & (t < n), t * ((nb - 1) // (n - 1)), -1).int()
    a = args_dev(c)
    wide = torch.full((32768 // block,), -1, dtype=torch.int32)
    wide[:len(c["pt"])] = far(c["pt"])
    a["prefix_table"], a["block_tables"] = wide.to(DEV), far(c["tables"]).to(DEV)
    both = torch.empty((nb * sb,), dtype=torch.bfloat16, device=DEV)     # 34 GB, most of it not touched
    at = far(torch.arange(n)).long().to(DEV)
    for i, name in enumerate(("k", "v")):
        cache = both.as_strided((nb, block, Hkv, D), (sb, st, sh, 1), i * 8192)
        cache[at] = c[name + "c"].to(DEV)
        a[name + "_cache"] = cache
    out, lse = swa.thd_attn_shared_prefix(**a)
    compare(out, lse, reference(c), D)
    many = torch.zeros((9 * 2, Hq, D), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(swa.ThdAttnError):                                # 72 rows a kv head
        swa.thd_attn_shared_prefix(**dict(a, q=many, block_tables=a["block_tables"][:1].expand(9, -1).contiguous(),
                                          kv_lens=a["kv_lens"][:1].expand(9).contiguous()))
