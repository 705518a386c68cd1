"""The serving oracle against the packed-attention oracle and hand examples."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as OS
from sliding_window_gqa_cu_b200 import workloads


@pytest.mark.parametrize("P,lens,n_q,window,sinks", [
    (21, [1, 7, 16, 30], 1, 0, False),
    (0, [3, 20], 2, 0, True),
    (16, [5, 40], 3, 12, True),
    (33, [2, 9], 2, 40, False),
])
def test_equals_the_packed_oracle_on_whole_sequences(P, lens, n_q, window, sinks):
    Hq, Hkv, D, block = 4, 2, 16, 4
    rng = np.random.default_rng(P + len(lens))
    pages = lambda n: -(-n // block)
    n_blocks = pages(P) + sum(map(pages, lens))
    kc = rng.standard_normal((n_blocks, block, Hkv, D))
    vc = rng.standard_normal((n_blocks, block, Hkv, D))
    perm = rng.permutation(n_blocks)
    pt, at = perm[:pages(P)], pages(P)
    tables = np.full((len(lens), max(map(pages, lens))), -1)
    for b, n in enumerate(lens):
        tables[b, :pages(n)] = perm[at:at + pages(n)]
        at += pages(n)
    q = rng.standard_normal((len(lens) * n_q, Hq, D))
    snk = rng.standard_normal(Hq) if sinks else None
    out, lse, _, _ = OS.shared_prefix_attention(q, kc, vc, tables, np.array(lens), pt if P else None, P, window,
                                                0.25, snk)
    flat_k, flat_v = kc.reshape(-1, Hkv, D), vc.reshape(-1, Hkv, D)
    for b, n in enumerate(lens):
        slot = [pt[j // block] * block + j % block for j in range(P)] + \
               [tables[b, j // block] * block + j % block for j in range(n)]
        L = P + n
        # the packed oracle on the whole sequence; the queries before the last n_q are zeros
        qq = np.zeros((L, Hq, D))
        qq[L - n_q:] = q[b * n_q:(b + 1) * n_q]
        as_t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
        # bf16-exact inputs are needed by the packed oracle: round them, and compare on the rounded ones
        o2, l2 = oracle.attention(as_t(qq), as_t(flat_k[slot]), as_t(flat_v[slot]), [0, L], window, 0.25,
                                  torch.from_numpy(snk.astype(np.float32)) if sinks else None)
        r = lambda x: as_t(x).double().numpy()
        o1, l1, _, _ = OS.shared_prefix_attention(
            r(q[b * n_q:(b + 1) * n_q]), r(kc), r(vc), tables[b:b + 1], np.array([n]), pt if P else None, P, window,
            0.25, snk.astype(np.float32) if sinks else None)
        assert np.abs(o1 - o2[L - n_q:]).max() < 1e-12 and np.abs(l1 - l2[L - n_q:]).max() < 1e-12
    assert np.isfinite(out).all() and np.isfinite(lse).all()


def test_empty_rows_bad_pages_and_vacant_requests():
    kc = np.ones((2, 2, 1, 4))
    vc = np.arange(16, dtype=float).reshape(2, 2, 1, 4)
    q = np.ones((3, 1, 4))
    tables = np.array([[0, 1], [7, 1], [0, 0]])
    out, lse, _, _ = OS.shared_prefix_attention(q, kc, vc, tables, np.array([0, 3, -1]), scale=0.5)
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf          # no key
    assert np.allclose(out[1, 0], vc[1, 0, 0])                   # page 7 does not exist: one key is left
    assert np.isnan(out[2]).all()                                # vacant
    out, lse, _, _ = OS.shared_prefix_attention(q[:1], kc, vc, tables[:1], np.array([0]), scale=0.5,
                                                sinks=np.array([0.75]))
    assert (out[0] == 0).all() and lse[0, 0] == 0.75


def test_block_tables_by_hand():
    # pages of 4 tokens; request 0 grows into a new page, 1 ends (two pages
    # back), 2 begins with 5 tokens, 3 is vacant, 4 adds a token inside its page
    table = [[3, -1, -1], [5, 6, -1], [-1, -1, -1], [-1, -1, -1], [8, -1, -1]]
    r = OS.block_tables([4, 7, 0, -1, 2], [1, -1, 5, 9, 1], table, [9, 2, 0, 0], 2, 4, 9, first_position=100)
    assert r["free"].tolist() == [9, 2, 5, 6] and r["free_count"] == 1 and r["refused"] == 0
    assert r["table"].tolist() == [[3, 6, -1], [5, 6, -1], [5, 2, -1], [-1] * 3, [8, -1, -1]]
    assert r["seq_lens"].tolist() == [5, -1, 5, -1, 3]
    assert r["cu"].tolist() == [0, 1, 1, 6, 6, 7]
    assert r["slots"].tolist() == [24, 20, 21, 22, 23, 8, 34, -1, -1]
    assert r["positions"].tolist() == [104, 100, 101, 102, 103, 104, 102, 0, 0]


def test_block_tables_refusals_by_hand():
    # two free pages: request 0 wants two, 1 wants one (none left), 2 none, 3 too wide
    table = [[-1] * 2, [-1] * 2, [4, -1], [-1] * 2]
    r = OS.block_tables([0, 0, 1, 0], [5, 2, 2, 9], table, [7, 8], 2, 4, 20)
    assert r["refused"] == 2 and r["seq_lens"].tolist() == [5, 0, 3, 0] and r["free_count"] == 0
    assert r["slots"].tolist() == [32, 33, 34, 35, 28, -1, -1, 17, 18] + [-1] * 11
    # rows: the second request does not fit three rows, the third neither
    r = OS.block_tables([0, 0, 0], [2, 2, 1], [[-1]] * 3, [1, 2, 3], 3, 4, 3)
    assert r["refused"] == 2 and r["slots"].tolist() == [12, 13, -1] and r["free_count"] == 2


def test_kv_write_by_hand():
    cache = np.zeros((2, 2, 1, 1))
    got = OS.kv_write(np.array([[[1.0]], [[2.0]], [[3.0]]]), [3, -1, 4], cache)
    assert got.reshape(-1).tolist() == [0, 0, 0, 1]
