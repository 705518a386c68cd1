"""The serving step as a server runs it: steps without requests, steps replayed
from a captured graph, block tables of every size class."""
import numpy as np
import pytest
import torch

from oracle import serving as OS
import sliding_window_gqa_cu_b200 as swa
from sliding_window_gqa_cu_b200 import build

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
