"""What follows a stalled kernel of the shared-prefix attention: calls write nothing,
every stream that asks is told, and after that calls compute again.  The status
word is set from the host (a hook of the debug build); nothing stalls."""
import ctypes
import os

import pytest
import torch

import sliding_window_gqa_cu_b200 as swa
from sliding_window_gqa_cu_b200 import build
from test_serving_gpu import args_dev, compare, make_case, reference

pytestmark = pytest.mark.gpu
TIMEOUT = -4                   # THD_ERR_TIMEOUT


@pytest.fixture(scope="module")
def debug_lib():
    build.build()
    swa.load_library()
    out = os.path.join(os.path.dirname(swa.library_path()), "libthdattn_debug.so")
    return swa.bind(ctypes.CDLL(build.build(out=out, defines=("THD_DEBUG=1",))))


@pytest.fixture
def lib(debug_lib):
    regular, swa._lib = swa._lib, debug_lib
    yield debug_lib
    torch.cuda.synchronize()
    debug_lib.thd_attn_shared_prefix_set_status(0)
    swa._lib = regular


@pytest.fixture(scope="module")
def case():
    # one that the prefix kernel takes part in, one without
    return [make_case(41, P=900, lens=[300, 20, 77] * 6, n_q=1, Hq=16, Hkv=2, D=128, block=16),
            make_case(42, P=40, lens=[50, 3], n_q=1, Hq=8, Hkv=2, D=64, block=16)]


def buffers(c):
    T, Hq, D = c["q"].shape
    return dict(out=torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda:0"),
                lse=torch.full((T, Hq), 5.0, device="cuda:0"))


@pytest.mark.parametrize("which", [0, 1])
def test_calls_after_a_stall_write_nothing_and_every_stream_is_told(lib, case, which):
    c = case[which]
    a, want = args_dev(c), reference(c)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:                                       # (reports of earlier tests)
        swa.thd_attn_shared_prefix_get_error(s)
        assert swa.thd_attn_shared_prefix_get_error(s) == 0
    assert lib.thd_attn_shared_prefix_set_status(TIMEOUT) == 0
    res = [buffers(c) for _ in streams]
    torch.cuda.synchronize()
    for s, r in zip(streams, res):
        swa.thd_attn_shared_prefix(**a, **r, stream=s)
    torch.cuda.synchronize()
    for r in res:
        assert (r["out"] == 3).all() and (r["lse"] == 5).all()
    assert swa.thd_attn_shared_prefix_get_error(streams[0]) == TIMEOUT     # read once ...
    assert swa.thd_attn_shared_prefix_get_error(streams[0]) == 0           # ... then cleared
    # the others' rows were left too: they hear of it, once each
    for s in streams[1:]:
        assert swa.thd_attn_shared_prefix_get_error(s) == TIMEOUT
        assert swa.thd_attn_shared_prefix_get_error(s) == 0
    # and the next calls compute
    for s, r in zip(streams, res):
        swa.thd_attn_shared_prefix(**a, **r, stream=s)
        assert swa.thd_attn_shared_prefix_get_error(s) == 0
        compare(r["out"], r["lse"], want, c["q"].shape[2])


def test_a_report_waits_for_calls_on_other_streams(lib, case):
    c = case[0]
    a = args_dev(c)
    late, asking = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (late, asking):
        swa.thd_attn_shared_prefix_get_error(s)
        assert swa.thd_attn_shared_prefix_get_error(s) == 0
    r = buffers(c)
    lib.thd_attn_shared_prefix_set_status(TIMEOUT)
    torch.cuda.synchronize()
    with torch.cuda.stream(late):
        torch.cuda._sleep(50_000_000)                       # (some 25 ms)
    swa.thd_attn_shared_prefix(**a, **r, stream=late)
    # the status is not taken back under a call that has yet to end
    assert swa.thd_attn_shared_prefix_get_error(asking) == TIMEOUT
    assert late.query()
    assert (r["out"] == 3).all() and (r["lse"] == 5).all()
    assert swa.thd_attn_shared_prefix_get_error(late) == TIMEOUT
    assert swa.thd_attn_shared_prefix_get_error(late) == 0 == swa.thd_attn_shared_prefix_get_error(asking)
