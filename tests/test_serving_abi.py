"""Refusals of the serving entry points: they return before any CUDA call, so
they need no GPU; the wrappers' own checks raise before the library is called."""
import ctypes

import pytest
import torch

import sliding_window_gqa_cu_b200 as swa
from sliding_window_gqa_cu_b200 import build

PTR = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return swa.load_library()


def _tables(lib, seq=PTR, new=PTR, n_req=2, block=16, table=PTR, max_blocks=4, free=PTR, cap=8, count=PTR, first=None,
            rows=4, seq_out=PTR, count_out=PTR, cu=PTR, slots=PTR, positions=PTR, refused=PTR):
    return lib.thd_kv_block_tables(seq, new, n_req, block, table, max_blocks, free, cap, count, first, rows, seq_out,
                                   count_out, cu, slots, positions, refused, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=-1), -1), (dict(block=0), -1), (dict(max_blocks=0), -1), (dict(rows=-1), -1), (dict(cap=-1), -1),
    (dict(cap=1 << 31), -1), (dict(rows=1 << 31), -1), (dict(block=1 << 16, max_blocks=1 << 15), -1),
    (dict(seq=0), -1), (dict(new=0), -1), (dict(table=0), -1), (dict(free=0), -1), (dict(count=0), -1),
    (dict(seq_out=0), -1), (dict(count_out=0), -1), (dict(cu=0), -1), (dict(slots=0), -1), (dict(positions=0), -1),
    (dict(refused=0), -1), (dict(seq=PTR + 2), -1), (dict(slots=PTR + 1), -1), (dict(first=PTR + 2), -1),
    (dict(n_req=8193), -2), (dict(n_req=0, seq=0), 0),
])
def test_block_tables_refuses(lib, kw, code):
    assert _tables(lib, **kw) == code


def _write(lib, k=PTR, v=PTR, k_row=256, v_row=256, slots=PTR, rows=4, Hkv=2, D=128, kc=PTR, vc=PTR, nb=4, block=16,
           sb=16 * 256, st=256, sh=128):
    return lib.thd_kv_write(k, v, k_row, v_row, slots, rows, Hkv, D, kc, vc, nb, block, sb, st, sh, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(Hkv=0), -1), (dict(nb=-1), -1), (dict(block=0), -1), (dict(nb=1 << 28), -1),
    (dict(k=0), -1), (dict(v=0), -1), (dict(slots=0), -1), (dict(kc=0), -1), (dict(vc=0), -1),
    (dict(k=PTR + 8), -1), (dict(kc=PTR + 8), -1), (dict(slots=PTR + 2), -1), (dict(k_row=248), -1),
    (dict(v_row=260), -1), (dict(st=120), -1), (dict(sh=64), -1), (dict(sb=-8), -1), (dict(sb=4100), -1),
    (dict(D=96), -2), (dict(D=32), -2), (dict(rows=0, k=0), 0), (dict(nb=0, kc=0), 0),
])
def test_kv_write_refuses(lib, kw, code):
    assert _write(lib, **kw) == code


def _attend(lib, q=PTR, kc=PTR, vc=PTR, nb=8, block=16, sb=16 * 256, st=256, sh=128, pt=None, n_pt=0, plen=None,
            tables=PTR, max_blocks=4, lens=PTR, n_req=2, n_q=1, Hq=8, Hkv=2, D=128, window=0, scale=0.1, sinks=None,
            out=PTR, lse=None, ws=PTR, ws_bytes=1 << 40):
    return lib.thd_attn_shared_prefix(q, kc, vc, nb, block, sb, st, sh, pt, n_pt, plen, tables, max_blocks, lens, n_req,
                                      n_q, Hq, Hkv, D, window, scale, sinks, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=-1), -1), (dict(n_q=0), -1), (dict(Hq=7), -1), (dict(Hkv=0), -1), (dict(window=-1), -1),
    (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(nb=-1), -1),
    (dict(max_blocks=-1), -1), (dict(n_pt=-1), -1), (dict(nb=1 << 28), -1), (dict(max_blocks=1 << 27), -1),
    (dict(pt=PTR, n_pt=1 << 26, plen=PTR, max_blocks=1 << 26), -1), (dict(pt=PTR, n_pt=4), -1), (dict(plen=PTR), -1),
    (dict(q=0), -1), (dict(kc=0), -1), (dict(vc=0), -1), (dict(tables=0), -1), (dict(lens=0), -1), (dict(out=0), -1),
    (dict(ws=0), -1), (dict(ws_bytes=0), -1), (dict(q=PTR + 8), -1), (dict(kc=PTR + 2), -1), (dict(lse=PTR + 2), -1),
    (dict(sinks=PTR + 1), -1), (dict(ws=PTR + 4), -1), (dict(st=64), -1), (dict(sh=132), -1),
    (dict(D=96), -2), (dict(block=8), -2), (dict(block=48), -2), (dict(block=512, sb=512 * 256), -2),
    (dict(Hq=258, Hkv=2), -2), (dict(n_req=4097), -2), (dict(n_req=300, n_q=512), -2), (dict(n_req=0, q=0), 0),
])
def test_attend_refuses(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_workspace_covers_the_documented_range(lib):
    f = swa.thd_attn_shared_prefix_workspace_bytes
    assert f(0, 1, 8, 2, 128) == 0
    assert 0 < f(1, 1, 8, 2, 128) <= f(64, 1, 8, 2, 128) <= f(64, 4, 8, 2, 128)


def test_wrappers_refuse_host_tensors_and_wrong_types():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    c = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        swa.thd_kv_block_tables(i, i, torch.zeros((2, 4), dtype=torch.int32), i, i[:1], 16, 2)
    with pytest.raises(ValueError):
        swa.thd_kv_write(x, x, i, c, c)
    with pytest.raises(ValueError):
        swa.thd_attn_shared_prefix(x, c, c, torch.zeros((2, 4), dtype=torch.int32), i)


def test_cache_layouts():
    dev = torch.device("cpu")
    strides = swa._cache_strides
    c = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)
    assert strides(c, c, dev) == (4, 16, 2, 128, 4096, 256, 128)
    h = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16).transpose(1, 2)
    assert strides(h, h, dev) == (4, 16, 2, 128, 4096, 128, 2048)
    both = torch.zeros((4, 2, 16, 2, 128), dtype=torch.bfloat16)          # k and v interleaved page by page
    assert strides(both[:, 0], both[:, 1], dev) == (4, 16, 2, 128, 8192, 256, 128)
    one = torch.zeros((4, 16, 1, 128), dtype=torch.bfloat16)
    assert strides(one, one.as_strided(one.shape, (2048, 128, 1, 1)), dev) == (4, 16, 1, 128, 2048, 128, 128)
    with pytest.raises(ValueError):
        strides(c, h, dev)                                                # different strides
    with pytest.raises(ValueError):
        strides(c[..., ::2], c[..., ::2], dev)                            # head_dim not dense
    with pytest.raises(ValueError):
        strides(c[:1].expand(4, 16, 2, 128), c[:1].expand(4, 16, 2, 128), dev)  # overlapping blocks
    with pytest.raises(ValueError):
        strides(c, c.float(), dev)


def test_attend_refuses_places_beyond_32_bits(lib):
    # blocks whose distance shares no more than 8 elements with the heads': more
    # places than the tensor map counts (33 rows, so the prefix goes through it)
    kw = dict(nb=1 << 20, sb=(1 << 20) + 8, pt=PTR, n_pt=4, plen=PTR, n_req=33, Hq=2, Hkv=2)
    assert _attend(lib, **kw) == -2


def test_workspace_of_unsupported_sizes(lib):
    f = swa.thd_attn_shared_prefix_workspace_bytes
    assert f(4097, 1, 8, 2, 128) == 0 and f(1 << 20, 1 << 20, 8, 2, 128) == 0 and f(2, 1, 258, 2, 128) == 0
    assert f(2, 1, 8, 2, 96) == 0 and f(2, 1, 7, 2, 128) == 0
    assert f(4096, 1, 8, 8, 64) > 0 and f(1, 4096 * 128, 8, 8, 64) > 0


def test_status_is_read_on_the_streams_device(monkeypatch):
    # a stream of the second device, the first one current: that device's word
    class Library:
        def thd_attn_shared_prefix_get_error(self, handle):
            seen.append((current[-1], handle.value))
            return -4

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *_):
            current.pop()

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0x1234

    seen, current = [], [0]
    monkeypatch.setattr(swa, "load_library", Library)
    monkeypatch.setattr(torch.cuda, "device", Device)
    assert swa.thd_attn_shared_prefix_get_error(Stream()) == -4
    assert seen == [(1, 0x1234)] and current == [0]
