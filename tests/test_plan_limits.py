"""Page plans at the ends of what their sizes allow."""
import ctypes

import pytest
import torch

import bit_level_weight_gb300 as cas

GOOD = 0x10000  # a 16-byte aligned address that no refused call touches
MOST = 2 ** 31 - 1


def built():
    from bit_level_weight_gb300 import build
    build.build()
    return cas.lib()


@pytest.mark.parametrize("batch", [MOST, MOST - 1023])
def test_batches_whose_rounds_pass_32_bits_are_refused(batch):
    """Kernels go over the sequences in rounds of up to 1024, counted in 32 bits."""
    L = built()
    pool = cas.cas_page_pool(batch, 3, 16, 8, GOOD, GOOD, GOOD, GOOD)
    assert L.cas_paged_plan(ctypes.byref(pool), None, GOOD, 4, GOOD, None, None, None, GOOD, 1 << 62, None) == -1
    b = ctypes.byref(cas.cas_paged_batch(batch, 2, 3, 0, GOOD, GOOD, GOOD))
    kv = ctypes.byref(cas.cas_paged4_kv(2, 16, 8, GOOD, 16 * 288, 288, 144))
    assert L.cas_paged4_append(kv, b, GOOD, 0, 4, None, None, 1e-6, 1e4, GOOD, None) == -1
    assert L.cas_paged4_read(kv, b, GOOD, GOOD, None) == -1
    assert L.cas_paged4_attn(kv, b, GOOD, 4, GOOD, GOOD, 1 << 62, None) == -1
    kv = ctypes.byref(cas.cas_paged_kv(2, 16, 8, GOOD, GOOD, 16 * 256, 256, 128))
    assert L.cas_paged_append(kv, b, GOOD, 0, 4, None, None, 1e-6, 1e4, GOOD, None) == -1
    assert L.cas_paged_attn(kv, b, GOOD, 4, GOOD, GOOD, 1 << 62, None) == -1


def pool_on_gpu():
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32([[1, 0, 0], [0, 0, 0]]), i32([9, 0]), i32([2, 3, 0, 0]), i32([2]), i32([30, 5])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2049, MOST - 255, MOST - 254, MOST])
def test_plan_without_places_of_rows(rows):
    """As many rows as an int holds, positions and slots not wanted: tables, lengths and bounds are made."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L = built()
    t, h, f, n, add = pool_on_gpu()
    start, granted = torch.full((3,), -9, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(L.cas_paged_plan_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    pool = cas.cas_page_pool(2, 3, 16, 4, t.data_ptr(), h.data_ptr(), f.data_ptr(), n.data_ptr())
    st = torch.cuda.current_stream().cuda_stream
    assert L.cas_paged_plan(ctypes.byref(pool), None, add.data_ptr(), rows, start.data_ptr(), granted.data_ptr(), None, None,
                            ws.data_ptr(), ws.numel(), st) == 0
    torch.cuda.synchronize()
    # 9 + 30 tokens need two pages more, the five of the other one that is not there
    assert granted.tolist() == [30, 0] and start.tolist() == [0, 30, 30] and h.tolist() == [39, 0]
    assert t.tolist() == [[1, 3, 2], [0, 0, 0]] and n.item() == 0


@pytest.mark.gpu
def test_plan_with_places_of_as_many_rows_as_an_int_holds():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    built()
    t, h, f, n, add = pool_on_gpu()
    start, pos, slots, granted = cas.paged_plan(t, h, f, n, 16, add, MOST)
    assert start.tolist() == [0, 30, 30] and granted.tolist() == [30, 0]
    assert pos[:30].tolist() == list(range(9, 39))
    assert slots[:30].tolist() == [([1, 3, 2][p // 16]) * 16 + p % 16 for p in range(9, 39)]
    assert pos.shape == slots.shape == (MOST,) and (pos[30:] == -1).all() and (slots[30:] == -1).all()
    del pos, slots
    torch.cuda.empty_cache()
