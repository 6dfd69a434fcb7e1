"""Table operators at the largest numbers of pages, and of entries per row, that a call may have."""
import pytest
import torch

from _gpu_util import i32

pytestmark = pytest.mark.gpu


def _outs(dev, width, pages):
    return [torch.full((1, width), -7, dtype=torch.int32, device=dev), i32([0], dev), i32([0], dev),
            torch.full((pages,), -7, dtype=torch.int32, device=dev)]


def test_most_pages(kvq, cuda_dev):
    """Pools of almost 2^31 pages (of 3 bytes): two sequences' worth of counts, all others' carried over."""
    pages = 2 ** 31 - 1 - 2048
    pool = kvq.Pool.empty(4, 1, 2, 1, pages, cuda_dev)
    refs = torch.ones(pages, dtype=torch.int32, device=cuda_dev)
    refs[[3, 70000]] = 0
    refs[-1] = 5
    pool.codes[-1], pool.scales[-1] = 9, 2.0
    outs = _outs(cuda_dev, 8, pages)
    err = i32([0], cuda_dev)
    kvq.kvq_table_update([pool], i32([[pages - 1, pages - 2, 0, 0, 0, 0, 0, 0]], cuda_dev), i32([2], cuda_dev),
                         i32([2], cuda_dev), refs, i32([0], cuda_dev), i32([2], cuda_dev), *outs,
                         kvq.table_workspace(pages, 1, cuda_dev), err)
    assert err.item() == 0 and outs[1].item() == 2 and outs[2].item() == 4
    assert outs[0][0].tolist() == [pages - 1, pages - 2, 3, 70000, -7, -7, -7, -7]
    refs[[3, 70000]] = 1
    assert torch.equal(outs[3], refs)


def test_most_entries(kvq, cuda_dev):
    """A row of 2^31 - 1 entries (of one token each), almost all of them one page's."""
    width = 2 ** 31 - 1
    pool = kvq.Pool.empty(4, 1, 64, 1, 5, cuda_dev)
    pool.codes.copy_(torch.arange(5, dtype=torch.uint8)[:, None, None, None])
    pool.scales.copy_(torch.arange(5)[:, None, None])
    table = torch.zeros((1, width), dtype=torch.int32, device=cuda_dev)
    table[0, -1], table[0, -300] = 4, 2
    refs = i32([width - 2, 0, 1, 0, 1], cuda_dev)
    outs = _outs(cuda_dev, width, 5)
    ws, err = kvq.table_workspace(5, 1, cuda_dev), i32([0], cuda_dev)
    kvq.kvq_table_update([pool], table, i32([width], cuda_dev), i32([width], cuda_dev), refs, i32([0], cuda_dev),
                         i32([0], cuda_dev), *outs, ws, err)
    assert err.item() == 0 and outs[1].item() == width and outs[2].item() == width
    assert torch.equal(outs[0], table) and torch.equal(outs[3], refs)
    live = i32([0], cuda_dev)
    outs[0].fill_(-7)
    kvq.kvq_table_compact([pool], table, i32([width], cuda_dev), refs, outs[0], outs[3], live, ws, err)
    assert err.item() == 0 and live.item() == 3 and outs[3].tolist() == [width - 2, 1, 1, 0, 0]
    table[0, -1] = 1
    assert torch.equal(outs[0], table) and (pool.codes[1] == 4).all() and (pool.scales[1] == 4).all()
