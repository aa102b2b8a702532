"""Forked sequences read what their parents read, whatever the free pages held."""

import pytest
import torch

from gpu_harness import gpu_or_skip

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rows(plane, row, n):
    """The first n tokens of a sequence in a plane, [n][Hkv][D]; pages that do not exist read as zeros."""
    pages, hkv, page, d = plane.shape
    out = torch.zeros((n, hkv, d), dtype=plane.dtype)
    for t in range(n):
        if 0 <= row[t // page] < pages:
            out[t] = plane[row[t // page], :, t % page]
    return out


@pytest.mark.parametrize("missing", [-1, 999, 2**31 - 1, -(2**31), None])
@pytest.mark.parametrize("hkv,page,d,rest", [(2, 16, 64, 9), (8, 64, 128, 63), (1, 16, 8, 1)])
def test_a_child_of_a_partial_page_that_does_not_exist_reads_zeros(hkv, page, d, rest, missing):
    """The parent's partial page is none of the pool's (or, for comparison, one
    that is): the child gets a fresh page of its own, whose rows read as the
    parent's do and not as the sequence's that had the page before."""
    _, q_ = gpu_or_skip()
    pages, planes, n = 9, 3, 2 * page + rest
    print(f"fork of a missing partial page {missing}: {hkv} {page} {d} {rest}", flush=True)
    g = torch.Generator()
    g.manual_seed(page + rest)
    cache = (torch.randn((planes, pages, hkv, page, d), generator=g) + 3).to(torch.bfloat16)  # no zeros
    partial = 5 if missing is None else missing
    tables = [[2, 7, partial, -1], [-1] * 4, [0, 1, -1, -1]]
    refs = [1, 1, 1, 0, 0, 1, 0, 1, 0]
    dev, t, r, lens = cache.to(DEV), _ints(tables), _ints(refs), _ints([n, 0, page + 1])
    status = q_.tf_kv_fork(dev, r, t, lens, _ints([0]), _ints([1]))
    torch.cuda.synchronize()
    assert status.tolist() == [0] and lens.tolist() == [n, n, page + 1]
    assert t.tolist() == [tables[0], [2, 7, 3, -1], tables[2]]
    assert r.tolist() == [1, 1, 2, 1, 0, 1, 0, 2, 0]
    after = dev.cpu()
    for p in range(planes):
        assert torch.equal(_rows(after[p], t[1].tolist(), n), _rows(cache[p], tables[0], n)), f"plane {p}"
    others = [p for p in range(pages) if p != 3]
    assert torch.equal(after[:, others], cache[:, others]) and torch.equal(after[:, 3, :, rest:], cache[:, 3, :, rest:])


def test_a_page_released_too_often_is_free_to_both_calls():
    """A count below zero: compacting drops the page, so forking may take it."""
    _, q_ = gpu_or_skip()
    print("negative references", flush=True)
    cache = torch.arange(6 * 16 * 8, dtype=torch.int16).view(1, 6, 1, 16, 8)
    start = [[1, -1, 0, 1, -7, 1], [[0, 3, -1], [-1, -1, -1], [5, -1, -1]], [20, 0, 16]]
    dev, r, t, lens = cache.to(DEV).view(torch.float16), *(_ints(x) for x in start)
    status = q_.tf_kv_fork(dev, r, t, lens, _ints([0]), _ints([1]))
    torch.cuda.synchronize()
    assert status.tolist() == [0] and r.tolist() == [2, 1, 0, 1, -7, 1] and t[1].tolist() == [0, 1, -1]
    assert torch.equal(dev[0, 1, :, :4].cpu().view(torch.int16), cache[0, 3, :, :4])
    moved = q_.tf_kv_compact(dev, r, t)
    torch.cuda.synchronize()
    assert moved.tolist() == [0, 1, -1, 3, -1, 2] and r.tolist() == [2, 1, 1, 1, 0, 0]
    assert t.tolist() == [[0, 3, -1], [0, 1, -1], [2, -1, -1]]
    # short of pages by one: the zero and the negative page both count
    r, t, lens = (_ints(x) for x in ([1, -1, 0, 1], [[0, 3], [-1, -1], [-1, -1], [-1, -1]], [20, 0, 0, 0]))
    status = q_.tf_kv_fork(dev[:, :4].contiguous(), r, t, lens, _ints([0, 0, 0]), _ints([1, 2, 3]))
    torch.cuda.synchronize()
    assert status.tolist() == [1]
