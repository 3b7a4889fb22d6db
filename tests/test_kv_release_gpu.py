"""Releases that the table or the free list does not bear out."""
import pytest
import torch

from tests.test_kv_cache_gpu import i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_released_twice(cuda_lib):
    """The second release of a request, its length still given, adds nothing and sets the status; a plan after it takes real pages."""
    bs = cuda_lib
    table, lens, done = i32([[3, 5, -1, -1], [7, 1, 9, -1]]), i32([30, 40]), i32([0, 1])
    free, n = i32([0, 2, 4, 6, 8, 10, -5, -5, -5, -5]), i32([6])
    bs.clear_device_status()
    bs.kv_release(lens, done, table, free, n, 16)
    assert bs.device_status()[0] == bs.BS_OK
    assert free.tolist()[:9] == [0, 2, 4, 6, 8, 10, 7, 1, 9] and n.item() == 9
    bs.kv_release(lens, done, table, free, n, 16)
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()
    assert n.item() == 9 and free.tolist() == [0, 2, 4, 6, 8, 10, 7, 1, 9, -5]
    _, _, slots, left = bs.kv_plan(i32([30, 0]), i32([1, 20]), table, free, n, 16, 21)
    assert bs.device_status()[0] == bs.BS_OK
    assert slots.tolist() == [5 * 16 + 14] + [9 * 16 + i for i in range(16)] + [16 + i for i in range(4)]


@pytest.mark.parametrize("B,width,gap", [(3, 5, 3), (700, 9, 4), (1500, 3, 2)])
def test_missing_entries(cuda_lib, B, width, gap):
    """Tables with entries missing here and there: the others go back, in request order."""
    bs = cuda_lib
    rows = [[b * width + j if (b * width + j) % gap else -1 for j in range(width)] for b in range(B)]
    lens = [(b * 37) % (16 * width + 1) for b in range(B)]
    done = [int(b % 3 != 1) for b in range(B)]
    want, after = [99], [list(r) for r in rows]
    for b in range(B):
        for j in range(-(-lens[b] // 16) if done[b] else 0):
            if rows[b][j] >= 0:
                want.append(rows[b][j])
            after[b][j] = -1
    table, free, n = i32(rows), torch.full((B * width + 1,), -5, dtype=torch.int32, device=DEV), i32([1])
    free[0] = 99
    bs.clear_device_status()
    bs.kv_release(i32(lens), i32(done), table, free, n, 16)
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()
    assert n.item() == len(want) and free.tolist() == want + [-5] * (B * width + 1 - len(want))
    assert table.tolist() == after


def test_no_room(cuda_lib):
    """A free list that is too short takes what it has room for; the other pages stay in the table."""
    bs = cuda_lib
    table, free, n = i32([[3, 5, 6], [7, 1, 9]]), i32([0, 2, -5, -5]), i32([2])
    bs.clear_device_status()
    bs.kv_release(i32([48, 48]), i32([1, 1]), table, free, n, 16)
    assert bs.device_status()[0] == bs.BS_ERR_PAGES
    bs.clear_device_status()
    assert n.item() == 4 and free.tolist() == [0, 2, 3, 5] and table.tolist() == [[-1, -1, 6], [7, 1, 9]]
