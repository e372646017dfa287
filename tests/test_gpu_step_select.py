"""spec_cache_append's select: what it holds behind a sequence's count, or for a sequence left out, is not looked at."""
import pytest
import torch

import sampling_online_softmax_gb300 as sv
from test_gpu_step_cache import append, cells, expected, make, read

pytestmark = pytest.mark.gpu
BF, i32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("q8", [True, False])
def test_entries_behind_the_count_are_not_looked_at(q8):
    B, N, kv, D, page = 4, 5, 2, 64, 16
    c, g = make(B, 2, kv, D, page, BF, q8, 3)
    k = torch.randn((B, N, kv, D), generator=g).to(BF).cuda()
    select = torch.tensor([[4, 0, 1 << 30, N], [1, 2, 3, N], [N, 1 << 30, N, 2 ** 31 - 1], [N + 1, N, 1, 0]], dtype=i32).cuda()
    start, count = torch.tensor([3, 0, 7, -1], dtype=i32).cuda(), torch.tensor([2, 3, 0, 4], dtype=i32).cuda()
    assert int(append(c, k, k, start, select=select, count=count)["status"][0]) == 0
    got = read(c, start, 4)["k"].double().cpu()
    for b, rows in enumerate(([4, 0], [1, 2, 3], [], [])):
        assert torch.equal(got[b, : len(rows)], expected(k[b, rows].cpu(), BF, q8)) and (got[b, len(rows):] == 0).all()
    # one that counts is reported, its row is not written, and the others are
    before = cells(c)
    assert int(append(c, k, k, start, select=select, count=torch.tensor([0, 0, 1, 0], dtype=i32).cuda())["status"][0]) == sv.DEV_BAD_LENGTH
    assert all(torch.equal(x, y) for x, y in zip(before, cells(c)))
