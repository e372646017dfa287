"""Plain decoding (one token of each sequence) with queries, keys and values that are slices of a fused projection."""
import pytest
import torch

import test_gpu_step_attention as att
from test_gpu_step_cache import append, cells, make

pytestmark = pytest.mark.gpu
BF, F16, i32 = torch.bfloat16, torch.float16, torch.int32


def fused(*parts):
    """The same tensors as slices of the heads of one."""
    wide, cuts, at = torch.cat(parts, 2).contiguous(), [], 0
    for x in parts:
        cuts.append(wide[:, :, at:at + x.shape[2]])
        at += x.shape[2]
    return cuts


@pytest.mark.parametrize("dtype,q8", [(BF, False), (BF, True), (F16, False)])
@pytest.mark.parametrize("B,kv,group,D,shared", [(5, 2, 4, 128, 100), (40, 1, 8, 64, 128), (1, 2, 3, 128, 64), (7, 4, 1, 64, 0), (3, 1, 128, 128, 33)])
def test_one_token_of_a_fused_projection(dtype, q8, B, kv, group, D, shared):
    s = att.problem(B, 1, group * kv, kv, D, 16, [shared + 31 * b for b in range(B)], dtype, q8, seed=7, shared=shared)
    want = att.call(s)
    att.check(want, s)
    q, k, v = fused(s["q"], s["k"], s["v"])
    for first in (False, True):  # (the token axis' own stride: the batch's, or anything)
        if first:
            q, k, v = (x.as_strided(x.shape, (x.stride(0), 8, D, 1)) for x in (q, k, v))
        r = att.call(dict(s, q=q, k=k, v=v))
        assert int(r["status"][0]) == 0 and torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])


def test_one_token_of_a_fused_projection_into_the_cache():
    for q8 in (False, True):
        (c, g), (d, _) = (make(6, 2, 2, 64, 16, BF, q8, 4) for _ in range(2))
        k, v = (torch.randn((6, 1, 2, 64), generator=g).to(BF).cuda() for _ in range(2))
        start = torch.tensor([0, 5, 15, 16, 31, -1], dtype=i32).cuda()
        _, k2, v2 = fused(torch.zeros((6, 1, 8, 64), dtype=BF, device="cuda"), k, v)
        assert int(append(c, k, v, start)["status"][0]) == 0 and int(append(d, k2, v2, start)["status"][0]) == 0
        assert all(torch.equal(x, y) for x, y in zip(cells(c), cells(d)))
