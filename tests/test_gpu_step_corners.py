"""Calls of the attention at the corners of what its documentation allows."""
import pytest
import torch

import sampling_online_softmax_gb300 as sv
import test_gpu_step_attention as att

pytestmark = pytest.mark.gpu
BF, F8, i32, u8 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.uint8


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("width", [0, 3])
def test_a_cache_without_pages(q8, width):
    """Nothing is cached yet, anywhere: the nodes attend to one another alone."""
    s = att.problem(2, 7, 8, 2, 64, 16, [0, 0], BF, q8)
    want = att.call(s)
    shape = (0, 2, 16, 64)
    c = dict(k_cache=torch.zeros(shape, dtype=F8 if q8 else BF, device="cuda"), v_cache=torch.zeros(shape, dtype=F8 if q8 else BF, device="cuda"),
             page_table=torch.full((2, width), -1, dtype=i32, device="cuda"))
    if q8:
        c.update(k_scale=torch.zeros(shape[:3], dtype=u8, device="cuda"), v_scale=torch.zeros(shape[:3], dtype=u8, device="cuda"))
    r = att.call(dict(s, c=c))
    assert int(r["status"][0]) == 0 and torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
    att.check(r, s)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("N,H", [(3, 4), (50, 16)])
def test_sequences_left_out_beside_a_prefix(q8, N, H):
    """Sequence 0 among them: its page table still names the prefix.  All of them: nothing is written."""
    s = att.problem(4, N, H, 2, 64, 16, [-1, 200, -1, 160], BF, q8, seed=5, shared=160)
    out = dict(out=torch.full_like(s["q"], 9.0), lse=torch.full(s["q"].shape[:3], 9.0, device="cuda"))
    r = att.call(s, out=out)
    assert int(r["status"][0]) == 0 and (out["out"][[0, 2]] == 9.0).all() and (out["lse"][[0, 2]] == 9.0).all()
    att.check(r, s)
    for shared in (0, 160):
        none = dict(s, lens=torch.full((4,), -1, dtype=i32, device="cuda"), shared=shared)
        out = dict(out=torch.full_like(s["q"], 9.0), lse=torch.full(s["q"].shape[:3], 9.0, device="cuda"))
        assert int(att.call(none, out=out)["status"][0]) == 0 and (out["out"] == 9.0).all() and (out["lse"] == 9.0).all()


def test_a_bad_page_of_the_prefix_is_reported():
    s = att.problem(3, 5, 4, 2, 64, 16, [100, 90, 200], BF, False, seed=2, shared=64)
    s["c"]["page_table"][0, 1] = s["c"]["k_cache"].shape[0]
    assert int(att.call(s)["status"][0]) == sv.DEV_BAD_PAGE


def test_more_sequences_than_threads():
    s = att.problem(1500, 1, 2, 1, 64, 16, [(7 * b) % 40 - 1 for b in range(1500)], BF, True, seed=6)
    r = att.call(s)
    assert int(r["status"][0]) == 0
    att.check(r, s)
