"""The attention's bounded waits, run out: the call ends by itself with its status bit, its copies and products awaited and its tensor
memory given back, and the calls after it are right.

As for the verify's waits, a copy of the library is built with SPEC_TEST_HOOKS and a short limit: one CTA then leaves out
arrivals that others wait for (a worker's, a softmax warp's, the announcement of its pieces), which nothing else makes."""
import ctypes

import pytest
import torch

import context_reference as ref
import sampling_online_softmax_gb300 as sv
import test_gpu_step_attention as att
from test_timeout_recovery import hooks  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
P = ctypes.c_void_p


def attend(lib, s):
    c, (B, N, H, D) = s["c"], s["q"].shape
    kv = s["k"].shape[2]
    pages, _, page, _ = c["k_cache"].shape
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    code = sv._CODES[s["q"].dtype]
    cache = sv._Cache(ptr(c["k_cache"]), ptr(c["v_cache"]), ptr(c.get("k_scale")), ptr(c.get("v_scale")), ptr(c["page_table"]),
                      sv.SPEC_E4M3 if "k_scale" in c else code, pages, page, kv, D, c["page_table"].shape[1])
    out, lse, status = torch.zeros_like(s["q"]), torch.zeros((B, N, H), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    room = sv.spec_workspace_bytes_attention(B, N, H, kv, D, s["shared"])
    ws, mask = torch.empty(room, dtype=torch.uint8, device="cuda"), ref.tree_words(s["seen"]).cuda()
    f = lib.spec_tree_attention
    f.argtypes, f.restype = sv.load_library().spec_tree_attention.argtypes, ctypes.c_int
    st = f(ptr(s["q"]), ptr(s["k"]), ptr(s["v"]), code, B, N, H, None, ctypes.addressof(cache), ptr(s["lens"]), s["shared"], ptr(mask), s["scale"], ptr(out), ptr(lse),
           ptr(status), ptr(ws), room, torch.cuda.current_stream().cuda_stream)
    assert st == 0, lib.spec_last_error()
    torch.cuda.synchronize()
    return dict(out=out, lse=lse, status=status)


@pytest.mark.parametrize("what", [0, 1, 2])
@pytest.mark.parametrize("dtype,q8,B,N,H,kv,D,shared", [
    (BF, False, 4, 40, 8, 2, 128, 0), (BF, True, 4, 40, 8, 2, 128, 0), (F16, True, 5, 3, 8, 4, 64, 0), (BF, False, 5, 3, 8, 4, 64, 0), (BF, True, 6, 50, 4, 1, 128, 512)])
def test_a_wait_that_runs_out(hooks, what, dtype, q8, B, N, H, kv, D, shared):  # noqa: F811
    s = att.problem(B, N, H, kv, D, 64, [6000 + 700 * b for b in range(B)], dtype, q8, seed=17, shared=shared)
    want = att.call(s)
    att.check(want, s)
    for cta in (0, 75):
        hooks.spec_test_set_withhold(4 * cta + what)
        try:
            r = attend(hooks, s)
        finally:
            hooks.spec_test_set_withhold(-1)
        assert int(r["status"][0]) == sv.DEV_TIMEOUT
        r = attend(hooks, s)  # tensor memory and barriers are as a first call finds them
        assert int(r["status"][0]) == 0 and torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
    again = att.call(s)
    assert torch.equal(again["out"], want["out"]) and int(again["status"][0]) == 0
