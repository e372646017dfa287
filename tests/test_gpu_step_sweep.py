"""spec_cache_append, spec_cache_read and spec_adjust_logits over seeded random calls, against their definitions in 64 bits."""
import gc

import pytest
import torch

import context_reference as ref
import sampling_online_softmax_gb300 as sv
import test_gpu_step_adjust as adj
from test_gpu_step_cache import append, cells, expected, make, read

pytestmark = pytest.mark.gpu
BF, F16, i32, f32 = torch.bfloat16, torch.float16, torch.int32, torch.float32


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def dice(seed):
    g = torch.Generator().manual_seed(seed)
    pick = lambda *x: x[int(torch.randint(0, len(x), (1,), generator=g))]  # noqa: E731
    between = lambda a, b: int(torch.randint(a, b + 1, (1,), generator=g))  # noqa: E731
    along = lambda a, b: int(a * (b / a) ** float(torch.rand(1, generator=g)))  # noqa: E731
    return g, pick, between, along


@pytest.mark.parametrize("seed", range(40))
def test_random_appends_and_reads(seed):
    """Rows picked from strided tokens, under starts, counts and entries that leave some out: what is written is the definition's, and
    nothing else is."""
    g, pick, between, along = dice(2000 + seed)
    dtype, q8, D, page, kv = pick(BF, F16), pick(False, True), pick(64, 128), pick(16, 32, 64, 128, 256), pick(1, 2, 3, 5, 8, 17, 40)
    N = along(1, 200)
    B = max(1, min(along(1, 40), 40000 // (N * kv)))
    S = pick(N, between(1, N))
    width = (S + 60) // page + 1
    c, _ = make(B, width, kv, D, page, dtype, q8, seed)
    wide = (torch.randn((B, N, 2 * kv + 1, D), generator=g) * torch.exp2(torch.randint(-9, 6, (B, N, 2 * kv + 1, 1), generator=g).float())).to(dtype)
    on = wide.cuda()
    k, v = on[:, :, :kv], on[:, :, kv:2 * kv]
    start = torch.randint(-8, 50, (B,), generator=g).to(i32)
    count = torch.randint(-2, S + 3, (B,), generator=g).to(i32) if pick(False, True) else None
    select = torch.randint(-2, N, (B, S), generator=g).to(i32) if S != N or pick(False, True) else None
    before = cells(c)
    assert int(append(c, k, v, start.cuda(), count=None if count is None else count.cuda(), select=None if select is None else select.cuda())["status"][0]) == 0
    went = torch.zeros((B * width + 2, page), dtype=torch.bool)
    got = read(c, start.cuda(), S, dtype=dtype)
    assert int(got["status"][0]) == 0
    want = {n: torch.zeros((B, S, kv, D), dtype=torch.float64) for n in ("k", "v")}
    full = {n: expected(x.cpu(), dtype, q8) for n, x in (("k", k), ("v", v))}
    for b in range(B):
        for i in range(S):
            token = i if select is None else int(select[b, i])
            if int(start[b]) < 0 or token < 0 or (count is not None and i >= int(count[b])):
                continue
            pos = int(start[b]) + i
            went[int(c["page_table"][b, pos // page]), pos % page] = True
            for n in ("k", "v"):
                want[n][b, i] = full[n][b, token]
    for n in ("k", "v"):
        assert torch.equal(got[n].double().cpu(), want[n])
    for was, now in zip(before, cells(c)):
        assert ((was == now).reshape(was.shape[0], kv, page, -1).all(-1).all(1) | went).all()


@pytest.mark.parametrize("seed", range(40))
def test_random_adjustments(seed):
    """Each argument there or not, at every place on the 16-byte grid, in place and not."""
    g, pick, between, along = dice(3000 + seed)
    dtype, N = pick(f32, BF), along(1, 70)
    B, V = along(1, 4), along(1, 20000)
    c = adj.make(B, N, V, dtype, pick(0, along(1, 3000)), pick(0, along(1, 200)), pick(False, True), pick(False, True), pick(False, True), seed)
    for n in ("rep", "freq", "pres", "prompt", "total"):
        if pick(True, False, False):
            c[n] = None
    if pick(True, False, False):
        c["rep"] = None if c["rep"] is None else torch.ones(B)
    want = adj.expect(c)
    n, a, b = c["x"].numel(), between(0, 7), between(0, 7)
    src, dst = (torch.full((n + 16,), x, dtype=dtype, device="cuda") for x in (3.0, 5.0))
    src[a:a + n] = c["x"].cuda().flatten()
    x = src[a:a + n].view(B, N, V)
    out = dst[b:b + n].view(B, N, V)
    r = adj.call(c, x, out=dict(logits=out))
    assert int(r["status"][0]) == 0 and torch.equal(x.cpu(), c["x"])
    adj.check(out, want, c, dtype)
    assert (dst[:b] == 5.0).all() and (dst[b + n:] == 5.0).all()
    kept = out.clone()
    adj.call(c, x, out=dict(logits=x))
    assert torch.equal(x, kept) and (src[:a] == 3.0).all() and (src[a + n:] == 3.0).all()
    assert torch.equal(adj.call(c, out=dict(logits=dst[b:b + n].view(B, N, V)))["logits"], kept)
