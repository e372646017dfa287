"""spec_tree_attention over blocks of unequal sizes: a CTA's next block, or its part of the next sequence after a shared prefix,
has fewer rows than the one before, so that warps that had rows have none.  What they still read of the one must not be written
over by the other's products: every result is the definition's (bounds as in test_gpu_step_attention) and the same bit for
bit from call to call."""
import gc

import pytest
import torch

import context_reference as ref
import test_gpu_step_attention as att

pytestmark = pytest.mark.gpu
BF, F16, i32 = torch.bfloat16, torch.float16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def on_the_device(q, k, v, keys, values, lens, seen, scale):
    """context_reference.attention, a sequence at a time, in 64 bits on the GPU."""
    B, N, H, D = q.shape
    kv, inf = k.shape[2], float("inf")
    out, weight = (torch.zeros((B, N, H, D), dtype=torch.float64) for _ in range(2))
    lse, mass = torch.full((B, N, H), -inf, dtype=torch.float64), torch.zeros((B, N, H), dtype=torch.float64)
    for b in range(B):
        if lens[b] < 0:
            continue
        kk, vv = (torch.cat([x[b].cuda(), y[b].double()]).transpose(0, 1) for x, y in ((keys, k), (values, v)))  # [kv, len + N, D]
        on = torch.cat([torch.ones((N, kk.shape[1] - N), dtype=torch.bool), seen], 1).cuda().view(1, N, 1, -1)
        x = q[b].double().view(N, kv, H // kv, D).permute(1, 0, 2, 3).reshape(kv, -1, D)
        each = lambda y: y.view(kv, N, H // kv, -1).transpose(0, 1).reshape(N, H, -1).cpu()  # noqa: E731
        s = (x @ kk.transpose(1, 2)).view(kv, N, H // kv, -1).masked_fill(~on, -inf) * scale
        m = (x.abs() @ kk.abs().transpose(1, 2)).view(kv, N, H // kv, -1).masked_fill(~on, 0.0) * scale
        empty = ~on.any(-1, keepdim=True)
        p = torch.softmax(s.masked_fill(empty, 0.0), -1).masked_fill(empty, 0.0).view(kv, N * (H // kv), -1)
        out[b], weight[b] = each(p @ vv), each(p @ vv.abs())
        lse[b], mass[b] = each(torch.logsumexp(s, -1))[..., 0], each(m.amax(-1))[..., 0]
    return out, lse, weight, mass


@pytest.fixture(autouse=True)
def quick_definition(monkeypatch):
    monkeypatch.setattr(ref, "attention", on_the_device)


def test_the_definition_on_the_device(monkeypatch):
    s = att.problem(3, 9, 6, 2, 64, 16, [40, -1, 0], BF, False, seed=2, seen=torch.rand((9, 9), generator=torch.Generator().manual_seed(1)) < 0.3)
    args = (s["q"], s["k"], s["v"], s["keys"], s["values"], s["host_lens"], s["seen"], s["scale"])
    got = on_the_device(*args)
    monkeypatch.undo()
    for x, y in zip(got, ref.attention(*args)):
        assert torch.equal(torch.isinf(x), torch.isinf(y)) and torch.allclose(x, y, rtol=1e-12, atol=1e-12)


def same_every_time(s, times=6):
    r = att.call(s)
    assert int(r["status"][0]) == 0
    att.check(r, s)
    live = torch.tensor([x >= 0 for x in s["host_lens"]], device="cuda")
    for _ in range(times):
        t = att.call(s)
        assert int(t["status"][0]) == 0 and torch.equal(t["out"][live], r["out"][live]) and torch.equal(t["lse"][live], r["lse"][live])
    return r


@pytest.mark.parametrize("dtype,q8", [(BF, False), (BF, True), (F16, True)])
@pytest.mark.parametrize("B,N,group,kv,D", [  # (a block's rows)
    (40, 97, 4, 2, 128),   # 196, 192: warps of the second half with rows 3, 2
    (12, 200, 8, 2, 64),   # 232 six times, 208: 4, 3
    (48, 57, 8, 2, 128),   # 232, 224: 4, 3
    (100, 3, 128, 1, 128),  # 256, 128: 4, none
    (100, 5, 64, 2, 64),   # 192, 128: 2, none
    (60, 5, 100, 1, 128),  # 200 twice, 100
    (30, 9, 65, 2, 64),    # 130 four times, 65
    (50, 37, 16, 1, 128),  # 208 twice, 176: 3, 2
    (80, 6, 31, 3, 64),    # 186 (one block), many sequences behind each other
])
def test_unequal_blocks(dtype, q8, B, N, group, kv, D):
    same_every_time(att.problem(B, N, group * kv, kv, D, 32, [(37 * b) % 290 for b in range(B)], dtype, q8, seed=N))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,N,group,kv,D,shared", [
    (48, 9, 4, 2, 128, 600),   # 248 and 240 rows of the prefix, then 36: 4, 4, and one product a tile
    (30, 37, 4, 2, 64, 200),   # the prefix's 252, then 148
    (20, 57, 8, 1, 128, 333),  # 256, then 232 and 224
    (70, 3, 128, 1, 64, 128),  # 256, then 256 and 128
    (40, 5, 100, 1, 128, 500),
    (200, 1, 8, 2, 128, 900),  # one token of many sequences
])
def test_fewer_rows_behind_a_prefix(q8, B, N, group, kv, D, shared):
    same_every_time(att.problem(B, N, group * kv, kv, D, 16, [shared + (29 * b) % 210 for b in range(B)], BF, q8, seed=B, shared=shared))


@pytest.mark.parametrize("seed", range(60))
def test_random_calls(seed):
    """Calls over the range of types, head layouts, lengths, prefixes, masks and strides; some with sequences left out, some
    with a node that is not finite."""
    g = torch.Generator().manual_seed(1000 + seed)
    pick = lambda *x: x[int(torch.randint(0, len(x), (1,), generator=g))]  # noqa: E731
    between = lambda a, b: int(torch.randint(a, b + 1, (1,), generator=g))  # noqa: E731
    along = lambda a, b: int(a * (b / a) ** float(torch.rand(1, generator=g)))  # noqa: E731
    dtype, q8, D, page = pick(BF, F16), pick(False, True), pick(64, 128), pick(16, 32, 64, 128, 256)
    group, kv, N = pick(1, 2, 3, 4, 5, 7, 8, 12, 16, 24, 31, 64, 65, 100, 128), pick(1, 2, 3, 4, 5), along(1, 300)
    shared, top = pick(0, 0, between(1, 700)), along(1, 2500)
    B = max(1, min(along(1, 150), 60000 // (N * group * kv), 60000 // ((shared + top) * kv)))
    lens = [shared + between(0, top) if b == 0 or pick(True, True, True, False) else pick(shared, -1) for b in range(B)]
    seen = pick(None, torch.rand((N, N), generator=g) < 0.4)
    s = att.problem(B, N, group * kv, kv, D, page, lens, dtype, q8, seed=seed, shared=shared, chain=pick(False, True), seen=seen)
    if pick(False, True):  # slices of a fused projection's tokens
        wide = torch.zeros((B, N, (group + 2) * kv, D), dtype=dtype, device="cuda")
        cuts = dict(q=slice(0, group * kv), k=slice(group * kv, (group + 1) * kv), v=slice((group + 1) * kv, (group + 2) * kv))
        for n, cut in cuts.items():
            wide[:, :, cut] = s[n]
            s[n] = wide[:, :, cut]
    r = same_every_time(s, 2)
    b, m = between(0, B - 1), between(0, N - 1)
    if lens[b] < 0:
        return
    t = dict(s, v=s["v"].clone())
    t["v"][b, m, kv - 1, 5] = float("nan")
    got, hit = att.call(t)["out"], s["seen"][:, m].cuda()
    live = torch.tensor([x >= 0 for x in lens], device="cuda").view(B, 1, 1, 1).expand_as(got).clone()
    assert torch.isnan(got[b, hit, -group:, 5]).all()
    live[b, hit, -group:, 5] = False
    assert torch.equal(got[live], r["out"][live])
