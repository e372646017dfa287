"""spec_cache_append and spec_cache_read on the GPU against their definitions in 64 bits."""
import gc

import pytest
import torch

import context_reference as ref
import sampling_online_softmax_gb300 as sv

pytestmark = pytest.mark.gpu
BF, F16, F8, i32, u8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    """What these tests keep cached (gigabytes) goes back to the device."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def make(B, width, kv, D, page, dtype, q8, seed, spare=2):
    g = torch.Generator().manual_seed(seed)
    pages = B * width + spare
    table = torch.randperm(pages, generator=g)[: B * width].view(B, width).to(i32).cuda()
    shape = (pages, kv, page, D)
    c = dict(page_table=table, k_cache=torch.zeros(shape, dtype=F8 if q8 else dtype, device="cuda"),
             v_cache=torch.zeros(shape, dtype=F8 if q8 else dtype, device="cuda"))
    if q8:
        c["k_scale"], c["v_scale"] = torch.zeros(shape[:3], dtype=u8, device="cuda"), torch.zeros(shape[:3], dtype=u8, device="cuda")
    return c, g


def append(c, k, v, start, **kw):
    return sv.spec_cache_append(k, v, c["k_cache"], c["v_cache"], c["page_table"], start, k_scale=c.get("k_scale"), v_scale=c.get("v_scale"), **kw)


def read(c, start, n, **kw):
    return sv.spec_cache_read(c["k_cache"], c["v_cache"], c["page_table"], start, n, k_scale=c.get("k_scale"), v_scale=c.get("v_scale"), **kw)


def cells(c):
    return [t.view(u8).cpu().clone() if t.dtype is F8 else t.cpu().clone() for t in (c[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in c)]


def expected(x, dtype, q8):
    return ref.quantised(x, dtype is F16)[0] if q8 else x.double()


@pytest.mark.parametrize("dtype,q8", [(BF, True), (F16, True), (BF, False), (F16, False)])
@pytest.mark.parametrize("B,N,kv,D,page", [(1, 1, 1, 64, 16), (3, 7, 2, 128, 16), (2, 37, 5, 64, 32), (5, 130, 8, 128, 64), (2, 300, 3, 128, 256)])
def test_rows_come_back_as_the_definition_has_them(dtype, q8, B, N, kv, D, page):
    """Exact: one rounding, to the nearest, and powers of two."""
    width = (N + 40) // page + 1
    c, g = make(B, width, kv, D, page, dtype, q8, 5)
    k = (torch.randn((B, N, kv, D), generator=g) * torch.exp2(torch.randint(-12, 8, (B, N, kv, 1), generator=g).float())).to(dtype)
    v = torch.randn((B, N, kv, D), generator=g).to(dtype)
    v[0, 0, 0] = 0
    start = torch.randint(0, 40, (B,), generator=g).to(i32).cuda()
    r = append(c, k.cuda(), v.cuda(), start)
    got = read(c, start, N, dtype=dtype)
    assert int(r["status"][0]) == 0 and int(got["status"][0]) == 0
    assert torch.equal(got["k"].double().cpu(), expected(k, dtype, q8)) and torch.equal(got["v"].double().cpu(), expected(v, dtype, q8))
    if q8:
        at = (start.long().unsqueeze(1) + torch.arange(N, device="cuda"))
        e = c["k_scale"][c["page_table"].gather(1, at // page).long(), :, at % page].cpu()
        assert torch.equal(e, ref.quantised(k, dtype is F16)[1])


def test_extreme_rows():
    """The largest and least values, ties, rows of one value, fp16's end, and rows with an infinity or a NaN."""
    for dtype in (BF, F16):
        c, _ = make(1, 4, 1, 64, 16, dtype, True, 3)
        x = torch.zeros((1, 12, 1, 64))
        top, least = torch.finfo(dtype).max, 2.0 ** (-133 if dtype is BF else -24)
        x[0, 0, 0, :4] = torch.tensor([top, -top, top / 2, 1.0])
        x[0, 1, 0, :3] = torch.tensor([least, -3 * least, 5 * least])
        x[0, 2, 0, :6] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9])
        x[0, 3, 0, :2] = torch.tensor([450.0, 1.0])
        x[0, 4] = -1.0
        x[0, 5, 0, :2] = torch.tensor([63488.0, 61440.0]) if dtype is F16 else torch.tensor([2.0 ** 120, 2.0 ** 100])
        x = x.to(dtype)
        bad = torch.tensor([float("inf"), float("-inf"), float("nan")]).to(dtype)
        for i in range(3):
            x[0, 9 + i, 0, 5 * i] = bad[i]
        start = torch.tensor([2], dtype=i32, device="cuda")
        append(c, x.cuda(), x.cuda(), start)
        got = read(c, start, 12, dtype=dtype)["k"].double().cpu()
        assert torch.equal(got[:, :9], ref.quantised(x[:, :9], dtype is F16)[0])
        assert torch.isnan(got[0, 9:]).all()


@pytest.mark.parametrize("q8", [True, False])
def test_selected_paths_counts_and_rows_that_stay(q8):
    """As a tree's verify names the rows: -1 behind the path; other slots and outputs stay as they were."""
    B, N, S, kv, D, page = 4, 20, 6, 2, 64, 16
    c, g = make(B, 3, kv, D, page, BF, q8, 9)
    before = cells(c)
    k, v = torch.randn((B, N, kv, D), generator=g).to(BF).cuda(), torch.randn((B, N, kv, D), generator=g).to(BF).cuda()
    path = torch.tensor([[0, 3, 7, -1, -1, -1], [0, 1, 2, 5, 9, 19], [0, -1, -1, -1, -1, -1], [0, 4, 5, 6, -1, -1]], dtype=i32).cuda()
    start = torch.tensor([14, 0, 31, -1], dtype=i32).cuda()
    assert int(append(c, k, v, start, select=path)["status"][0]) == 0
    n = [3, 6, 1, 0]
    out = dict(k=torch.full((B, S, kv, D), 7.0, dtype=BF, device="cuda"), v=torch.full((B, S, kv, D), 7.0, dtype=BF, device="cuda"))
    count = torch.tensor([3, 9, 1, 4], dtype=i32).cuda()
    got = read(c, start, S, count=count, out=out)
    for b in range(B):
        assert torch.equal(got["v"][b, : n[b]].double().cpu(), expected(v[b][path[b, : n[b]].long()].cpu(), BF, q8))
        assert (got["v"][b, n[b]:] == 7.0).all()
    written = torch.zeros((B * 3 + 2, page), dtype=torch.bool)
    for b in range(B):
        for i in range(n[b]):
            pos = int(start[b]) + i
            written[int(c["page_table"][b, pos // page]), pos % page] = True
    for was, now in zip(before, cells(c)):
        same = (was == now).reshape(was.shape[0], kv, page, -1).all(-1).all(1)
        assert (same | written).all()
    # counts: below zero none, above S all
    c2, _ = make(B, 3, kv, D, page, BF, q8, 9)
    append(c2, k, v, torch.zeros(B, dtype=i32).cuda(), count=torch.tensor([-3, 0, 2, 99], dtype=i32).cuda())
    got = read(c2, torch.zeros(B, dtype=i32).cuda(), N)["k"]
    for b, n in enumerate((0, 0, 2, N)):
        assert torch.equal(got[b, :n].double().cpu(), expected(k[b, :n].cpu(), BF, q8)) and (got[b, n:] == 0).all()


def test_bad_places_are_reported_and_left():
    B, N, kv, D, page = 2, 4, 1, 64, 16
    for what, bit in (("page", sv.DEV_BAD_PAGE), ("page_high", sv.DEV_BAD_PAGE), ("position", sv.DEV_BAD_LENGTH), ("far", sv.DEV_BAD_LENGTH), ("select", sv.DEV_BAD_LENGTH)):
        c, g = make(B, 2, kv, D, page, BF, True, 4)
        k = torch.randn((B, N, kv, D), generator=g).to(BF).cuda()
        start = torch.tensor([14, 1], dtype=i32).cuda()
        kw = {}
        if what.startswith("page"):
            c["page_table"][0, 1] = -5 if what == "page" else c["k_cache"].shape[0]
        elif what == "position":
            start[0] = 30
        elif what == "far":
            start[0] = 2 ** 31 - 2
        else:
            kw["select"] = torch.tensor([[0, 1, N, 1 << 30], [0, 1, 2, 3]], dtype=i32).cuda()
        assert int(append(c, k, k, start, **kw)["status"][0]) == bit
        got = read(c, start, N)
        assert int(got["status"][0]) == (0 if what == "select" else bit)
        good = {"page": 2, "page_high": 2, "position": 2, "far": 0, "select": 2}[what]
        assert torch.equal(got["k"][0, :good].double().cpu(), expected(k[0, :good].cpu(), BF, True)) and (got["k"][0, good:] == 0).all()
        assert torch.equal(got["k"][1].double().cpu(), expected(k[1].cpu(), BF, True))


def test_strided_tokens_streams_and_graphs():
    B, N, kv, D, page = 3, 9, 2, 128, 32
    c, g = make(B, 2, kv, D, page, BF, True, 6)
    wide = torch.randn((B, N + 2, 3 * kv, D), generator=g).to(BF).cuda()
    k, v = wide[:, 1:-1, :kv], wide[:, 1:-1, kv:2 * kv]
    start = torch.zeros(B, dtype=i32).cuda()
    side = torch.cuda.Stream()
    append(c, k, v, start, stream=side)
    got = read(c, start, N, stream=side)
    side.synchronize()
    assert torch.equal(got["k"].double().cpu(), expected(k.cpu(), BF, True)) and torch.equal(got["v"].double().cpu(), expected(v.cpu(), BF, True))
    # captured, and replayed on new values
    st, out = torch.zeros(1, dtype=i32).cuda(), dict(k=torch.zeros((B, N, kv, D), dtype=BF).cuda(), v=torch.zeros((B, N, kv, D), dtype=BF).cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append(c, k, v, start, status=st)
        read(c, start, N, out=out, status=st)
    wide.copy_(torch.randn(wide.shape, generator=g))
    start.fill_(20)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["k"].double().cpu(), expected(k.cpu(), BF, True)) and int(st[0]) == 0


def test_places_past_32_bits():
    """A cache of more than 2^32 values: rows at its very end."""
    kv, D, page = 8, 128, 256
    pages = 2 ** 32 // (kv * D * page) + 3
    c = dict(page_table=torch.tensor([[pages - 1, 0], [1, pages - 2]], dtype=i32).cuda())
    for n in ("k", "v"):
        c[n + "_cache"] = torch.empty((pages, kv, page, D), dtype=F8, device="cuda")
        c[n + "_scale"] = torch.empty((pages, kv, page), dtype=u8, device="cuda")
    g = torch.Generator().manual_seed(2)
    k = torch.randn((2, 300, kv, D), generator=g).to(BF)
    start = torch.tensor([200, 3], dtype=i32).cuda()
    append(c, k.cuda(), k.cuda(), start)
    got = read(c, start, 300)
    assert torch.equal(got["k"].double().cpu(), expected(k, BF, True)) and torch.equal(got["v"], got["k"])
    del c, got
    torch.cuda.empty_cache()


def test_a_gradient_through_what_was_overwritten_is_refused():
    c, g = make(1, 1, 1, 64, 16, BF, False, 1)
    x = torch.ones((), device="cuda", requires_grad=True)
    y = (c["k_cache"].float() * x).sum()
    z = (c["k_cache"] * x.to(BF)).sum()  # saves the cache itself
    k = torch.randn((1, 2, 1, 64), generator=g).to(BF).cuda()
    append(c, k, k, torch.zeros(1, dtype=i32).cuda())
    y.backward()
    with pytest.raises(RuntimeError):
        z.backward()


def test_empty_calls():
    c, _ = make(2, 1, 1, 64, 16, BF, True, 1)
    none = torch.zeros((2, 0, 1, 64), dtype=BF, device="cuda")
    append(c, none, none, torch.zeros(2, dtype=i32).cuda())
    assert read(c, torch.zeros(2, dtype=i32).cuda(), 0)["k"].shape == (2, 0, 1, 64)
    e, _ = make(0, 1, 1, 64, 16, BF, True, 1)
    assert read(e, torch.zeros(0, dtype=i32).cuda(), 3)["k"].shape == (0, 3, 1, 64)
