"""spec_tree_attention on the GPU against its definition in 64 bits.

Bounds, with u the half step of the type (2^-8 in bf16, 2^-11 in fp16):
  a score is a sum of D exact products in fp32, times scale and log2 e in fp32, so off by at most
      d = (D + 4) 2^-24 sum |q k| scale + 2^-22 |s|, which moves a weight by a factor of 1 +- 2 d, say;
  a weight is an exponential good to 2^-21, rounded to the type (u), the sums are fp32 sums of at most `keys` terms;
  so |out - exact| <= (u + 4 d + 2^-20 + keys 2^-24) sum p |v| + u |out|, the last for the result's rounding,
  and |lse - exact| <= 2 d + 2^-20 + keys 2^-24 + |lse| 2^-22."""
import gc
import math
import os
import subprocess
import sys

import pytest
import torch

import context_reference as ref
import sampling_online_softmax_gb300 as sv
from test_gpu_step_cache import append, make

pytestmark = pytest.mark.gpu
BF, F16, F8, i32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int32


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    """What these tests keep cached (gigabytes) goes back to the device."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def problem(B, N, H, kv, D, page, lens, dtype, q8, seed=1, shared=0, chain=False, spread=1.5, seen=None, width=None):
    """A cache filled through spec_cache_append, and what it holds, per sequence, in 64 bits."""
    lens = list(lens)
    width = (max(max(lens), 1) + page - 1) // page if width is None else width
    c, g = make(B, width, kv, D, page, dtype, q8, seed)
    full = max(max(lens), 1)
    k = (torch.randn((B, full, kv, D), generator=g) * torch.exp2(torch.randint(-2, 2, (B, full, kv, 1), generator=g).float())).to(dtype)
    v = (torch.randn((B, full, kv, D), generator=g) + 0.3).to(dtype)
    if shared:
        k[:, :shared], v[:, :shared] = k[:1, :shared], v[:1, :shared]
        c["page_table"][:, : shared // page] = c["page_table"][:1, : shared // page].clone()
    count = torch.tensor([max(x, 0) for x in lens], dtype=i32).cuda()
    zero = torch.zeros(B, dtype=i32).cuda()
    append(c, k.cuda(), v.cuda(), zero, count=count)
    held = [ref.quantised(x, dtype is F16)[0] if q8 else x.double() for x in (k, v)]
    _, tree = ref.tree(N, seed, chain)
    seen = tree if seen is None else seen
    s = dict(c=c, q=(torch.randn((B, N, H, D), generator=g) * spread).to(dtype).cuda(), k=torch.randn((B, N, kv, D), generator=g).to(dtype).cuda(),
             v=torch.randn((B, N, kv, D), generator=g).to(dtype).cuda(), lens=torch.tensor(lens, dtype=i32).cuda(), host_lens=lens, seen=seen, shared=shared,
             scale=D ** -0.5, keys=[held[0][b, : max(x, 0)] for b, x in enumerate(lens)], values=[held[1][b, : max(x, 0)] for b, x in enumerate(lens)])
    return s


def call(s, mask=True, **kw):
    c = s["c"]
    m = ref.tree_words(s["seen"]).cuda() if mask else None
    return sv.spec_tree_attention(s["q"], s["k"], s["v"], c["k_cache"], c["v_cache"], c["page_table"], s["lens"], mask=m, shared_len=s["shared"],
                                  scale=s["scale"], k_scale=c.get("k_scale"), v_scale=c.get("v_scale"), lse=True, **kw)


def check(r, s, live=None):
    out, lse, weight, mass = ref.attention(s["q"], s["k"], s["v"], s["keys"], s["values"], s["host_lens"], s["seen"], s["scale"])
    D, u = s["q"].shape[3], 2.0 ** -8 if s["q"].dtype is BF else 2.0 ** -11
    count = max(max(s["host_lens"]), 0) + s["q"].shape[1]
    d = (D + 4) * 2.0 ** -24 * mass + 2.0 ** -22 * mass
    got, got_lse = r["out"].double().cpu(), r["lse"].double().cpu()
    live = torch.tensor([x >= 0 for x in s["host_lens"]]) if live is None else live
    off = (got - out).abs()[live]
    tol = (u + 4 * d.unsqueeze(-1) + 2.0 ** -20 + count * 2.0 ** -24) * weight + u * out.abs() + 2.0 ** -40
    assert torch.isfinite(got[live]).all()
    worst = (off / tol[live]).max() if off.numel() else 0.0
    assert worst <= 1.0, "out is %.3g times the bound off" % worst
    empty = torch.isneginf(lse)
    assert torch.equal(torch.isneginf(got_lse[live]), empty[live]) and (got[live][empty[live]] == 0).all()
    fine = ~empty[live]
    tol = 2 * d + 2.0 ** -20 + count * 2.0 ** -24 + torch.where(empty, 0.0, lse.abs()) * 2.0 ** -22
    assert ((got_lse - lse).abs()[live][fine] <= tol[live][fine]).all()


SHAPES = [  # B, N, heads, kv heads, D, page, lengths
    (1, 1, 1, 1, 64, 16, [0]),
    (1, 1, 8, 8, 128, 16, [1]),
    (2, 1, 8, 2, 128, 64, [127, 128]),
    (3, 5, 4, 1, 64, 32, [129, 0, 300]),
    (4, 3, 14, 2, 64, 16, [17, 255, 256, 257]),
    (2, 33, 12, 4, 128, 64, [500, 31]),
    (1, 64, 8, 2, 128, 128, [1000]),
    (2, 64, 10, 2, 128, 256, [640, 77]),
    (2, 128, 3, 1, 64, 64, [200, 130]),
    (1, 129, 2, 1, 128, 16, [383]),
    (1, 200, 16, 2, 64, 32, [150]),
    (9, 2, 6, 3, 128, 32, [0, 1, 2, 64, 65, 191, 192, 193, 640]),
]


@pytest.mark.parametrize("dtype,q8", [(BF, False), (BF, True), (F16, False), (F16, True)])
@pytest.mark.parametrize("B,N,H,kv,D,page,lens", SHAPES)
def test_against_the_definition(dtype, q8, B, N, H, kv, D, page, lens):
    s = problem(B, N, H, kv, D, page, lens, dtype, q8)
    r = call(s)
    assert int(r["status"][0]) == 0
    check(r, s)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,N,H,kv,D,page,shared,lens", [
    (3, 1, 4, 2, 128, 64, 128, [128, 200, 512]), (2, 5, 8, 2, 64, 16, 16, [16, 400]), (4, 9, 6, 2, 128, 32, 300, [300, 301, 700, 431]),
    (5, 64, 4, 1, 128, 64, 640, [640, 650, 700, 900, 641]), (40, 7, 4, 2, 64, 16, 1000, [1000 + 3 * i for i in range(40)]), (1, 3, 2, 1, 64, 16, 100, [150])])
def test_a_shared_prefix(q8, B, N, H, kv, D, page, shared, lens):
    s = problem(B, N, H, kv, D, page, lens, BF, q8, shared=shared, seed=3)
    r = call(s)
    assert int(r["status"][0]) == 0
    check(r, s)


def test_many_sequences_and_long_contexts():
    """More work than CTAs, and contexts that many CTAs share."""
    def check_all(s):
        r = call(s)
        assert int(r["status"][0]) == 0
        check(r, s)
    check_all(problem(120, 2, 4, 2, 64, 16, [(37 * b) % 300 for b in range(120)], BF, True, seed=4))
    check_all(problem(1, 2, 2, 1, 128, 128, [40000], BF, False, seed=5))
    check_all(problem(2, 3, 8, 4, 64, 64, [9000, 5], F16, True, seed=6))
    check_all(problem(2, 80, 8, 2, 128, 64, [3000, 2900], BF, True, seed=7))


@pytest.mark.parametrize("q8", [False, True])
def test_long_contexts_behind_each_other(q8):
    """Many rounds of the ring of tiles between the ones that plain loads bring (the ends of contexts, the nodes), and many of
    the latter between the others."""
    for s in (problem(16, 64, 8, 2, 128, 32, [1500 - 60 * b for b in range(16)], BF, q8, seed=11),
              problem(40, 3, 8, 4, 128, 64, [(2000 * b) % 1777 + 1 for b in range(40)], BF, q8, seed=12),
              problem(12, 40, 8, 2, 64, 16, [1300 - 100 * b for b in range(12)], F16, q8, seed=13),
              problem(3, 1024, 1, 1, 128, 64, [900, 1100, 300], BF, q8, seed=14)):
        r = call(s)
        assert int(r["status"][0]) == 0
        check(r, s)


def test_masks():
    """Rows that see no node, none that sees itself, all nodes; a chain without a mask; rows that see nothing at all."""
    N = 40
    g = torch.Generator().manual_seed(3)
    seen = torch.rand((N, N), generator=g) < 0.3
    seen[5] = False
    seen[6] = True
    seen[7] = False
    seen[7, 39] = True
    for lens in ([70, 0], [0, 128]):
        s = problem(2, N, 4, 2, 64, 16, lens, BF, False, seen=seen)
        check(call(s), s)
    s = problem(2, N, 4, 2, 128, 16, [90, 3], BF, True, chain=True)
    check(call(s, mask=False), s)
    r, t = call(s, mask=False), call(s)
    assert torch.equal(r["out"], t["out"]) and torch.equal(r["lse"], t["lse"])


def test_what_a_row_does_not_see_has_no_part_in_it():
    """NaN and infinities in the cache behind a sequence's end, in other sequences' pages, and in nodes off a row's path."""
    for dtype, q8 in ((BF, False), (BF, True), (F16, False)):
        s = problem(2, 40, 4, 2, 64, 32, [75, 130], dtype, q8, seed=9)
        c, before = s["c"], call(s)
        for n in ("k", "v"):
            t, used = c[n + "_cache"], torch.zeros(c["k_cache"].shape[0], 32, dtype=torch.bool)
            for b, length in enumerate(s["host_lens"]):
                for i in range(length):
                    used[int(c["page_table"][b, i // 32]), i % 32] = True
            junk = ~used.cuda().view(-1, 1, 32).expand(t.shape[:3])
            if q8:
                t.view(torch.uint8)[junk] = 0x7F
                c[n + "_scale"][junk] = 255
            else:
                t[junk] = math.nan if n == "k" else math.inf
        again = call(s)
        assert torch.equal(before["out"], again["out"]) and torch.equal(before["lse"], again["lse"])
        check(again, s)
        # node 11 of sequence 0: only the rows that see it become non-finite
        for value in (math.nan, math.inf):
            t = dict(s, k=s["k"].clone(), v=s["v"].clone())
            t["v"][0, 11, 1, 3] = value
            r = call(t)
            hit = s["seen"][:, 11]
            assert not torch.isfinite(r["out"][0, hit.cuda(), 2:, 3]).any()
            ok = torch.ones_like(r["out"], dtype=torch.bool)
            ok[0, hit.cuda(), 2:, 3] = False
            assert torch.equal(r["out"][ok], before["out"][ok]) and torch.equal(r["lse"], before["lse"])
        t = dict(s, k=s["k"].clone())
        t["k"][0, 11, 0, 5] = math.nan
        r = call(t)
        assert torch.isnan(r["out"][0, hit.cuda(), :2]).all() and torch.isnan(r["lse"][0, hit.cuda(), :2]).all()
        ok = torch.ones_like(r["out"], dtype=torch.bool)
        ok[0, hit.cuda(), :2] = False
        assert torch.equal(r["out"][ok], before["out"][ok])
        # a query that is not finite: its own row alone
        t = dict(s, q=s["q"].clone())
        t["q"][1, 3, 2, 0] = math.nan
        r = call(t)
        assert torch.isnan(r["out"][1, 3, 2]).all()
        ok = torch.ones(r["lse"].shape, dtype=torch.bool, device="cuda")
        ok[1, 3, 2] = False
        assert torch.equal(r["out"][ok], before["out"][ok])


def test_large_scores():
    """Scores of hundreds, rising and falling along the context, so that the maximum moves on late."""
    for q8 in (False, True):
        s = problem(2, 3, 2, 1, 64, 16, [700, 699], BF, q8, seed=2, spread=40.0)
        check(call(s), s)
        s["scale"] = 3.0
        check(call(s), s)
    s = problem(1, 2, 2, 2, 64, 16, [600], BF, False, seed=2)
    s["scale"] = 1e-6
    check(call(s), s)


def test_sequences_left_out_and_bad_data():
    s = problem(4, 3, 4, 2, 64, 16, [100, -1, 33, -7], BF, False, seed=2)
    out = dict(out=torch.full_like(s["q"], 9.0), lse=torch.full(s["q"].shape[:3], 9.0, device="cuda"))
    r = call(s, out=out)
    assert int(r["status"][0]) == 0 and (out["out"][[1, 3]] == 9.0).all() and (out["lse"][[1, 3]] == 9.0).all()
    check(r, s)
    # a page outside the cache, a length past the table: reported, and the other sequences are right
    others = torch.tensor([False, True])
    for what, bit in (("page", sv.DEV_BAD_PAGE), ("page_low", sv.DEV_BAD_PAGE), ("length", sv.DEV_BAD_LENGTH)):
        s = problem(2, 3, 4, 2, 64, 16, [100, 90], BF, what != "page", seed=2)
        if what == "length":
            s["lens"][0] = 1 << 30
        else:
            s["c"]["page_table"][0, 3] = -1 if what == "page_low" else s["c"]["k_cache"].shape[0]
        r = call(s)
        assert int(r["status"][0]) == bit
        check(r, s, live=others)
    s = problem(2, 3, 4, 2, 64, 16, [100, 90], BF, False, seed=2, shared=64)
    s["lens"][0] = 63
    r = call(s)
    assert int(r["status"][0]) == sv.DEV_BAD_LENGTH
    check(r, s, live=others)


def test_strides_streams_workspaces_and_graphs():
    s = problem(3, 7, 8, 2, 128, 32, [300, 41, 129], BF, True, seed=8)
    want = call(s)
    wide = torch.zeros((3, 9, 12, 128), dtype=BF, device="cuda")  # a fused projection's queries, keys and values
    wide[:, 1:8, :8], wide[:, 1:8, 8:10], wide[:, 1:8, 10:] = s["q"], s["k"], s["v"]
    t = dict(s, q=wide[:, 1:8, :8], k=wide[:, 1:8, 8:10], v=wide[:, 1:8, 10:])
    side = torch.cuda.Stream()
    r = call(t, stream=side)
    side.synchronize()
    assert torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
    need = sv.spec_workspace_bytes_attention(3, 7, 8, 2, 128, 0)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # whatever it holds
    for _ in range(2):
        assert torch.equal(call(s, workspace=ws)["out"], want["out"])
    with pytest.raises(sv.SpecError):
        call(s, workspace=ws[:-16])
    # two captured graphs, replayed in turn on new values
    mask = ref.tree_words(s["seen"]).cuda()
    c, st = s["c"], torch.zeros(1, dtype=i32).cuda()
    go = lambda o: sv.spec_tree_attention(s["q"], s["k"], s["v"], c["k_cache"], c["v_cache"], c["page_table"], s["lens"], mask=mask, k_scale=c["k_scale"],  # noqa: E731
                                          v_scale=c["v_scale"], lse=True, out=o, status=st)
    outs = [dict(out=torch.zeros_like(s["q"]), lse=torch.zeros((3, 7, 8), device="cuda")) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, o in zip(graphs, outs):
        with torch.cuda.graph(graph):
            go(o)
    s["q"].copy_(s["q"].flip(1))
    s["lens"].copy_(torch.tensor([17, 41, 100], dtype=i32))
    want = go(dict(out=torch.zeros_like(s["q"]), lse=torch.zeros((3, 7, 8), device="cuda")))
    for graph in (graphs[0], graphs[1], graphs[0]):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    assert int(st[0]) == 0


def test_two_calls_at_once():
    a, b = (problem(2, 5, 8, 2, 128, 64, [900, 700], BF, False, seed=x) for x in (1, 2))
    want = [call(a)["out"].clone(), call(b)["out"].clone()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[call(p, stream=x)["out"] for p, x in zip((a, b), streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for one in got:
        assert torch.equal(one[0], want[0]) and torch.equal(one[1], want[1])


def test_pages_past_32_bits():
    kv, D, page = 8, 128, 128
    pages = 2 ** 32 // (kv * D * page) + 5
    table = torch.tensor([[pages - 1, 2, pages - 3]], dtype=i32).cuda()
    for q8 in (False, True):
        s = problem(1, 2, 8, kv, D, page, [300], BF, q8, seed=4)
        small = s["c"]
        big = dict(page_table=table)
        for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
            if n in small:
                big[n] = torch.zeros((pages, *small[n].shape[1:]), dtype=small[n].dtype, device="cuda")
                big[n].view(torch.uint8)[table[0].long()] = small[n].view(torch.uint8)[small["page_table"][0].long()]
        t = dict(s, c=big)
        want = call(s)["out"]
        assert torch.equal(call(t)["out"], want)
        check(call(t), t)
        del big, t
        torch.cuda.empty_cache()


def test_a_round_of_the_operators_together():
    """Mask, attention, adjusted logits, the tree's verify, and the accepted path into the cache: what the next step then
    attends to is what a plain chain of those tokens would have written."""
    B, N, H, kv, D, V, page = 3, 12, 8, 2, 64, 500, 16
    parents, seen = ref.tree(N, 21)
    s = problem(B, N, H, kv, D, page, [40, 77, 5], BF, True, seed=21, seen=seen, width=8)
    m = sv.spec_tree_mask(parents.cuda())
    c = s["c"]
    cache = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    r = sv.spec_tree_attention(s["q"], s["k"], s["v"], c["k_cache"], c["v_cache"], c["page_table"], s["lens"], mask=m["mask"], scale=s["scale"], lse=True, **cache)
    check(r, s)
    g = torch.Generator().manual_seed(5)
    head = (torch.randn((H * D, V), generator=g)).to(BF).cuda()
    logits = torch.matmul(r["out"].view(B * N, H * D), head).view(B, N, V).contiguous()
    nodes = torch.randint(0, V, (B, N), generator=g).to(i32)
    history = torch.randint(0, V, (B, 30), generator=g).to(i32)
    allowed = torch.randint(-(1 << 31), 1 << 31, (B, N, (V + 31) // 32), generator=g).to(i32)
    rep, freq = torch.full((B,), 1.3), torch.full((B,), 0.4)
    adj = sv.spec_adjust_logits(logits, tokens=history.cuda(), node_tokens=nodes.cuda(), mask=m["mask"], repetition=rep.cuda(), frequency=freq.cuda(), allowed=allowed.cuda())
    want = ref.adjusted(logits, seen, history, None, None, nodes, rep, freq, None, None, None, allowed)
    fine = torch.isfinite(want)
    got = adj["logits"].double().cpu()
    assert torch.equal(torch.isneginf(got), ~fine) and ((got - want).abs()[fine] <= want.abs()[fine] * 2.0 ** -8 + 2.0 ** -10).all()
    # candidates that agree with the target along one path
    best = adj["logits"].float().argmax(2).to(i32).cpu()
    for b in range(B):
        for n in range(1, N):
            nodes[b, n] = best[b, parents[n]] if n % 2 else nodes[b, n]
    depth = int(m["depth"].max())
    t = sv.spec_verify_tree(adj["logits"], parents.cuda(), nodes.cuda(), depth)
    path, n_acc = t["path_nodes"], t["path_len"].cpu() + 1
    assert int(t["status"][0]) == 0 and int(n_acc.max()) > 1
    assert int(sv.spec_cache_append(s["k"], s["v"], c["k_cache"], c["v_cache"], c["page_table"], s["lens"], select=path, **cache)["status"][0]) == 0
    new = s["lens"].cpu() + n_acc
    for name, keys in (("k", s["keys"]), ("v", s["values"])):
        for b in range(B):
            rows = ref.quantised(s[name][b][path[b, : n_acc[b]].long()].cpu())[0]
            keys[b] = torch.cat([keys[b], rows])
    s["host_lens"], s["lens"] = new.tolist(), new.to(i32).cuda()
    check(sv.spec_tree_attention(s["q"], s["k"], s["v"], c["k_cache"], c["v_cache"], c["page_table"], s["lens"], mask=m["mask"], scale=s["scale"], lse=True, **cache), s)


def test_empty_batch():
    s = problem(1, 3, 4, 2, 64, 16, [5], BF, False)
    c = s["c"]
    r = sv.spec_tree_attention(s["q"][:0], s["k"][:0], s["v"][:0], c["k_cache"], c["v_cache"], c["page_table"][:0], s["lens"][:0])
    assert r["out"].shape == (0, 3, 4, 64)


def test_an_8_bit_cache_with_powers_that_fp16_lacks():
    """Rows as bf16 ones leave them: powers of two below 2^-24 and above 2^15, whose products with the 8-bit values fp16 holds or rounds."""
    lens, page, D = [200, 37], 16, 64
    s = problem(2, 3, 4, 2, D, page, lens, F16, True, seed=31)
    c, g = s["c"], torch.Generator().manual_seed(31)
    for n, top in (("k", 16), ("v", 22)):
        shape = c[n + "_cache"].shape
        raw = torch.randint(0, 127, shape, generator=g)
        raw[:, 1] = torch.randint(0, 8, shape, generator=g)[:, 1]  # multiples of 2^-9
        raw = raw + 128 * torch.randint(0, 2, shape, generator=g)
        e = torch.randint(-45, -19, shape[:3], generator=g)
        e[:, 1] = torch.randint(10, top + 1, shape[:3], generator=g)[:, 1]
        c[n + "_cache"].view(torch.uint8).copy_(raw.to(torch.uint8))
        c[n + "_scale"].copy_((e + 127).to(torch.uint8))
        x = torch.ldexp(raw.to(torch.uint8).view(F8).double(), e.unsqueeze(-1).double()).to(F16).double()
        assert torch.isfinite(x).all()
        at = [torch.arange(length) for length in lens]
        table = c["page_table"].cpu().long()
        s["keys" if n == "k" else "values"] = [x[table[b, i // page], :, i % page] for b, i in enumerate(at)]
    s["v"].zero_()  # (the nodes' values would hide the context's)
    r = call(s)
    assert int(r["status"][0]) == 0
    out, lse, weight, mass = ref.attention(s["q"], s["k"], s["v"], s["keys"], s["values"], lens, s["seen"], s["scale"])
    d, count = ((D + 4) * 2.0 ** -24 + 2.0 ** -22) * mass, 203
    tol = (2.0 ** -11 + 4 * d.unsqueeze(-1) + 2.0 ** -20 + count * 2.0 ** -24) * weight + 2.0 ** -11 * out.abs() + 2.0 ** -25  # (half of fp16's least step)
    assert ((r["out"].double().cpu() - out).abs() <= tol).all()
    assert ((r["lse"].double().cpu() - lse).abs() <= 2 * d + 2.0 ** -20 + count * 2.0 ** -24 + lse.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("q8", [False, True])
def test_tokens_before_sequences(q8):
    """q, k, v laid out [N, B, heads, head_dim]: a sequence's stride is smaller than a token's."""
    s = problem(3, 6, 8, 2, 64, 32, [90, 0, 200], BF, q8, seed=15)
    want = call(s)
    t = dict(s, **{n: s[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v")})
    r = call(t)
    assert torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
    t = dict(problem(3, 6, 8, 2, 64, 32, [90, 70, 200], BF, q8, seed=15, shared=64))
    t["q"] = t["q"].transpose(0, 1).contiguous().transpose(0, 1)  # the batch's rows are then not on one axis
    with pytest.raises(sv.SpecError):
        call(t)


FIRST_CALL_CAPTURED = """
import torch, sampling_online_softmax_gb300 as sv
torch.manual_seed(0)
d, BF, F8, i32 = "cuda", torch.bfloat16, torch.float8_e4m3fn, torch.int32
q, k, v = (torch.randn((2, 3, h, 64), device=d).to(BF) for h in (4, 2, 2))
kc, vc = (torch.zeros((8, 2, 16, 64), device=d).to(F8) for _ in range(2))
ks, vs = (torch.zeros((8, 2, 16), dtype=torch.uint8, device=d) for _ in range(2))
table, start = torch.arange(8, dtype=i32, device=d).view(2, 4), torch.tensor([5, 20], dtype=i32, device=d)
hist, logits = torch.randint(0, 100, (2, 9), device=d).to(i32), torch.randn((2, 3, 100), device=d)
rep = torch.full((2,), 1.5, device=d)
def step():
    a = sv.spec_cache_append(k, v, kc, vc, table, start, k_scale=ks, v_scale=vs)
    r = sv.spec_cache_read(kc, vc, table, start, 3, k_scale=ks, v_scale=vs)
    t = sv.spec_tree_attention(q, k, v, kc, vc, table, start, k_scale=ks, v_scale=vs, lse=True)
    j = sv.spec_adjust_logits(logits, tokens=hist, repetition=rep)
    return [r["k"], r["v"], t["out"], t["lse"], j["logits"]], [a["status"], r["status"], t["status"], j["status"]]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got, status = step()
for _ in range(3):
    graph.replay()
torch.cuda.synchronize()
want, _ = step()
assert all(torch.equal(x, y) for x, y in zip(got, want)) and not any(int(s[0]) for s in status)
print("captured")
"""


def test_a_first_call_that_is_captured():
    """A process whose first calls are captured into a graph: kernels, their attributes and the driver's encoder are all first met there."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
