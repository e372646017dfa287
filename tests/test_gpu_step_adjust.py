"""spec_adjust_logits on the GPU against its definition in 64 bits.

A value passes through at most five roundings to fp32 (bias sums, bias, repetition, frequency's product and difference,
presence) and one to the logits' type, each off by half a step of what it rounds: the bound below counts 2^-24 of the
largest magnitude on the way for each of M + 6, and half a step of the type of the result."""
import gc
import math

import pytest
import torch

import context_reference as ref
import sampling_online_softmax_gb300 as sv

pytestmark = pytest.mark.gpu
i32, f32, BF = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    """What these tests keep cached (gigabytes) goes back to the device."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def make(B, N, V, dtype, L=30, M=5, allowed=True, nodes=True, chain=False, seed=1, spread=6.0):
    g = torch.Generator().manual_seed(seed)
    _, seen = ref.tree(N, seed, chain)
    some = lambda *s: (V * torch.rand(s, generator=g) ** 3).long().clamp(max=V - 1).to(i32)  # noqa: E731
    c = dict(x=(torch.randn((B, N, V), generator=g) * spread).to(dtype), seen=seen, tokens=some(B, L), total=torch.randint(0, L + 1, (B,), generator=g).to(i32),
             nodes=some(B, N) if nodes else None, rep=torch.rand(B, generator=g) + 0.6, freq=torch.rand(B, generator=g) - 0.3, pres=torch.rand(B, generator=g) - 0.3,
             bias_ids=some(B, M) if M else None, bias=torch.randn((B, M), generator=g) if M else None, allowed=None)
    c["prompt"] = (c["total"].float() * torch.rand(B, generator=g)).to(i32)
    if L:
        c["tokens"][torch.rand((B, L), generator=g) < 0.1] = -1
    if nodes:
        c["nodes"][torch.rand((B, N), generator=g) < 0.1] = -1
    if M:
        c["bias_ids"][torch.rand((B, M), generator=g) < 0.2] = -1
    if allowed:
        w = torch.randint(-(1 << 31), 1 << 31, (B, N, (V + 31) // 32), generator=g)
        kind = torch.randint(0, 4, (B, N, 1), generator=g)
        c["allowed"] = torch.where(kind == 0, 0, torch.where(kind == 1, -1, torch.where(kind == 2, w, w | (w >> 3) | (w >> 7)))).to(i32)
    return c


def gpu(t):
    return None if t is None else t.cuda()


def call(c, x=None, **kw):
    x = c["x"].cuda() if x is None else x
    return sv.spec_adjust_logits(x, tokens=gpu(c["tokens"]), prompt_len=gpu(c["prompt"]), total_len=gpu(c["total"]), node_tokens=gpu(c["nodes"]),
                                 mask=gpu(ref.tree_words(c["seen"])), repetition=gpu(c["rep"]), frequency=gpu(c["freq"]), presence=gpu(c["pres"]),
                                 bias_ids=gpu(c["bias_ids"]), bias=gpu(c["bias"]), allowed=gpu(c["allowed"]), **kw)


def expect(c):
    return ref.adjusted(c["x"], c["seen"], c["tokens"], c["prompt"], c["total"], c["nodes"], c["rep"], c["freq"], c["pres"], c["bias_ids"], c["bias"], c["allowed"])


def check(got, want, c, dtype):
    got, x = got.double().cpu(), c["x"].double()
    M = 0 if c["bias"] is None else c["bias"].shape[1]
    add = 0.0 if c["bias"] is None else float(c["bias"].abs().sum(1).max())
    scale = (x.abs() + add) * 2.0 + (0 if c["tokens"] is None else c["tokens"].shape[1] + c["x"].shape[1]) + 1.0  # penalties here: factors to 1.7, |f|, |p| < 1
    tol = scale * (M + 6) * 2.0 ** -24 + want.abs() * (0 if dtype is f32 else 2.0 ** -8)
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine])
    assert torch.isfinite(got[fine]).all() and ((got - want).abs()[fine] <= tol[fine]).all()
    untouched = (want == x) & fine  # what no step changes comes back bit for bit
    assert torch.equal(got[untouched], x[untouched])


@pytest.mark.parametrize("dtype", [f32, BF])
@pytest.mark.parametrize("B,N,V,L,M,allowed", [
    (1, 1, 1, 3, 1, True), (2, 3, 31, 9, 2, True), (1, 1, 33, 0, 0, True), (3, 5, 1000, 40, 0, False), (2, 9, 4099, 500, 20, True), (4, 1, 5003, 2100, 7, False),
    (1, 33, 8192, 300, 40, True), (2, 64, 8193, 64, 1, True), (1, 2, 50257, 10000, 300, True), (2, 70, 1023, 10, 1024, True)])
def test_against_the_definition(dtype, B, N, V, L, M, allowed):
    c = make(B, N, V, dtype, L, M, allowed)
    r = call(c)
    assert int(r["status"][0]) == 0
    check(r["logits"], expect(c), c, dtype)


@pytest.mark.parametrize("dtype", [f32, BF])
@pytest.mark.parametrize("V", [8, 4095, 20001])
def test_in_place_and_unaligned(dtype, V):
    """In place, and at every place on the 16-byte grid, logits and output alike and not."""
    c = make(2, 4, V, dtype, 60, 6, True)
    want = expect(c)
    x = c["x"].cuda()
    r = call(c, x, out=dict(logits=x))
    assert r["logits"].data_ptr() == x.data_ptr()
    check(x, want, c, dtype)
    n, each = c["x"].numel(), 16 // c["x"].element_size()
    for a, b in ((1, 1), (0, 1), (each - 1, each // 2), (3, 3)):
        src, dst = torch.full((n + 16,), 3.0, dtype=dtype).cuda(), torch.full((n + 16,), 5.0, dtype=dtype).cuda()
        src[a:a + n] = c["x"].cuda().flatten()
        call(c, src[a:a + n].view(c["x"].shape), out=dict(logits=dst[b:b + n].view(c["x"].shape)))
        check(dst[b:b + n].view(c["x"].shape), want, c, dtype)
        assert (dst[:b] == 5.0).all() and (dst[b + n:] == 5.0).all() and torch.equal(src[a:a + n], c["x"].cuda().flatten())
        call(c, src[a:a + n].view(c["x"].shape), out=dict(logits=src[a:a + n].view(c["x"].shape)))
        check(src[a:a + n].view(c["x"].shape), want, c, dtype)
        assert (src[:a] == 3.0).all() and (src[a + n:] == 3.0).all()


def test_each_argument_alone():
    for dtype in (f32, BF):
        c = make(3, 6, 2000, dtype, 100, 9, True, seed=5)
        nothing = dict(c, tokens=None, prompt=None, total=None, nodes=None, rep=None, freq=None, pres=None, bias_ids=None, bias=None, allowed=None)
        assert torch.equal(call(nothing)["logits"].cpu(), c["x"])
        for keep in (("tokens", "rep"), ("tokens", "prompt", "rep"), ("tokens", "total", "freq"), ("tokens", "pres"), ("nodes", "freq"), ("nodes", "rep"),
                     ("bias_ids", "bias"), ("allowed",), ("nodes", "tokens", "total", "prompt"), ("freq",)):
            d = dict(nothing, **{n: c[n] for n in keep})
            check(call(d)["logits"], expect(d), d, dtype)
        chain = make(3, 6, 2000, dtype, 100, 9, True, chain=True, seed=5)
        got = sv.spec_adjust_logits(chain["x"].cuda(), node_tokens=gpu(chain["nodes"]), presence=gpu(chain["pres"]))["logits"]  # no mask: a chain
        d = dict(nothing, x=chain["x"], seen=chain["seen"], nodes=chain["nodes"], pres=chain["pres"])
        check(got, expect(d), d, dtype)


@pytest.mark.parametrize("dtype", [f32, BF])
def test_special_values(dtype):
    """-inf and the type's lowest value under every step, NaN and +inf in masked places, rows with nothing allowed."""
    c = make(2, 3, 600, dtype, 80, 6, True, seed=8)
    c["x"][:, :, ::7] = -math.inf
    c["x"][:, :, 1::7] = torch.finfo(dtype).min
    c["x"][:, :, 2::7] = -0.0
    c["allowed"][0, 0] = 0
    off = ((c["allowed"].long().unsqueeze(-1) >> torch.arange(32)) & 1).reshape(2, 3, -1)[..., :600] == 0
    c["x"][off & (torch.arange(600) % 3 == 0)] = math.nan
    c["x"][off & (torch.arange(600) % 3 == 1)] = math.inf
    c["rep"][:] = 1.5
    want = expect(c)
    limit = torch.finfo(dtype).max
    got = call(c)["logits"].double().cpu()
    over = want < -1.01 * limit  # well past the type's lowest value: -inf
    assert torch.isneginf(got[over]).all() and torch.isneginf(got[torch.isneginf(want)]).all()
    low = ~over & (want < -1e30)
    assert torch.allclose(got[low], want[low], rtol=2.0 ** -7)
    rest = ~over & ~low
    assert torch.isfinite(got[rest]).all() and ((got - want).abs()[rest] <= 1e-3 + want.abs()[rest] * 2.0 ** -8).all()
    # an allowed NaN stays one, touched or not
    d = make(1, 1, 64, dtype, 10, 0, False, seed=3)
    d["x"][0, 0, :] = math.nan
    assert torch.isnan(call(d)["logits"]).all()


def test_bad_data_is_reported():
    c = make(3, 4, 500, f32, 20, 4, False, seed=2)
    for name, value, bit in (("tokens", 500, sv.DEV_BAD_TOKEN), ("tokens", -2, sv.DEV_BAD_TOKEN), ("nodes", 1 << 30, sv.DEV_BAD_TOKEN), ("nodes", -7, sv.DEV_BAD_TOKEN),
                             ("bias_ids", 500, sv.DEV_BAD_TOKEN), ("bias_ids", -2, sv.DEV_BAD_TOKEN)):
        d = dict(c, total=torch.full((3,), 20, dtype=i32))
        d[name] = c[name].clone()
        d[name][1, 2] = value
        r = call(d)
        assert int(r["status"][0]) == bit
        check(r["logits"], expect(d), d, f32)  # (the reference leaves such a token out)
    for name, value, as_if in (("total", 21, 20), ("total", -1, 0), ("prompt", -4, 0)):
        d, e = dict(c), dict(c)
        d[name], e[name] = c[name].clone(), c[name].clone()
        d[name][2], e[name][2] = value, as_if
        if name == "total":
            d["prompt"] = e["prompt"] = torch.zeros(3, dtype=i32)
        r = call(d)
        assert int(r["status"][0]) == sv.DEV_BAD_LENGTH
        check(r["logits"], expect(e), e, f32)
    for name, value in (("rep", 0.0), ("rep", -1.0), ("rep", math.inf), ("rep", math.nan), ("freq", math.inf), ("pres", math.nan)):
        d, e = dict(c), dict(c)
        d[name], e[name] = c[name].clone(), c[name].clone()
        d[name][0], e[name][0] = value, 1.0 if name == "rep" else 0.0
        r = call(d)
        assert int(r["status"][0]) == sv.DEV_BAD_PARAM
        check(r["logits"], expect(e), e, f32)


def test_many_equal_tokens_and_biases():
    """One token over and over, in the history, on the path and among the biases (summed in slot order)."""
    B, N, V, L, M = 2, 40, 300, 5000, 1000
    g = torch.Generator().manual_seed(4)
    c = make(B, N, V, f32, L, M, False, chain=True)
    c["tokens"][:], c["total"][:], c["prompt"][:] = 17, L, 100
    c["nodes"][:], c["bias_ids"][:] = 17, 17
    c["bias"] = torch.randn((B, M), generator=g)
    r1, r2 = call(c)["logits"], call(c)["logits"]
    assert torch.equal(r1, r2)
    s = torch.zeros(B)
    for i in range(M):
        s += c["bias"][:, i]
    x = c["x"][:, :, 17] + s.view(B, 1)
    rep = c["rep"].view(B, 1)
    x = torch.where(x > 0, x / rep, x * rep)
    count = (4900 + torch.arange(N)).float()
    x = x - c["freq"].view(B, 1) * count
    x = x - c["pres"].view(B, 1)
    assert torch.equal(r1[:, :, 17].cpu(), x)


def test_streams_graphs_and_repeats():
    c = make(4, 9, 9000, BF, 200, 8, True, seed=12)
    want = expect(c)
    side = torch.cuda.Stream()
    r = call(c, stream=side)
    side.synchronize()
    check(r["logits"], want, c, BF)
    x, out, st = c["x"].cuda(), dict(logits=torch.empty_like(c["x"].cuda())), torch.zeros(1, dtype=i32).cuda()
    fixed = {n: gpu(c[n]) for n in ("tokens", "prompt", "total", "nodes", "rep", "freq", "pres", "bias_ids", "bias", "allowed")}
    mask = gpu(ref.tree_words(c["seen"]))
    go = lambda: sv.spec_adjust_logits(x, tokens=fixed["tokens"], prompt_len=fixed["prompt"], total_len=fixed["total"], node_tokens=fixed["nodes"], mask=mask,  # noqa: E731
                                       repetition=fixed["rep"], frequency=fixed["freq"], presence=fixed["pres"], bias_ids=fixed["bias_ids"], bias=fixed["bias"],
                                       allowed=fixed["allowed"], out=out, status=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    d = make(4, 9, 9000, BF, 200, 8, True, seed=13)
    x.copy_(d["x"])
    for n, t in fixed.items():
        t.copy_(d[n])
    mask.copy_(ref.tree_words(d["seen"]))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check(out["logits"], expect(d), d, BF)


def test_empty_batch():
    x = torch.zeros((0, 3, 50), device="cuda")
    assert sv.spec_adjust_logits(x)["logits"].shape == (0, 3, 50)
