"""Filtered sampling and the largest logits on the GPU, against 64 bits.

Tokens, ids and values must be equal: the inputs' draws lie further than
2^-36 from every border of the distribution (asserted; the kernel's weights
are right to about 2^-38), so no tolerance is needed.
"""
import numpy as np
import pytest
import torch

import rows_reference as ref
import sampling_online_softmax_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    """What these tests keep cached (gigabytes) goes back to the device."""
    yield
    torch.cuda.empty_cache()

NEAR = 2.0 ** -36


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def rows(B, V, dtype, sigma, seed, masked=0.0, offset=0):
    """Logits whose first element lies `offset` elements into an allocation."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, V), generator=g) * sigma
    if masked:
        x[torch.rand((B, V), generator=g) < masked] = float("-inf")
        x[:, V // 2] = 0.5
    flat = torch.zeros(B * V + offset, dtype=dtype, device=DEV)
    flat[offset:] = x.to(dtype).reshape(-1).to(DEV)
    return flat[offset:].view(B, V)


def params(B, seed, T=(1.0,), k=(0,), p=(1.0,), mp=(0.0,)):
    r = np.random.RandomState(seed)
    pick = lambda v, dt: torch.tensor([v[r.randint(len(v))] for _ in range(B)], dtype=dt, device=DEV)  # noqa: E731
    return dict(temperature=pick(T, torch.float32), top_k=pick(k, torch.int32), top_p=pick(p, torch.float32),
                min_p=pick(mp, torch.float32))


def check_sample(x, u, q, status=0, **kw):
    r = sv.spec_sample_filtered(x, u, q["temperature"], top_k=q.get("top_k"), top_p=q.get("top_p"), min_p=q.get("min_p"), **kw)
    torch.cuda.synchronize()
    got = r["tokens"].cpu().numpy()
    assert int(r["status"][0]) == status
    at = lambda n, b, none: none if q.get(n) is None else float(q[n][b])  # noqa: E731
    for b in range(x.shape[0]):
        tok, far = ref.sample_filtered(host(x[b]), float(u[b]), at("temperature", b, 1.0), int(at("top_k", b, 0)), at("top_p", b, 1.0),
                                       at("min_p", b, 0.0))
        assert far > NEAR, "the input lies on a border: row %d" % b
        assert got[b] == tok, (b, got[b], tok, {n: at(n, b, None) for n in q})
    return got


MIXED = dict(T=(0.0, 0.3, 0.7, 1.0, 2.0), k=(0, 1, 2, 50, 300, 5000), p=(1.0, 0.999, 0.9, 0.5, 0.0), mp=(0.0, 0.0, 0.02, 0.5, 1.0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 257, 1000, 5003, 32000, 50257, 131072])
def test_mixed_filters(V, dtype):
    B = 24 if V < 60000 else 8
    x = rows(B, V, dtype, 3.0, V, masked=0.3 if V % 2 else 0.0, offset=V % 5)
    u = torch.rand(B, generator=torch.Generator().manual_seed(V + 1)).to(DEV)
    check_sample(x, u, params(B, V, **MIXED))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name,q", [
    ("none", {}), ("k", dict(k=(40,))), ("k_large", dict(k=(3000,))), ("p", dict(p=(0.9,))), ("p_flat", dict(T=(3.0,), p=(0.97,))),
    ("mp", dict(mp=(0.05,))), ("mp_flat", dict(T=(3.0,), mp=(0.01,))), ("all", dict(T=(0.8,), k=(64,), p=(0.9,), mp=(0.02,))),
    ("k_p_large", dict(T=(2.0,), k=(4000,), p=(0.8,))), ("cold", dict(T=(1e-6, 1e-3, 0.01))), ("hot", dict(T=(50.0, 1e6), p=(0.5, 1.0)))])
def test_each_filter(name, q, dtype):
    B, V = 20, 20011
    x = rows(B, V, dtype, 2.5, 77)
    u = torch.rand(B, generator=torch.Generator().manual_seed(5)).to(DEV)
    check_sample(x, u, params(B, 3, **q))


def test_no_filter_arrays():
    x = rows(9, 4001, torch.float32, 3.0, 2)
    u = torch.rand(9, generator=torch.Generator().manual_seed(6)).to(DEV)
    check_sample(x, u, dict(temperature=torch.full((9,), 0.9, device=DEV)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties(dtype):
    """Equal logits in their thousands: the cuts fall inside a tie, which the lower indices win."""
    V = 30000
    x = torch.zeros((6, V), dtype=dtype, device=DEV)
    x[1] = -3.0e38                               # all at (nearly) the type's lowest value
    x[2, ::3] = 1.0
    x[3, 100:] = -0.0                            # -0 and +0 are equal
    x[4, V - 1] = 5.0
    x[5, 5000:6000] = 2.0
    u = torch.tensor([0.1, 0.3, 0.77, 0.9, 0.4, 0.61], device=DEV)
    for k, p, mp in ((7, 1.0, 0.0), (0, 0.37, 0.0), (12345, 1.0, 0.0), (0, 1.0, 1.0), (9000, 0.123, 0.0), (0, 1.0, 0.0), (0, 0.0, 0.0)):
        check_sample(x, u, params(6, 0, T=(1.0,), k=(k,), p=(p,), mp=(mp,)))
    check_sample(x, u, params(6, 0, T=(0.0,)))


def test_extreme_uniforms_and_magnitudes():
    V = 9000
    x = torch.randn((8, V), generator=torch.Generator().manual_seed(9)).to(DEV) * 2
    x[2] *= 1e37
    x[3, 17] = 3.4e38
    x[3, 18] = -3.4e38
    x[4] *= 1e-40                                # subnormal
    x[5] = float("-inf")
    x[5, 8999] = -7.0
    x[6, :4000] = -200.0                         # weights below a double's smallest at T = 0.1
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5, 0.5, 0.37, 0.99, 0.0, 2.0 ** -60], device=DEV)
    T = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 0.1, 1.0], device=DEV)
    r = sv.spec_sample_filtered(x, u, T)
    torch.cuda.synchronize()
    for b in range(8):
        assert int(r["tokens"][b]) == ref.sample_filtered(host(x[b]), float(u[b]), float(T[b]))[0], b


def test_bad_rows_leave_the_others():
    V = 3001
    x = rows(10, V, torch.float32, 2.0, 4)
    x[1, 5] = float("nan")
    x[2, 3000] = float("inf")
    x[3] = float("-inf")
    u = torch.full((10,), 0.43, device=DEV)
    q = params(10, 0, T=(0.8,), k=(30,), p=(0.9,), mp=(0.0,))
    r = sv.spec_sample_filtered(x, u, q["temperature"], top_k=q["top_k"], top_p=q["top_p"], min_p=q["min_p"])
    assert int(r["status"][0]) == sv.DEV_NONFINITE
    q["temperature"][4], q["temperature"][5], q["top_p"][6], q["min_p"][7] = -1.0, float("nan"), 1.5, float("nan")
    u[8] = 1.0
    r = sv.spec_sample_filtered(x, u, q["temperature"], top_k=q["top_k"], top_p=q["top_p"], min_p=q["min_p"])
    got = r["tokens"].cpu().numpy()
    assert int(r["status"][0]) == sv.DEV_NONFINITE | sv.DEV_BAD_PARAM
    assert (got[1:9] == -1).all()
    for b in (0, 9):
        assert got[b] == ref.sample_filtered(host(x[b]), 0.43, 0.8, 30, 0.9)[0]


def test_sampling_is_repeatable_and_captures():
    B, V = 40, 12289
    x = rows(B, V, torch.bfloat16, 2.0, 11)
    u = torch.rand(B, generator=torch.Generator().manual_seed(8)).to(DEV)
    q = params(B, 5, **MIXED)
    want = check_sample(x, u, q)
    out, status = dict(tokens=torch.zeros(B, dtype=torch.int32, device=DEV)), torch.zeros(1, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            sv.spec_sample_filtered(x, u, out=out, status=status, **q)
    for _ in range(3):
        out["tokens"].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert (out["tokens"].cpu().numpy() == want).all() and int(status[0]) == 0
    other = sv.spec_sample_filtered(x, u, stream=torch.cuda.Stream(), **q)
    torch.cuda.synchronize()
    assert (other["tokens"].cpu().numpy() == want).all()


def check_top(x, k, T=1.0, lse=True):
    r = sv.spec_top_logits(x, k, temperature=T, lse=lse)
    torch.cuda.synchronize()
    assert int(r["status"][0]) == 0
    for b in range(x.shape[0]):
        v, i, z = ref.top_logits(host(x[b]), k, T)
        assert np.array_equal(host(r["values"][b]), v), b
        assert np.array_equal(r["ids"][b].cpu().numpy(), i), b
        if lse:
            # fp32: the last rounding and log's (2^-24 |lse| + 2 * 2^-24 |log S|), and S's relative
            # error: each weight 2^-21 (ex2's 2^-22, its argument's rounding up to |x| 2^-24 where
            # weights below 2^-8 count little) and sums in trees, together below 2^-20
            tol = 2.0 ** -20 + 2.0 ** -22 * abs(z) if np.isfinite(z) else 0.0
            got = float(r["lse"][b])
            assert got == z or abs(got - z) <= tol, (b, got, z)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 9, 64, 1000, 5003, 32000, 50257, 131072])
def test_top_logits(V, dtype):
    x = rows(7, V, dtype, 3.0, V + 9, masked=0.4 if V % 2 else 0.0, offset=V % 3)
    for k in (1, 8, 100, 777, 1024):
        check_top(x, k, 0.7 if k == 8 else 1.0, lse=k != 100)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_logits_ties(dtype):
    V = 40001
    x = torch.zeros((5, V), dtype=dtype, device=DEV)
    x[1] = float("-inf")
    x[1, 39990:] = 1.5
    x[2, ::2] = 3.0
    x[3] = torch.arange(V, device=DEV).to(dtype) / 4096   # rising: the largest are neighbours
    x[4] = float("-inf")
    for k in (1, 5, 11, 500, 1024):
        check_top(x, k)


def test_top_logits_nonfinite_rows():
    x = rows(4, 6000, torch.float32, 2.0, 4)
    x[1, 5] = float("nan")
    x[2, 77] = float("inf")
    r = sv.spec_top_logits(x, 10, lse=True)
    assert int(r["status"][0]) == sv.DEV_NONFINITE
    for b in (1, 2):
        assert torch.isnan(r["values"][b]).all() and (r["ids"][b] == -1).all() and torch.isnan(r["lse"][b])
    for b in (0, 3):
        v, i, _ = ref.top_logits(host(x[b]), 10)
        assert np.array_equal(host(r["values"][b]), v) and np.array_equal(r["ids"][b].cpu().numpy(), i)


def test_the_longest_row_and_the_next():
    for dtype, V in ((torch.float32, 262144), (torch.bfloat16, 524288)):
        x = rows(2, V, dtype, 3.0, 5)
        check_top(x, 50)
        u = torch.tensor([0.3, 0.8], device=DEV)
        check_sample(x, u, params(2, 0, T=(0.9,), p=(0.95,)))
        with pytest.raises(sv.SpecError) as e:
            sv.spec_top_logits(torch.zeros((1, V + 1), dtype=dtype, device=DEV), 4)
        assert e.value.status == sv.SPEC_ERR_UNSUPPORTED


def test_offsets_past_32_bits():
    B, V = 17000, 131072                           # 4.5 GB of bf16
    x = torch.zeros((B, V), dtype=torch.bfloat16, device=DEV)
    x[-1] = rows(1, V, torch.bfloat16, 3.0, 8)[0]
    x[:, 7] += 1
    r = sv.spec_top_logits(x, 3)
    v, i, _ = ref.top_logits(host(x[-1]), 3)
    assert np.array_equal(host(r["values"][-1]), v) and np.array_equal(r["ids"][-1].cpu().numpy(), i)
    assert (r["ids"][:-1].cpu() == torch.tensor([7, 0, 1], dtype=torch.int32)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V,T,k,p,mp", [
    (5, 150001, 3.0, 0, 0.9, 0.0), (5, 150001, 3.0, 0, 1.0, 0.0), (3, 150001, 2.0, 20000, 0.6, 0.0), (3, 200000, 1.5, 3000, 1.0, 0.01),
    (700, 4099, 2.0, 0, 0.95, 0.0), (700, 4099, 1.0, 0, 1.0, 0.02), (400, 9001, 5.0, 2000, 0.9, 0.0), (2, 70000, 1e6, 0, 0.5, 0.0),
    (4, 60000, 0.05, 0, 0.999, 0.0), (4, 60000, 0.7, 1024, 0.99, 0.0), (4, 60000, 0.7, 1025, 0.99, 0.0)])
def test_long_rows_of_which_many_tokens_are_kept(B, V, T, k, p, mp, dtype):
    x = rows(B, V, dtype, 2.0, V + B)
    u = torch.rand(B, generator=torch.Generator().manual_seed(B)).to(DEV)
    check_sample(x, u, params(B, 0, T=(T,), k=(k,), p=(p,), mp=(mp,)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_few_unmasked_tokens_of_a_long_row(dtype):
    B, V = 6, 90001
    x = torch.full((B, V), float("-inf"), dtype=dtype, device=DEV)
    g = torch.Generator().manual_seed(1)
    for b, live in enumerate((1, 2, 40, 300, 1500, 5000)):
        at = torch.randperm(V, generator=g)[:live].to(DEV)
        x[b, at] = torch.randn(live, generator=g).to(dtype).to(DEV)
    u = torch.rand(B, generator=g).to(DEV)
    for q in (dict(), dict(k=(50,)), dict(p=(0.9,)), dict(mp=(0.3,)), dict(k=(1000,), p=(0.5,)), dict(k=(4000,), p=(0.5,))):
        check_sample(x, u, params(B, 0, **q))
    check_top(x, 100)
    check_top(x, 1024)


@pytest.mark.parametrize("scale", [1e30, 3e37, 1e-30])
def test_magnitudes(scale):
    """Logits whose products with log2(e) / T overflow, or are all but equal."""
    x = rows(4, 5003, torch.float32, 1.0, 3) * scale
    u = torch.tensor([0.1, 0.4, 0.7, 0.95], device=DEV)
    for q in (dict(p=(0.9,), T=(0.01,)), dict(p=(0.9,), T=(1e-6,)), dict(mp=(0.1,), T=(0.5,)), dict(T=(1e6,)), dict(k=(10,), T=(1e6,), p=(0.7,))):
        check_sample(x, u, params(4, 0, **q))
    r = sv.spec_top_logits(x, 20, lse=True)
    for b in range(4):
        v, i, z = ref.top_logits(host(x[b]), 20)
        assert np.array_equal(r["ids"][b].cpu().numpy(), i) and np.array_equal(host(r["values"][b]), v)
        assert abs(float(r["lse"][b]) - z) <= 2.0 ** -20 + 2.0 ** -22 * abs(z)


def test_a_zero_uniform_draws_the_first_kept_token():
    """u = 0 under each filter, with weights below half a unit among the kept (2^-60 and 2^-100 of the largest)."""
    for V in (300, 6000):
        x = torch.full((4, V), -50.0 * 0.6931, device=DEV)
        x[:, V - 1] = 0.0
        x[:, 3] = -60.0 * 0.6931
        x[:, 1] = -100.0 * 0.6931
        u = torch.zeros(4, device=DEV)
        for q in (dict(), dict(mp=(1e-20,)), dict(mp=(1e-25,)), dict(k=(V - 1,)), dict(mp=(1e-16,)), dict(k=(100,), mp=(1e-25,)), dict(k=(5000,), mp=(1e-25,)),
                  dict(mp=(0.5,)), dict(p=(0.5,))):
            q = params(4, 0, **q)
            r = sv.spec_sample_filtered(x, u, **q)
            want = [ref.sample_filtered(host(x[b]), 0.0, 1.0, int(q["top_k"][b]), float(q["top_p"][b]), float(q["min_p"][b]))[0] for b in range(4)]
            assert r["tokens"].tolist() == want


def test_the_first_call_may_be_captured():
    """In a process of its own: each operator's first call inside a graph capture."""
    import subprocess
    import sys
    code = """
import torch, sampling_online_softmax_gb300 as sv
x = torch.randn((6, 5003), device="cuda:0")
u, T = torch.rand(6, device="cuda:0"), torch.ones(6, device="cuda:0")
status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
o1 = dict(tokens=torch.zeros(6, dtype=torch.int32, device="cuda:0"))
o2 = dict(values=torch.zeros((6, 9), device="cuda:0"), ids=torch.zeros((6, 9), dtype=torch.int32, device="cuda:0"))
o3 = dict(loss=torch.zeros(6, device="cuda:0"), stats=torch.zeros((6, 2), device="cuda:0"), grad=torch.zeros_like(x))
g3 = torch.zeros_like(x)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    sv.spec_sample_filtered(x, u, T, out=o1, status=status)
    sv.spec_top_logits(x, 9, out=o2, status=status)
    sv.spec_distill(x, o2["ids"], o2["values"], grad=True, out=o3, status=status)
    sv.spec_distill_backward(x, o2["ids"], o2["values"], o3["stats"], T, out=g3, status=status)
g.replay()
torch.cuda.synchronize()
a = sv.spec_sample_filtered(x, u, T)["tokens"]
b = sv.spec_top_logits(x, 9)
c = sv.spec_distill(x, b["ids"], b["values"], grad=True)
torch.cuda.synchronize()
assert torch.equal(a, o1["tokens"]) and torch.equal(b["ids"], o2["ids"]) and torch.equal(c["grad"], o3["grad"]) and int(status[0]) == 0
assert (g3 - o3["grad"]).abs().max() < 1e-5
print("ok")
"""
    import os
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def test_another_stream_waits_for_the_inputs():
    """Inputs still being made on the current stream when the call goes to another one, and freed after it."""
    side = torch.cuda.Stream()
    big = torch.zeros((2048, 131072), device=DEV)
    want = None
    for _ in range(3):
        for _ in range(20):
            big.add_(1.0)                        # a millisecond or two before the logits are written
        x = torch.zeros((64, 9001), device=DEV)
        x[torch.arange(64, device=DEV), torch.arange(64, device=DEV) * 100 + 7] = 30.0
        u, T = torch.full((64,), 0.5, device=DEV), torch.ones(64, device=DEV)
        top = sv.spec_top_logits(x, 3, stream=side)
        tok = sv.spec_sample_filtered(x, u, T, stream=side)
        with torch.cuda.stream(side):
            r = sv.spec_distill(x, top["ids"], top["values"], grad=True)
        x.record_stream(side)
        del x, u, T
        junk = torch.full((64, 9001), 9.0, device=DEV)
        torch.cuda.synchronize()
        want = torch.arange(64, device=DEV, dtype=torch.int32) * 100 + 7
        assert torch.equal(tok["tokens"], want) and torch.equal(top["ids"][:, 0], want) and torch.isfinite(r["loss"]).all()
        del junk


@pytest.mark.parametrize("V", [2, 300, 5003])
def test_min_p_at_its_border_with_a_zero_uniform(V):
    """Tokens whose weight lies within one fp32 step of min-p: the first token of each row is kept or
    not by 2^-26 to 2^-24 of its weight, which 64 bits (and whole-number weights, right to 2^-38) tell
    and fp32 logarithms do not.  At u = 0 the draw is that token where it is kept, else a later one."""
    B = 64
    g = torch.Generator().manual_seed(57)
    x = torch.full((B, V), -30.0)
    x[:, V - 1] = 0.0
    x[:, 0] = -torch.rand((B,), generator=g) * 6.0
    w = np.exp(x[:, 0].numpy().astype(np.float64))
    mp = w.astype(np.float32)  # the nearest fp32, above the weight or below it
    far = np.abs(mp.astype(np.float64) / w - 1)
    assert (far > NEAR).all() and ((mp > w).sum() > 8) and ((mp < w).sum() > 8)
    x = x.to(DEV)
    one = torch.ones(B, device=DEV)
    for u in (0.0, 1e-12):
        r = sv.spec_sample_filtered(x, one * u, one, min_p=torch.tensor(mp, device=DEV))
        assert int(r["status"][0]) == 0
        assert r["tokens"].tolist() == [0 if a <= b else V - 1 for a, b in zip(mp.astype(np.float64), w)]
    # the long way: nothing but min-p of a long flat row's tail
    V = 60001
    x = torch.zeros((B, V), device=DEV)
    x[:, 0] = torch.tensor(np.log(w), dtype=torch.float32)
    w = np.exp(x[:, 0].cpu().numpy().astype(np.float64))
    mp = w.astype(np.float32)
    assert (np.abs(mp.astype(np.float64) / w - 1) > NEAR).all()
    r = sv.spec_sample_filtered(x, one * 0.0, one, min_p=torch.tensor(mp, device=DEV))
    assert r["tokens"].tolist() == [0 if a <= b else 1 for a, b in zip(mp.astype(np.float64), w)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift,scale,T,k", [
    (0.0, 2.0, 1.2, 0),         # both sides of 0
    (40.0, 2.0, 1.5, 0),        # all above it
    (-40.0, 2.0, 1.5, 0),       # all below it
    (0.0, 0.01, 0.006, 0),      # around 0 on a small scale
    (0.3, 0.001, 1.0, 0),       # few different bf16 values: thousands of equal logits at the cut
    (-0.001, 1e-6, 1.0, 0),     # one value in bf16, next to 0
    (0.0, 3000.0, 1500.0, 0),   # wide
    (0.0, 1e30, 5e5, 0),        # next to nothing but the maximum
    (0.0, 2.0, 1.2, 3001),      # top-p of the first k, k past a list's reach
    (-3.0, 0.01, 1.0, 2999),
])
def test_the_cut_of_long_rows_wherever_their_logits_lie(shift, scale, T, k, dtype):
    B, V = 5, 20011
    g = torch.Generator().manual_seed(91)
    x = (torch.randn((B, V), generator=g) * scale + shift).to(dtype).to(DEV)
    x[1, ::3] = float("-inf")
    x[2, 7] = x[2].max() + 0.5 * scale
    u = torch.tensor([0.11, 0.37, 0.52, 0.71, 0.93], device=DEV)
    for p in (0.3, 0.9, 0.999):
        check_sample(x, u, params(B, 0, T=(T,), k=(k,), p=(p,)))


@pytest.mark.parametrize("B", [1, 3, 200])
def test_the_cut_among_logits_next_to_zero(B):
    """Most of the weight on tokens a millionth from 0, between logits of both signs: bf16 keys that no
    histogram of a few thousand bins has beside those of the others."""
    V = 30001
    g = torch.Generator().manual_seed(92)
    x = torch.randn((B, V), generator=g) * 1e-6
    x[:, ::10] = torch.randn((B, (V + 9) // 10), generator=g) * 2 - 8
    x[:, 5] = 3.0
    x = x.to(torch.bfloat16).to(DEV)
    u = torch.rand((B,), generator=g).to(DEV)
    n = min(B, 3)  # (the oracle's time)
    r = sv.spec_sample_filtered(x, u, torch.ones(B, device=DEV), top_p=torch.full((B,), 0.6, device=DEV))
    check_sample(x[:n].contiguous(), u[:n].contiguous(), params(n, 0, T=(1.0,), p=(0.6,)))
    assert r["tokens"][:n].tolist() == sv.spec_sample_filtered(
        x[:n].contiguous(), u[:n].contiguous(), torch.ones(n, device=DEV), top_p=torch.full((n,), 0.6, device=DEV))["tokens"].tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [129, 1000, 5003])
def test_min_p_over_rows_of_the_lowest_value(V, dtype):
    """Rows masked by the type's lowest value, whole, mixed with -inf, and near it; min-p alone and beside the others."""
    low = torch.finfo(dtype).min
    x = torch.full((6, V), low, dtype=dtype, device=DEV)
    x[1, ::2] = float("-inf")
    x[2] = float("-inf")
    x[2, V - 1] = low
    x[3, V // 2] = low * (1 - 2.0 ** -7)
    x[4, 3] = 1.0
    x[5, : V // 3] = -1.0
    u = torch.tensor([0.11, 0.37, 0.52, 0.71, 0.93, 0.23], device=DEV)
    for q in (dict(mp=(0.05,)), dict(mp=(1.0,)), dict(mp=(1e-30,)), dict(mp=(0.05,), T=(1e6,)), dict(mp=(0.05,), T=(1e-6,)),
              dict(mp=(0.05,), p=(0.7,)), dict(mp=(0.05,), k=(40,)), dict(mp=(0.05,), k=(3,), p=(0.5,))):
        check_sample(x, u, params(6, 0, **q))
    check_sample(x, torch.zeros_like(u), params(6, 0, mp=(0.05,)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [200.0, 1000.0, 3000.0, -3000.0])
def test_top_p_of_rows_far_from_zero(size, dtype):
    """Logits over T around 10^4, where the maximum times log2(e) / T rounds by 2^-10: the bounds of the
    row's weight that the short list's cut goes by hold all the same."""
    B, V, T = 24, 20011, 0.1
    g = torch.Generator().manual_seed(14)
    x = (size + torch.randn((B, V), generator=g) * (0.35 if dtype == torch.float32 else 8.0)).to(dtype).to(DEV)
    T = T if dtype == torch.float32 else 2.3
    u = torch.rand(B, generator=g).to(DEV)
    for p in (0.2, 0.5, 0.9):
        check_sample(x, u, params(B, 0, T=(T,), p=(p,)))
