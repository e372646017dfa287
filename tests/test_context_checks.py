"""Refusals of the operators on the paged cache and of spec_adjust_logits, on the CPU: the C ABI's host-side checks (nothing
is launched), the binding's checks of tensors, and the tests' own reference on worked examples."""
import contextlib
import ctypes
import math

import pytest
import torch

import context_reference as ref
import sampling_online_softmax_gb300 as sv
from sampling_online_softmax_gb300 import build as sv_build

FAKE = 0x10000  # never dereferenced: every call below ends on the host
ODD, HALF = 0x10001, 0x10008
INV, UNS, WS, OK = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_UNSUPPORTED, sv.SPEC_ERR_WORKSPACE, sv.SPEC_OK
i32, u8 = torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.load_library()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, page_table=FAKE, dtype=sv.SPEC_BF16, pages=4, page_size=16, kv_heads=2, head_dim=64, table_width=3)
    a.update(kw)
    return sv._Cache(*(a[n] for n, _ in sv._Cache._fields_))


BAD_CACHES = [(dict(dtype=sv.SPEC_F32), INV), (dict(dtype=sv.SPEC_F16), INV), (dict(pages=-1), INV), (dict(kv_heads=0), INV), (dict(kv_heads=1025), UNS),
              (dict(table_width=-1), INV), (dict(head_dim=96), UNS), (dict(page_size=24), UNS), (dict(page_size=8), UNS), (dict(page_size=512), UNS),
              (dict(k=None), INV), (dict(v=None), INV), (dict(k=HALF), INV), (dict(v=ODD), INV), (dict(page_table=None), INV), (dict(page_table=ODD), INV),
              (dict(dtype=sv.SPEC_E4M3), INV), (dict(dtype=sv.SPEC_E4M3, k_scale=FAKE), INV), (dict(table_width=1 << 28), UNS)]


def _append(lib, cache=None, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=sv.SPEC_BF16, B=2, N=3, strides=None, select=None, S=3, start=FAKE, count=None, st=FAKE)
    a.update(kw)
    strides = (ctypes.c_longlong * 4)(*a["strides"]) if a["strides"] else None
    return lib.spec_cache_append(a["k"], a["v"], a["dtype"], a["B"], a["N"], strides, a["select"], a["S"], a["start"], a["count"],
                                 None if cache == "null" else ctypes.byref(_cache(**(cache or {}))), a["st"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=sv.SPEC_F32), INV), (dict(dtype=9), INV), (dict(cache="null"), INV), (dict(B=-1), INV), (dict(N=-1, S=-1), INV), (dict(S=2), INV),
    (dict(k=None), INV), (dict(v=None), INV), (dict(start=None), INV), (dict(st=None), INV), (dict(k=HALF), INV), (dict(v=ODD), INV), (dict(start=ODD), INV),
    (dict(count=ODD), INV), (dict(select=ODD), INV), (dict(st=ODD), INV), (dict(strides=[128, 4, 128, 8]), INV), (dict(strides=[128, 128, -8, 128]), INV),
    (dict(B=0), OK), (dict(N=0, S=0), OK)] + [(dict(cache=c), e) for c, e in BAD_CACHES])
def test_cache_append_host_validation(lib, kw, expect):
    assert _append(lib, **kw) == expect
    assert (lib.spec_last_error().decode() == "") == (expect == OK)


def _read(lib, cache=None, **kw):
    a = dict(B=2, S=3, start=FAKE, count=None, k=FAKE, v=FAKE, dtype=sv.SPEC_BF16, st=FAKE)
    a.update(kw)
    return lib.spec_cache_read(ctypes.byref(_cache(**(cache or {}))), a["B"], a["S"], a["start"], a["count"], a["k"], a["v"], a["dtype"], a["st"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=sv.SPEC_E4M3), INV), (dict(B=-1), INV), (dict(S=-1), INV), (dict(k=None), INV), (dict(v=HALF), INV), (dict(start=None), INV),
    (dict(start=ODD), INV), (dict(count=ODD), INV), (dict(st=None), INV), (dict(B=0), OK), (dict(S=0), OK)] + [(dict(cache=c), e) for c, e in BAD_CACHES])
def test_cache_read_host_validation(lib, kw, expect):
    assert _read(lib, **kw) == expect
    assert (lib.spec_last_error().decode() == "") == (expect == OK)


def _attend(lib, cache=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=sv.SPEC_BF16, B=2, N=3, heads=4, strides=None, lens=FAKE, shared=0, mask=None, scale=0.1, out=FAKE, lse=None,
             st=FAKE, ws=FAKE, room=1 << 40)
    a.update(kw)
    strides = (ctypes.c_longlong * 6)(*a["strides"]) if a["strides"] else None
    return lib.spec_tree_attention(a["q"], a["k"], a["v"], a["dtype"], a["B"], a["N"], a["heads"], strides, ctypes.byref(_cache(**(cache or {}))), a["lens"],
                                   a["shared"], a["mask"], a["scale"], a["out"], a["lse"], a["st"], a["ws"], a["room"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=sv.SPEC_F32), INV), (dict(B=-1), INV), (dict(N=0), INV), (dict(N=sv.MAX_NODES + 1), UNS), (dict(heads=3), INV), (dict(heads=0), INV),
    (dict(shared=-1), INV), (dict(shared=49), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(lens=None), INV), (dict(out=None), INV), (dict(st=None), INV), (dict(q=HALF), INV),
    (dict(out=HALF), INV), (dict(lens=ODD), INV), (dict(mask=ODD), INV), (dict(lse=ODD), INV), (dict(ws=None), WS), (dict(ws=HALF), WS), (dict(room=0), WS),
    (dict(strides=[256, 4] + [256, 8] * 2), INV), (dict(B=1 << 20, N=1024, heads=4), UNS), (dict(B=0), OK)] + [(dict(cache=c), e) for c, e in BAD_CACHES])
def test_tree_attention_host_validation(lib, kw, expect):
    assert _attend(lib, **kw) == expect
    assert (lib.spec_last_error().decode() == "") == (expect == OK)


FAR = dict(k=FAKE + (1 << 20), v=FAKE + (1 << 20), out=FAKE + (1 << 21))  # B = 2, N = 3, 4 query heads of 64 on 1 or 2


@pytest.mark.parametrize("kw,expect", [
    (dict(heads=129, cache=dict(kv_heads=1)), UNS), (dict(FAR, strides=[0, 256] + [768, 256] * 2), INV), (dict(FAR, strides=[768, 256, 768, 0, 768, 256]), INV),
    (dict(FAR, strides=[1 << 38, 256] + [768, 256] * 2), INV), (dict(FAR, strides=[-768, 256] + [768, 256] * 2), INV),
    (dict(FAR, shared=16, strides=[1024, 256] + [768, 256] * 2), UNS), (dict(cache=dict(table_width=(1 << 26) + 1)), UNS),
    (dict(FAR, out=FAKE), INV), (dict(FAR, out=FAKE + 16), INV), (dict(FAR, out=FAR["k"] - 16), INV), (dict(FAR, out=FAR["v"] + 16), INV)])
def test_tree_attention_limits(lib, kw, expect):
    assert _attend(lib, **kw) == expect and lib.spec_last_error().decode()


LAST = dict(FAR, heads=1024, out=FAKE + (1 << 30), cache=dict(kv_heads=1024, table_width=1 << 26))  # (more tiles than a call takes: the last check)


@pytest.mark.parametrize("kw", [
    dict(N=1, shared=16, strides=[3 << 16, 1 << 16] + [3 << 16, 1 << 16] * 2),  # slices of a fused projection, as the binding passes them
    dict(N=1, shared=16, strides=[3 << 16, 3] + [3 << 16, 0] * 2), dict(N=1, shared=0, strides=[3 << 16, 1 << 50] * 3),
    dict(B=1, N=2, shared=16, strides=[0, 1 << 16] + [7, 1 << 16] * 2), dict(B=1, N=2, shared=16, strides=[1 << 50, 1 << 20] * 3),
    dict(B=1, N=1, shared=16, strides=[3, 5] * 3), dict(N=2, shared=16, strides=[2 << 16, 1 << 16] * 3)])
def test_an_axis_of_one_entry_has_any_stride(lib, kw):
    assert _attend(lib, **LAST, **kw) == UNS and "too much work" in lib.spec_last_error().decode()
    if kw.get("B") != 1 and kw["N"] == 1:  # the other axis' stride still counts
        for bad in (4, -8, 0, 1 << 38):
            assert _attend(lib, **LAST, **{**kw, "strides": [bad, 1 << 16] * 3}) == INV


def test_cache_call_limits(lib):
    assert _append(lib, B=1 << 20, N=64, S=64) == UNS and _read(lib, B=1 << 20, S=64) == UNS
    assert _append(lib, cache=dict(table_width=(1 << 26) + 1)) == UNS and _read(lib, cache=dict(table_width=(1 << 26) + 1)) == UNS


def test_attention_workspace_sizes(lib):
    size = sv.spec_workspace_bytes_attention
    assert size(4, 5, 8, 2, 128) > 0 and size(4, 5, 8, 2, 128, 1000) >= size(4, 5, 8, 2, 128)
    for bad in ((0, 5, 8, 2, 128), (4, 0, 8, 2, 128), (4, sv.MAX_NODES + 1, 8, 2, 128), (4, 5, 7, 2, 128), (4, 5, 0, 2, 128), (4, 5, 8, 0, 128), (4, 5, 8, 2, 80)):
        assert size(*bad) == 0
    assert size(4, 5, 8, 2, 128, -1) == 0


def _adjust(lib, **kw):
    a = dict(x=FAKE, dtype=1, B=2, N=3, V=100, tokens=None, L=0, prompt=None, total=None, nodes=None, mask=None, rep=None, freq=None, pres=None, ids=None,
             bias=None, M=0, allowed=None, out=FAKE + (1 << 20), st=FAKE)
    a.update(kw)
    return lib.spec_adjust_logits(a["x"], a["dtype"], a["B"], a["N"], a["V"], a["tokens"], a["L"], a["prompt"], a["total"], a["nodes"], a["mask"], a["rep"],
                                  a["freq"], a["pres"], a["ids"], a["bias"], a["M"], a["allowed"], a["out"], a["st"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=sv.SPEC_F16), INV), (dict(B=-1), INV), (dict(N=0), INV), (dict(V=0), INV), (dict(L=-1), INV), (dict(M=-1), INV), (dict(N=sv.MAX_NODES + 1), UNS),
    (dict(M=sv.MAX_BIASES + 1), UNS), (dict(L=1 << 24), UNS), (dict(V=sv.MAX_ROW_BYTES // 2 + 1), UNS), (dict(x=None), INV), (dict(out=None), INV),
    (dict(st=None), INV), (dict(L=4), INV), (dict(M=4), INV), (dict(M=4, ids=FAKE), INV), (dict(x=ODD), INV), (dict(out=ODD), INV), (dict(tokens=ODD), INV),
    (dict(prompt=ODD), INV), (dict(total=ODD), INV), (dict(nodes=ODD), INV), (dict(mask=ODD), INV), (dict(rep=ODD), INV), (dict(freq=ODD), INV),
    (dict(pres=ODD), INV), (dict(allowed=ODD), INV), (dict(out=FAKE + 1198), INV), (dict(out=FAKE - 1198), INV), (dict(B=0), OK)])
def test_adjust_logits_host_validation(lib, kw, expect):
    assert _adjust(lib, **kw) == expect
    assert (lib.spec_last_error().decode() == "") == (expect == OK)


@pytest.fixture
def fake(monkeypatch):
    """A library that records calls, and CPU tensors in the place of CUDA ones."""
    calls = []

    class FakeLib:
        def __getattr__(self, name):
            def f(*args):
                calls.append(name)
                return 0
            return f

    lib = FakeLib()
    real = sv._cuda

    class OnGpu:
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

    monkeypatch.setattr(sv, "load_library", lambda: lib)
    monkeypatch.setattr(sv, "_cuda", lambda t, *a: t if t is None or real(OnGpu(t), *a) is None else t)
    monkeypatch.setattr(sv, "_on_gpu", lambda t, name: None)
    monkeypatch.setattr(sv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(sv, "_alloc", lambda nbytes, stream: calls.append("alloc") or 256)
    monkeypatch.setattr(sv, "_free", lambda at: calls.append("free"))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return calls


B, N, H, G, D, P, W = 3, 5, 4, 2, 64, 16, 6
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def _tensors(dtype=BF, q8=False):
    shape = (10, G, P, D)
    s = dict(k=torch.zeros((B, N, G, D), dtype=dtype), v=torch.zeros((B, N, G, D), dtype=dtype),
             k_cache=torch.zeros(shape, dtype=F8 if q8 else dtype), v_cache=torch.zeros(shape, dtype=F8 if q8 else dtype),
             page_table=torch.zeros((B, W), dtype=i32), start=torch.zeros(B, dtype=i32))
    if q8:
        s.update(k_scale=torch.zeros(shape[:3], dtype=u8), v_scale=torch.zeros(shape[:3], dtype=u8))
    return s


def test_cache_append_binding(fake):
    call = lambda base, **kw: sv.spec_cache_append(**{**base, **kw})  # noqa: E731
    call(_tensors())
    call(_tensors(torch.float16, True), count=torch.zeros(B, dtype=i32), select=torch.zeros((B, 9), dtype=i32))
    wide = torch.zeros((B, N, 3 * G, D), dtype=BF)  # a fused projection's keys and values
    call(_tensors(), k=wide[:, :, :G], v=wide[:, :, G:2 * G])
    s, e = _tensors(), _tensors(q8=True)
    for base, bad in ((s, dict(k=s["k"][0])), (s, dict(v=s["v"][:, 1:])), (s, dict(k=s["k"].transpose(2, 3).contiguous().transpose(2, 3))),
                      (s, dict(k=torch.zeros((B, N, G, D + 4), dtype=BF)[..., :D])), (s, dict(k_cache=s["k_cache"][0])), (s, dict(k_cache=s["k_cache"][:, :1])),
                      (s, dict(v_cache=s["v_cache"][1:])), (s, dict(page_table=s["page_table"][1:])), (s, dict(page_table=s["page_table"][0])),
                      (s, dict(start=s["start"][1:])), (s, dict(count=torch.zeros(B + 1, dtype=i32))), (s, dict(select=torch.zeros(B, dtype=i32))),
                      (s, dict(select=torch.zeros((B + 1, 2), dtype=i32))), (s, dict(k_scale=e["k_scale"], v_scale=e["v_scale"])), (e, dict(k_scale=None)),
                      (e, dict(v_scale=e["v_scale"][1:])), (s, dict(status=torch.zeros(0, dtype=i32)))):
        with pytest.raises(ValueError):
            call(base, **bad)
    for base, bad in ((s, dict(k=s["k"].float())), (s, dict(v=s["v"].half())), (s, dict(k_cache=s["k_cache"].half())), (e, dict(k_scale=e["k_scale"].int())),
                      (s, dict(start=s["start"].long())), (s, dict(page_table=s["page_table"].long())), (s, dict(count=torch.zeros(B)))):
        with pytest.raises(TypeError):
            call(base, **bad)
    assert fake.count("spec_cache_append") == 3


def test_cache_read_binding(fake):
    def call(base, n=4, **kw):
        a = {**{x: y for x, y in base.items() if x not in ("k", "v")}, **kw}
        return sv.spec_cache_read(a.pop("k_cache"), a.pop("v_cache"), a.pop("page_table"), a.pop("start"), n, **a)
    s, e = _tensors(), _tensors(q8=True)
    assert call(s)["k"].shape == (B, 4, G, D) and call(e, dtype=torch.float16)["v"].dtype is torch.float16
    for base, bad in ((s, dict(n=-1)), (s, dict(start=s["start"][1:])), (s, dict(count=torch.zeros(1, dtype=i32))), (s, dict(k_cache=s["k_cache"][0])),
                      (s, dict(out=dict(k=torch.zeros((B, 4, G, D), dtype=BF)))), (e, dict(k_scale=None))):
        with pytest.raises(ValueError):
            call(base, **bad)
    for base, bad in ((e, dict(dtype=torch.float32)), (s, dict(v_cache=s["v_cache"].half()))):
        with pytest.raises(TypeError):
            call(base, **bad)
    assert fake.count("spec_cache_read") == 2


def test_tree_attention_binding(fake, monkeypatch):
    class Sized:
        def __getattr__(self, name):
            def f(*args):
                fake.append(name)
                return 4096 if name.startswith("spec_workspace") else 0
            return f
    monkeypatch.setattr(sv, "load_library", lambda: Sized())
    def call(base, **kw):
        a = {**base, "q": torch.zeros((B, N, H, D), dtype=base["k"].dtype), **kw}
        return sv.spec_tree_attention(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("k_cache"), a.pop("v_cache"), a.pop("page_table"), a.pop("start"), **a)
    s, e = _tensors(), _tensors(q8=True)
    assert call(s)["out"].shape == (B, N, H, D) and call(e, lse=True, mask=torch.zeros((N, 1), dtype=i32))["lse"].shape == (B, N, H)
    for base, bad in ((s, dict(q=torch.zeros((B, N, 3, D), dtype=BF))), (s, dict(q=torch.zeros((B, N, D), dtype=BF))), (s, dict(k=s["k"][0])),
                      (s, dict(v=s["v"][:, :, :1])), (s, dict(mask=torch.zeros((N, 2), dtype=i32))), (s, dict(start=s["start"][1:])),
                      (s, dict(out=dict(out=torch.zeros((B, N, G, D), dtype=BF)))), (s, dict(lse=True, out=dict(out=torch.zeros((B, N, H, D), dtype=BF)))),
                      (e, dict(v_scale=None))):
        with pytest.raises(ValueError):
            call(base, **bad)
    for base, bad in ((s, dict(q=torch.zeros((B, N, H, D)))), (s, dict(k=s["k"].half())), (s, dict(mask=torch.zeros((N, 1)))), (s, dict(start=s["start"].long()))):
        with pytest.raises(TypeError):
            call(base, **bad)
    assert fake.count("spec_tree_attention") == 2
    # the workspace goes back, once for each it came, also where the call is refused
    assert fake.count("alloc") == fake.count("free") == 2
    monkeypatch.setattr(sv, "_launch", lambda *a: (_ for _ in ()).throw(RuntimeError("refused")))
    with pytest.raises(RuntimeError):
        call(s)
    assert fake.count("alloc") == fake.count("free") == 3
    with pytest.raises(RuntimeError):
        call(s, workspace=torch.zeros(4096, dtype=torch.uint8))
    assert fake.count("alloc") == 3


def test_adjust_logits_binding(fake):
    V = 70
    x, per = torch.zeros((B, N, V)), torch.ones(B)
    full = dict(tokens=torch.zeros((B, 9), dtype=i32), prompt_len=torch.zeros(B, dtype=i32), total_len=torch.zeros(B, dtype=i32),
                node_tokens=torch.zeros((B, N), dtype=i32), mask=torch.zeros((N, 1), dtype=i32), repetition=per, frequency=per, presence=per,
                bias_ids=torch.zeros((B, 2), dtype=i32), bias=torch.zeros((B, 2)), allowed=torch.zeros((B, N, 3), dtype=i32))
    sv.spec_adjust_logits(x, **full)
    sv.spec_adjust_logits(x.bfloat16())
    version = x._version
    sv.spec_adjust_logits(x, out=dict(logits=x))
    assert x._version > version  # a graph that saved the logits is refused
    for bad in (dict(tokens=torch.zeros(9, dtype=i32)), dict(tokens=torch.zeros((B + 1, 9), dtype=i32)), dict(prompt_len=torch.zeros(1, dtype=i32)),
                dict(node_tokens=torch.zeros((B, N - 1), dtype=i32)), dict(mask=torch.zeros((N, 2), dtype=i32)), dict(repetition=torch.ones(B + 1)),
                dict(bias=None), dict(bias_ids=None), dict(bias=torch.zeros((B, 3))), dict(bias_ids=torch.zeros(B, dtype=i32)), dict(allowed=torch.zeros((B, N, 2), dtype=i32)),
                dict(out=dict(logits=x[:1].clone())), dict(out={})):
        with pytest.raises(ValueError):
            sv.spec_adjust_logits(x, **{**full, **bad})
    with pytest.raises(ValueError):
        sv.spec_adjust_logits(x[0])
    for bad in (dict(tokens=torch.zeros((B, 9))), dict(repetition=per.double()), dict(allowed=torch.zeros((B, N, 3))), dict(out=dict(logits=x.bfloat16()))):
        with pytest.raises(TypeError):
            sv.spec_adjust_logits(x, **{**full, **bad})
    with pytest.raises(TypeError):
        sv.spec_adjust_logits(x.half())
    assert fake.count("spec_adjust_logits") == 3


def test_the_reference_quantises_worked_rows():
    x = torch.tensor([[448.0, 17.0, -19.0, 2.0 ** -10], [449.0, 448.0, 1.0, 0.0], [0.0, 0.0, 0.0, 0.0], [1.75 * 2.0 ** -20, 0.0, 0.0, 0.0]])
    y, byte = ref.quantised(x)
    assert byte.tolist() == [127, 128, 17, 127 - 28]
    assert y[0].tolist() == [448.0, 16.0, -20.0, 0.0]  # 17 and -19 lie midway: to the even one; 2^-10 is half a step of 2^-9: to 0
    assert y[1].tolist() == [448.0, 448.0, 1.0, 0.0]   # 449 / 2 = 224.5: steps of 16
    assert y[3, 0] == 1.75 * 2.0 ** -20
    z, byte = ref.quantised(torch.tensor([[65504.0, 1.0]]), fp16=True)
    assert byte.tolist() == [135] and z[0, 0] == 61440.0


def test_the_reference_attends_a_worked_row():
    q = torch.zeros((1, 2, 1, 64))
    q[..., 0] = 2.0
    k = torch.zeros((1, 2, 1, 64))
    k[0, 1, 0, 0] = math.log(3.0) / 2.0
    v = torch.ones((1, 2, 1, 64))
    v[0, 1] = 5.0
    seen = torch.tensor([[True, False], [True, True]])
    out, lse, weight, mass = ref.attention(q, k, v, [torch.zeros((0, 1, 64), dtype=torch.float64)], [torch.zeros((0, 1, 64), dtype=torch.float64)], [0], seen, 1.0)
    assert abs(float(out[0, 1, 0, 0]) - (1 + 3 * 5) / 4) < 1e-6 and float(out[0, 0, 0, 0]) == 1.0 and abs(float(lse[0, 1, 0]) - math.log(4)) < 1e-6


def test_the_reference_adjusts_a_worked_row():
    x = torch.tensor([[[1.0, -2.0, 3.0, 4.0, 5.0]]])
    seen = torch.ones((1, 1), dtype=torch.bool)
    t = torch.tensor([[0, 1, 2, 2, -1]], dtype=i32)
    y = ref.adjusted(x, seen, t, torch.tensor([1]), None, None, torch.tensor([2.0]), torch.tensor([0.5]), torch.tensor([0.25]),
                     torch.tensor([[3, 3]], dtype=i32), torch.tensor([[1.0, 2.0]]), torch.tensor([[[0b01111]]], dtype=i32))
    assert y[0, 0].tolist() == [0.5, -2.0 * 2 - 0.5 - 0.25, 1.5 - 1.0 - 0.25, 7.0, -math.inf]
