"""Refusals of the operators on rows of logits, on the CPU: the C ABI's host-side
checks (nothing is launched) and the binding's checks of tensors."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import rows_reference as ref
import sampling_online_softmax_gb300 as sv
from sampling_online_softmax_gb300 import build as sv_build

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below ends on the host
ODD = ctypes.c_void_p(0x10001)
i32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.load_library()


def _sample(lib, **kw):
    a = dict(x=FAKE, dtype=1, B=2, V=100, T=FAKE, k=None, p=None, mp=None, u=FAKE, tok=FAKE, st=FAKE)
    a.update(kw)
    return lib.spec_sample_filtered(a["x"], a["dtype"], a["B"], a["V"], a["T"], a["k"], a["p"], a["mp"], a["u"], a["tok"], a["st"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=7), sv.SPEC_ERR_INVALID_ARG), (dict(B=-1), sv.SPEC_ERR_INVALID_ARG), (dict(V=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(x=None), sv.SPEC_ERR_INVALID_ARG), (dict(x=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(T=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(u=None), sv.SPEC_ERR_INVALID_ARG), (dict(tok=None), sv.SPEC_ERR_INVALID_ARG), (dict(st=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(k=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(p=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(mp=ODD), sv.SPEC_ERR_INVALID_ARG),
    (dict(V=sv.MAX_ROW_BYTES // 2 + 1), sv.SPEC_ERR_UNSUPPORTED), (dict(dtype=0, V=sv.MAX_ROW_BYTES // 4 + 1), sv.SPEC_ERR_UNSUPPORTED),
    (dict(B=0), sv.SPEC_OK)])
def test_sample_filtered_host_validation(lib, kw, expect):
    assert _sample(lib, **kw) == expect
    assert (lib.spec_last_error().decode() == "") == (expect == sv.SPEC_OK)


def _top(lib, **kw):
    a = dict(x=FAKE, dtype=1, B=2, V=100, K=5, T=1.0, v=FAKE, i=FAKE, lse=FAKE, st=FAKE)
    a.update(kw)
    return lib.spec_top_logits(a["x"], a["dtype"], a["B"], a["V"], a["K"], a["T"], a["v"], a["i"], a["lse"], a["st"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=-1), sv.SPEC_ERR_INVALID_ARG), (dict(B=-1), sv.SPEC_ERR_INVALID_ARG), (dict(V=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(K=0), sv.SPEC_ERR_INVALID_ARG), (dict(K=sv.MAX_TOP + 1), sv.SPEC_ERR_UNSUPPORTED), (dict(T=0.0), sv.SPEC_ERR_INVALID_ARG),
    (dict(T=float("nan")), sv.SPEC_ERR_INVALID_ARG), (dict(T=1e7), sv.SPEC_ERR_INVALID_ARG), (dict(x=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(x=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(v=None), sv.SPEC_ERR_INVALID_ARG), (dict(i=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(lse=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(st=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(V=sv.MAX_ROW_BYTES // 2 + 1), sv.SPEC_ERR_UNSUPPORTED), (dict(B=0, lse=None), sv.SPEC_OK)])
def test_top_logits_host_validation(lib, kw, expect):
    assert _top(lib, **kw) == expect
    assert (lib.spec_last_error().decode() == "") == (expect == sv.SPEC_OK)


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
        """A CPU tensor that says it is on the GPU."""
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

    monkeypatch.setattr(sv, "load_library", lambda: lib)
    monkeypatch.setattr(sv, "_cuda", lambda t, *a: t if t is None or real(OnGpu(t), *a) is None else t)
    monkeypatch.setattr(sv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)  # a CPU device's index
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return calls


B, V = 3, 50


def test_sample_filtered_binding(fake):
    x, u, T = torch.zeros((B, V)), torch.zeros(B), torch.ones(B)
    k, p = torch.zeros(B, dtype=i32), torch.ones(B)
    sv.spec_sample_filtered(x, u, T, top_k=k, top_p=p, min_p=p)
    sv.spec_sample_filtered(x.bfloat16(), u, T)
    assert fake.count("spec_sample_filtered") == 2
    for bad in (dict(x=x[0]), dict(x=torch.zeros((V, B)).t()), dict(u=torch.zeros(B + 1)), dict(u=None), dict(T=None), dict(T=torch.ones(1)),
                dict(k=torch.zeros(B - 1, dtype=i32)), dict(p=torch.zeros((B, 1))), dict(mp=torch.zeros(2 * B)[::2]),
                dict(out=dict(tokens=torch.zeros(B + 1, dtype=i32))), dict(out={}), dict(status=torch.zeros(0, dtype=i32))):
        with pytest.raises(ValueError):
            sv.spec_sample_filtered(bad.get("x", x), bad.get("u", u), bad.get("T", T), top_k=bad.get("k"), top_p=bad.get("p"),
                                    min_p=bad.get("mp"), out=bad.get("out"), status=bad.get("status"))
    for bad in (dict(x=x.half()), dict(u=u.double()), dict(k=torch.zeros(B, dtype=torch.int64)), dict(T=T.bfloat16())):
        with pytest.raises(TypeError):
            sv.spec_sample_filtered(bad.get("x", x), bad.get("u", u), bad.get("T", T), top_k=bad.get("k"))
    assert fake.count("spec_sample_filtered") == 2


def test_top_logits_binding(fake):
    x = torch.zeros((B, V))
    assert "lse" not in sv.spec_top_logits(x, 4)
    assert sv.spec_top_logits(x, 4, lse=True)["lse"].shape == (B,)
    for bad in (dict(x=x[0]), dict(k=0), dict(out=dict(values=torch.zeros((B, 4)))),
                dict(out=dict(values=torch.zeros((B, 5)), ids=torch.zeros((B, 4), dtype=i32)))):
        with pytest.raises(ValueError):
            sv.spec_top_logits(bad.get("x", x), bad.get("k", 4), out=bad.get("out"))
    with pytest.raises(TypeError):
        sv.spec_top_logits(x.double(), 4)
    assert fake.count("spec_top_logits") == 2


def test_the_reference_on_a_worked_row():
    """x = log [4, 2, 1, 1] at T = 1: weights 1, 1/2, 1/4, 1/4 of the largest."""
    x = np.log(np.array([1.0, 4.0, 1.0, 2.0]))
    assert list(ref.kept_order(x, 1.0)) == [1, 3, 0, 2]
    assert list(ref.kept_order(x, 1.0, p=0.76)) == [1, 3, 0]
    assert list(ref.kept_order(x, 1.0, k=3, p=0.5)) == [1]
    assert list(ref.kept_order(x, 1.0, min_p=0.3)) == [1, 3]
    assert [ref.sample_filtered(x, u, 1.0)[0] for u in (0.0, 0.1, 0.2, 0.6, 0.7, 0.99)] == [0, 0, 1, 1, 2, 3]
    assert [ref.sample_filtered(x, u, 1.0, k=2)[0] for u in (0.0, 0.6, 0.7)] == [1, 1, 3]
    assert ref.sample_filtered(x, 0.9, 0.0)[0] == 1


def _distill(lib, **kw):
    a = dict(x=FAKE, dtype=1, N=2, V=100, ids=FAKE, t=FAKE, K=5, lse=None, T=1.0, w=None, loss=FAKE, stats=FAKE, grad=FAKE, st=FAKE)
    a.update(kw)
    head = [a[n] for n in ("x", "dtype", "N", "V", "ids", "t", "K", "lse", "T", "w")]
    return (lib.spec_distill(*head, a["loss"], a["stats"], a["grad"], a["st"], None),
            lib.spec_distill_backward(*head, a["stats"], a["loss"], a["grad"], a["st"], None))


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), sv.SPEC_ERR_INVALID_ARG), (dict(N=-1), sv.SPEC_ERR_INVALID_ARG), (dict(V=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(K=0), sv.SPEC_ERR_INVALID_ARG), (dict(K=sv.MAX_TOP + 1), sv.SPEC_ERR_UNSUPPORTED), (dict(T=0.0), sv.SPEC_ERR_INVALID_ARG),
    (dict(T=float("inf")), sv.SPEC_ERR_INVALID_ARG), (dict(T=float("nan")), sv.SPEC_ERR_INVALID_ARG), (dict(x=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(x=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(ids=None), sv.SPEC_ERR_INVALID_ARG), (dict(t=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(lse=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(w=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(loss=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(stats=None), sv.SPEC_ERR_INVALID_ARG), (dict(grad=ODD), sv.SPEC_ERR_INVALID_ARG), (dict(st=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(V=sv.MAX_ROW_BYTES // 2 + 1), sv.SPEC_ERR_UNSUPPORTED), (dict(N=0), sv.SPEC_OK)])
def test_distill_host_validation(lib, kw, expect):
    assert _distill(lib, **kw) == (expect, expect)


def test_distill_backward_needs_a_gradient(lib):
    assert lib.spec_distill_backward(FAKE, 1, 2, 100, FAKE, FAKE, 5, None, 1.0, None, FAKE, FAKE, None, FAKE, None) == sv.SPEC_ERR_INVALID_ARG


def test_distill_binding(fake):
    N, K = 4, 6
    x, ids, t, n = torch.zeros((N, V)), torch.zeros((N, K), dtype=i32), torch.zeros((N, K)), torch.zeros(N)
    r = sv.spec_distill(x, ids, t, top_lse=n, row_weight=n)
    assert "grad" not in r and r["stats"].shape == (N, 2)
    assert sv.spec_distill(x.bfloat16(), ids, t, grad=True)["grad"].dtype == torch.bfloat16
    assert sv.spec_distill_backward(x, ids, t, r["stats"], n)["grad"].shape == (N, V)
    for bad in (dict(x=x[0]), dict(ids=ids[:2].contiguous()), dict(ids=None), dict(t=t[:, :3].contiguous()), dict(t=None), dict(ids=ids[:, :0], t=t[:, :0]),
                dict(lse=torch.zeros(N + 1)), dict(w=torch.zeros((N, 1))), dict(x=torch.zeros((V, N)).t())):
        with pytest.raises(ValueError):
            sv.spec_distill(bad.get("x", x), bad.get("ids", ids), bad.get("t", t), top_lse=bad.get("lse"), row_weight=bad.get("w"))
        with pytest.raises(ValueError):
            sv.spec_distill_backward(bad.get("x", x), bad.get("ids", ids), bad.get("t", t), r["stats"], n, top_lse=bad.get("lse"), row_weight=bad.get("w"))
    for kw in (dict(stats=None), dict(stats=n), dict(grad_loss=None), dict(grad_loss=torch.zeros(1)), dict(out=torch.zeros((N, V + 1)))):
        with pytest.raises(ValueError):
            sv.spec_distill_backward(x, ids, t, kw.get("stats", r["stats"]) if "stats" in kw else r["stats"],
                                     kw["grad_loss"] if "grad_loss" in kw else n, out=kw.get("out"))
    with pytest.raises(ValueError):
        sv.spec_distill(x, ids, t, grad=True, out=dict(loss=n, stats=torch.zeros((N, 2))))
    with pytest.raises(TypeError):
        sv.spec_distill(x, ids.long(), t)
    with pytest.raises(TypeError):
        sv.spec_distill(x, ids, t.bfloat16())
    with pytest.raises(TypeError):
        sv.spec_distill(x, ids, t, grad=True, out=dict(loss=n, stats=torch.zeros((N, 2)), grad=torch.zeros((N, V)).bfloat16()))


def test_the_distillation_reference_on_a_worked_row():
    """Student uniform over 4, teacher all on token 2: loss log 4, gradient 1/4 - [v = 2]; differences agree."""
    x, ids, t = np.zeros(4), np.array([2, -1], np.int32), np.array([5.0, 9.0])
    loss, (m, S), g = ref.distill(x, ids, t)
    assert abs(loss - np.log(4)) < 1e-15 and (m, S) == (0.0, 4.0) and np.allclose(g, [0.25, 0.25, -0.75, 0.25])
    r = np.random.RandomState(0)
    x, ids, t = r.randn(9), np.array([3, 7, 3, 0], np.int32), r.randn(4)
    for lse in (None, 1.7):
        _, _, g = ref.distill(x, ids, t, lse, 0.5, 2.0)
        for v in range(9):
            h = np.zeros(9)
            h[v] = 1e-6
            d = (ref.distill(x + h, ids, t, lse, 0.5, 2.0)[0] - ref.distill(x - h, ids, t, lse, 0.5, 2.0)[0]) / 2e-6
            assert abs(d - g[v]) < 1e-7


def test_a_gradient_over_saved_logits_is_refused_by_autograd(fake):
    """exp saves its result: a gradient written over it, by either call, makes the graph's backward an error, not a
    wrong gradient."""
    N, K = 4, 6
    ids, t, n = torch.zeros((N, K), dtype=i32), torch.zeros((N, K)), torch.zeros(N)
    for call in (lambda y: sv.spec_distill(y, ids, t, grad=True, out=dict(loss=n.clone(), stats=torch.zeros((N, 2)), grad=y)),
                 lambda y: sv.spec_distill_backward(y, ids, t, torch.zeros((N, 2)), n, out=y)):
        leaf = torch.zeros((N, V), requires_grad=True)
        y = leaf.exp()
        call(y.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        y = leaf.exp()
        sv.spec_distill(y.detach(), ids, t, grad=True, out=dict(loss=n.clone(), stats=torch.zeros((N, 2)), grad=torch.zeros((N, V))))
        sv.spec_distill_backward(y.detach(), ids, t, torch.zeros((N, 2)), n)
        y.sum().backward()
        with torch.inference_mode():
            call(torch.zeros((N, V)))


@pytest.mark.parametrize("dtype", [0, 1])
def test_a_gradient_that_overlaps_the_logits_in_part_is_refused(lib, dtype):
    """Over them or beside them, not shifted: by an element, a row, all but an element."""
    size = 2 * 100 * (4 if dtype == 0 else 2)
    for off in (4, size // 2, size - 4, -4, -size // 2, 4 - size):
        assert _distill(lib, dtype=dtype, grad=ctypes.c_void_p(0x10000 + off)) == (sv.SPEC_ERR_INVALID_ARG,) * 2
        assert "overlap" in lib.spec_last_error().decode()
