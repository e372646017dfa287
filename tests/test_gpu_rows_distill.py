"""Distillation on the GPU against 64 bits, its gradient also against differences.

Tolerances, from the arithmetic (fp32; eps = 2^-24 is half a step):
  weights e = 2^x, x = (s - m) log2(e) / T: the rounding of x moves e by |x| ln 2 * 3 eps relative
  (difference, product, constant), largest against the sum where e |x| is: e |x| <= 0.54 at x = -1.44;
  ex2 adds 2^-22.  A weight is off by at most (4 |x| eps + 4 eps) e <= 2^-21 of the largest weight 1,
  and the sum S (trees and short runs) by 2^-20 relative.
  gradient: (w / T) (P q - p): q's error 2^-20 relative plus 3 |x| eps; p's likewise through its own
  logarithm (|log p| <= 40: 2^-18): together 2^-17 of max(|P q|, p), then the output's rounding,
  finfo(dtype).eps / 2 of the value.
  loss: sum of p (log p - log q): |log p|, |log q| <= L gives 2^-20 L per unit of P.
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



def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(N, V, K, dtype, seed, sigma=3.0, tail=False, T=1.0, offset=0, repeat=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, V), generator=g) * sigma
    flat = torch.zeros(N * V + offset, dtype=dtype, device=DEV)
    flat[offset:] = x.to(dtype).reshape(-1).to(DEV)
    student = flat[offset:].view(N, V)
    teacher = x + torch.randn((N, V), generator=g)
    v, i = torch.topk(teacher, min(K, V), dim=1)
    values, ids = torch.full((N, K), float("-inf")), torch.full((N, K), -1, dtype=torch.int32)
    values[:, : v.shape[1]], ids[:, : v.shape[1]] = v, i.to(torch.int32)
    if repeat:
        ids[:, 1::2] = ids[:, 0::2][:, : ids[:, 1::2].shape[1]]
        ids[:, K // 2:] = ids[:, :1]
    lse = torch.logsumexp(teacher.double() / T, 1).float().to(DEV) if tail else None
    return student, ids.to(DEV).contiguous(), values.to(DEV).contiguous(), lse


def check(x, ids, t, lse, T, w, r, grad=None, up=None):
    """Loss, statistics and gradient of every row against 64 bits."""
    eps_out = torch.finfo(x.dtype).eps / 2
    for b in range(x.shape[0]):
        wb = 1.0 if w is None else float(w[b])
        z = None if lse is None else float(lse[b])
        loss, (m, S), g = ref.distill(host(x[b]), ids[b].cpu().numpy(), host(t[b]), z, T, wb)
        Td = float(np.float32(T))
        if wb == 0:  # an ignored row: zeros, whatever it holds
            assert r is None or (float(r["loss"][b]) == 0 and (r["stats"][b] == 0).all())
            assert grad is None or not grad[b].any()
            continue
        if r is not None:
            assert float(r["stats"][b, 0]) == m
            assert abs(float(r["stats"][b, 1]) - S) <= 2.0 ** -20 * S
            live = ids[b].cpu().numpy() >= 0
            span = (np.abs(host(x[b])).max() + np.abs(np.where(live & np.isfinite(host(t[b])), host(t[b]), 0.0)).max()) / Td + np.log(S + 1) + abs(z or 0.0) + 2
            assert abs(float(r["loss"][b]) - loss) <= 2.0 ** -20 * 2 * span * abs(wb), (b, float(r["loss"][b]), loss)
        if grad is not None:
            scale = 1.0 if up is None else float(up[b])
            q = np.exp((host(x[b]) - m) / Td) / S
            part = abs(scale * wb / Td) * np.maximum(q * 1.5, np.abs(g) / (abs(wb) / Td) + q)
            bound = 2.0 ** -17 * part + eps_out * np.abs(scale * g) * 1.01 + torch.finfo(x.dtype).tiny
            far = np.abs(host(grad[b]) - scale * g)
            assert (far <= bound).all(), (b, int((far - bound).argmax()), far.max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,K,T,tail", [(1, 1, 1.0, False), (2, 3, 1.0, True), (7, 7, 0.5, False), (9, 4, 1.0, True), (257, 20, 2.0, True),
                                        (5003, 64, 1.0, False), (32000, 128, 0.7, True), (50257, 1024, 1.0, True), (131072, 33, 1.0, False)])
def test_loss_and_gradient(V, K, T, tail, dtype):
    N = 9
    x, ids, t, lse = inputs(N, V, K, dtype, V + K, tail=tail, T=T, offset=V % 7)
    w = torch.rand(N, generator=torch.Generator().manual_seed(3)).to(DEV) + 0.25
    w[2], w[5] = 0.0, -0.5
    r = sv.spec_distill(x, ids, t, T, top_lse=lse, row_weight=w, grad=True)
    alone = sv.spec_distill(x, ids, t, T, top_lse=lse, row_weight=w)
    up = torch.rand(N, generator=torch.Generator().manual_seed(4)).to(DEV) - 0.3
    back = sv.spec_distill_backward(x, ids, t, alone["stats"], up, T, top_lse=lse, row_weight=w)
    torch.cuda.synchronize()
    assert int(r["status"][0]) == int(alone["status"][0]) == int(back["status"][0]) == 0
    check(x, ids, t, lse, T, w, r, r["grad"])
    check(x, ids, t, lse, T, w, alone)
    check(x, ids, t, lse, T, w, None, back["grad"], up)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_token_named_twice_counts_twice(dtype):
    x, ids, t, lse = inputs(6, 4099, 40, dtype, 5, tail=True, repeat=True)
    t = t - 3.0
    r = sv.spec_distill(x, ids, t, top_lse=lse, grad=True)
    check(x, ids, t, lse, 1.0, None, r, r["grad"])
    back = sv.spec_distill_backward(x, ids, t, r["stats"], torch.ones(6, device=DEV), top_lse=lse)
    check(x, ids, t, lse, 1.0, None, None, back["grad"])
    again = sv.spec_distill(x, ids, t, top_lse=lse, grad=True)
    assert torch.equal(again["grad"], r["grad"]) and torch.equal(again["loss"], r["loss"])


def test_gradient_against_differences():
    """d loss / d s at a few columns by central differences of the kernel's own loss (fp32, h = 1/32:
    truncation h^2 / 6 |L'''| <= h^2 / 6 = 2^-12.6; rounding 2 * 2^-20 * span / (2 h) <= 2^-20 * 40 * 16 < 2^-10)."""
    x, ids, t, _ = inputs(1, 200, 12, torch.float32, 8, sigma=1.5)
    r = sv.spec_distill(x, ids, t, grad=True)
    cols = [int(c) for c in ids[0, :4]] + [0, 77, 199]
    h = 1.0 / 32
    shifted = x.repeat(2 * len(cols), 1)
    for i, c in enumerate(cols):
        shifted[2 * i, c] += h
        shifted[2 * i + 1, c] -= h
    n = len(shifted)
    loss = host(sv.spec_distill(shifted.contiguous(), ids.repeat(n, 1), t.repeat(n, 1))["loss"])
    for i, c in enumerate(cols):
        assert abs((loss[2 * i] - loss[2 * i + 1]) / (2 * h) - float(r["grad"][0, c])) <= 2.0 ** -9


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,offset", [(4096, 0), (5003, 3)])
def test_in_place(V, offset, dtype):
    """The gradient over the logits: the same bits as beside them."""
    N, K = 14, 30
    x, ids, t, lse = inputs(N, V, K, dtype, 21, tail=True, offset=offset)
    ids[:, 3] = ids[:, 2]
    want = sv.spec_distill(x, ids, t, top_lse=lse, grad=True)
    y = x.clone() if offset == 0 else torch.cat([torch.zeros(offset, dtype=dtype, device=DEV), x.reshape(-1)])[offset:].view(N, V)
    out = dict(loss=torch.empty(N, device=DEV), stats=torch.empty((N, 2), device=DEV), grad=y)
    sv.spec_distill(y, ids, t, top_lse=lse, grad=True, out=out)
    assert torch.equal(y, want["grad"]) and torch.equal(out["loss"], want["loss"])
    up = torch.linspace(-1, 1, N, device=DEV)
    want = sv.spec_distill_backward(x, ids, t, want["stats"], up, top_lse=lse)["grad"]
    z = x.clone()
    sv.spec_distill_backward(z, ids, t, out["stats"], up, top_lse=lse, out=z)
    assert torch.equal(z, want)


def test_gradient_at_another_alignment():
    N, V = 5, 3001
    x, ids, t, lse = inputs(N, V, 10, torch.bfloat16, 2, offset=0)
    flat = torch.full((N * V + 9,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = dict(loss=torch.empty(N, device=DEV), stats=torch.empty((N, 2), device=DEV), grad=flat[1:1 + N * V].view(N, V))
    r = sv.spec_distill(x, ids, t, grad=True, out=out)
    check(x, ids, t, None, 1.0, None, r, r["grad"])
    assert flat[0] == 7 and (flat[1 + N * V:] == 7).all()  # nothing beside the gradient is written


def test_masked_and_empty_rows():
    N, V, K = 8, 6007, 16
    x, ids, t, _ = inputs(N, V, K, torch.float32, 6)
    x[0, ids[0, 0].item()] = float("-inf")         # the teacher's best token is masked: loss +inf
    x[1, 5000:] = float("-inf")
    x[1, ids[1].long()] = 1.0
    x[2] = torch.finfo(torch.float32).min          # all at the type's lowest value: q is uniform
    ids[3] = -1                                    # no teacher
    t[3] = float("nan")                            # what an empty slot holds is not used
    t[4] = float("-inf")                           # a teacher without weight
    ids[5, 3:] = -1
    x[6] = float("nan")                            # ignored below
    t[6] = float("nan")
    ids[7, 2] = V                                  # out of range: left out, with a status bit
    ids[7, 5] = -2
    w = torch.ones(N, device=DEV)
    w[6] = 0.0
    for _ in range(2):
        r = sv.spec_distill(x, ids, t, row_weight=w, grad=True)
        back = sv.spec_distill_backward(x, ids, t, r["stats"], torch.ones(N, device=DEV), row_weight=w)["grad"]
        assert int(r["status"][0]) == sv.DEV_BAD_TOKEN
        assert float(r["loss"][0]) == float("inf")
        for b in range(1, N):
            ok = ids[b] < V
            sub = slice(b, b + 1)
            idb = torch.where(ok, ids[b], -1)[None]
            check(x[sub], idb, torch.nan_to_num(t[sub], nan=0.0, neginf=float("-inf")), None, 1.0, w[sub],
                  dict(loss=r["loss"][sub], stats=r["stats"][sub]), r["grad"][sub])
            check(x[sub], idb, torch.nan_to_num(t[sub], nan=0.0, neginf=float("-inf")), None, 1.0, w[sub], None, back[sub], torch.ones(1))
        assert (r["grad"][3] == 0).all() and (r["grad"][4] == 0).all() and (r["grad"][6] == 0).all()
        assert torch.isfinite(r["grad"][0]).all()


def test_nonfinite_rows_leave_the_others():
    N, V, K = 7, 4000, 8
    x, ids, t, lse = inputs(N, V, K, torch.bfloat16, 6, tail=True)
    x[1, 9] = float("nan")
    x[2, 3999] = float("inf")
    x[3] = float("-inf")
    t[4, 2] = float("nan")
    lse[5] = float("inf")
    r = sv.spec_distill(x, ids, t, top_lse=lse, grad=True)
    assert int(r["status"][0]) == sv.DEV_NONFINITE
    back = sv.spec_distill_backward(x, ids, t, r["stats"], torch.ones(N, device=DEV), top_lse=lse)
    assert int(back["status"][0]) == sv.DEV_NONFINITE
    for b in range(1, 6):
        assert torch.isnan(r["loss"][b]) and torch.isnan(r["stats"][b]).all()
        assert torch.isnan(r["grad"][b]).all() and torch.isnan(back["grad"][b]).all()
    for b in (0, 6):
        sub = slice(b, b + 1)
        check(x[sub], ids[sub], t[sub], lse[sub], 1.0, None, dict(loss=r["loss"][sub], stats=r["stats"][sub]), r["grad"][sub])


def test_capture_and_other_stream():
    N, V, K = 33, 9001, 50
    x, ids, t, lse = inputs(N, V, K, torch.bfloat16, 16, tail=True)
    want = sv.spec_distill(x, ids, t, top_lse=lse, grad=True)
    out = dict(loss=torch.empty(N, device=DEV), stats=torch.empty((N, 2), device=DEV), grad=torch.empty_like(x))
    status, back = torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty_like(x)
    up = torch.full((N,), 2.0, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_distill(x, ids, t, top_lse=lse, grad=True, out=out, status=status)
        sv.spec_distill_backward(x, ids, t, out["stats"], up, top_lse=lse, out=back, status=status)
    for _ in range(2):
        out["grad"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["grad"], want["grad"]) and torch.equal(out["loss"], want["loss"]) and int(status[0]) == 0
    check(x, ids, t, lse, 1.0, None, None, back, up)
    other = sv.spec_distill(x, ids, t, top_lse=lse, grad=True, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(other["grad"], want["grad"])


def test_from_target_rows_to_a_step_of_the_draft():
    """The operators as they are used together: a verify's target rows are sampled under a request's
    filters and kept as a teacher's largest logits; the draft's rows are trained on them, its
    gradient going on through torch's own graph; the step brings the draft nearer the target."""
    B, K, V, D = 6, 3, 4007, 64
    gen = torch.Generator(device=DEV).manual_seed(2)
    target = torch.randn((B, K + 1, V), generator=gen, device=DEV) * 3
    hidden = torch.randn((B * K, D), generator=gen, device=DEV)
    head = (torch.randn((V, D), generator=gen, device=DEV) * 0.3).requires_grad_(True)
    rows = target[:, :K].reshape(B * K, V).contiguous()
    teacher = sv.spec_top_logits(rows, 64, lse=True)
    draft = hidden @ head.t()
    u = torch.rand(B * K, generator=gen, device=DEV)
    tokens = sv.spec_sample_filtered(draft.detach(), u, torch.ones(B * K, device=DEV))["tokens"]
    assert torch.equal(tokens, sv.spec_sample_rows(draft.detach(), u, 1.0)["tokens"])
    ver = sv.spec_verify_linear(target, draft.detach().view(B, K, V), tokens.view(B, K),
                                torch.rand((B, K), generator=gen, device=DEV), torch.rand(B, generator=gen, device=DEV), 1.0)
    assert int(ver["status"][0]) == 0
    w = torch.full((B * K,), 1.0 / (B * K), device=DEV)
    r = sv.spec_distill(draft.detach(), teacher["ids"], teacher["values"], top_lse=teacher["lse"], row_weight=w, grad=True)
    draft.backward(r["grad"])
    check(draft.detach(), teacher["ids"], teacher["values"], teacher["lse"], 1.0, w, r, r["grad"])
    want = host(r["grad"]).T @ host(hidden)
    got = host(head.grad)
    assert np.linalg.norm(got - want) <= 2.0 ** -8 * np.linalg.norm(want)  # torch's product may be in tf32


def test_offsets_past_32_bits():
    N, V, K = 17000, 131072, 4                      # 4.5 GB of bf16
    x = torch.zeros((N, V), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((N, K), dtype=torch.int32, device=DEV)
    t = torch.zeros((N, K), device=DEV)
    last, i, v, _ = inputs(1, V, K, torch.bfloat16, 4)
    x[-1], ids[-1], t[-1] = last[0], i[0], v[0]
    w = torch.zeros(N, device=DEV)
    w[-1] = 1.0
    out = dict(loss=torch.empty(N, device=DEV), stats=torch.empty((N, 2), device=DEV), grad=x)
    r = sv.spec_distill(x, ids, t, row_weight=w, grad=True, out=out)
    check(last, i, v, None, 1.0, None, dict(loss=r["loss"][-1:], stats=r["stats"][-1:]), x[-1:])
    assert (r["loss"][:-1] == 0).all() and not x[:-1].any()


def test_a_masked_teacher_row_and_the_longest_rows():
    """spec_top_logits of a masked row is a teacher without tokens: (-1, -inf, lse -inf)."""
    for dtype, V in ((torch.float32, 262144), (torch.bfloat16, 524288), (torch.bfloat16, 3001)):
        x, _, _, _ = inputs(3, V, 4, dtype, 9)
        teacher = (x + 0.5).clone()
        teacher[1] = float("-inf")
        top = sv.spec_top_logits(teacher, 40, lse=True, temperature=0.9)
        r = sv.spec_distill(x, top["ids"], top["values"], 0.9, top_lse=top["lse"], grad=True)
        back = sv.spec_distill_backward(x, top["ids"], top["values"], r["stats"], torch.ones(3, device=DEV), 0.9, top_lse=top["lse"])["grad"]
        assert int(r["status"][0]) == 0
        assert float(r["loss"][1]) == 0 and not r["grad"][1].any() and not back[1].any()
        for b in (0, 2):
            sub = slice(b, b + 1)
            check(x[sub], top["ids"][sub], top["values"][sub], top["lse"][sub], 0.9, None, dict(loss=r["loss"][sub], stats=r["stats"][sub]), r["grad"][sub])
            check(x[sub], top["ids"][sub], top["values"][sub], top["lse"][sub], 0.9, None, None, back[sub], torch.ones(1))


@pytest.mark.parametrize("N,V,dtype", [(700, 33000, torch.bfloat16), (1300, 2051, torch.float32), (260, 70001, torch.bfloat16)])
def test_many_rows_with_ignored_ones_between(N, V, dtype):
    """More rows than clusters are resident: each takes several, skipping ignored ones; odd rows, so that
    neighbours share vectors; in place."""
    x, ids, t, lse = inputs(N, V, 12, dtype, N, tail=True)
    w = (torch.rand(N, generator=torch.Generator().manual_seed(1)) < 0.6).float().to(DEV) * 0.5
    w[-3:] = 0
    y = x.clone()
    r = sv.spec_distill(x, ids, t, top_lse=lse, row_weight=w, grad=True)
    out = dict(loss=torch.empty(N, device=DEV), stats=torch.empty((N, 2), device=DEV), grad=y)
    sv.spec_distill(y, ids, t, top_lse=lse, row_weight=w, grad=True, out=out)
    assert torch.equal(y, r["grad"]) and torch.equal(out["loss"], r["loss"]) and torch.equal(out["stats"], r["stats"])
    pick = [int(b) for b in np.random.RandomState(0).choice(N, 25, replace=False)] + [0, 1, N - 4, N - 1]
    i = torch.tensor(pick, device=DEV)
    check(x[i], ids[i], t[i], lse[i], 1.0, w[i], dict(loss=r["loss"][i], stats=r["stats"][i]), r["grad"][i])
    # every row's gradient sums to w (P - P) = 0 but for rounding: at most 2^-8 of the summed sizes, 2 w = 1
    assert r["grad"].float().sum(1).abs().max() <= 2.0 ** -8


@pytest.mark.parametrize("split", [False, True])
def test_gradient_of_large_logits(split):
    """Logits around 200, where the maximum times log2 e rounds by up to 2^-16: the columns without a
    teacher's entry, against 64 bits.  Those within 4 octaves of the maximum are off by at most 4 |x|
    halves of 2^-23 ln 2 (l c, its c) and 4 of 2^-24 (ex2.approx) in the weight, as much in the
    exp-sum, and 6 more of 2^-24 in sums and products: 32 of 2^-24 in all."""
    V, K = 1501, 3
    g = torch.Generator().manual_seed(33)
    x = (torch.rand((8, V), generator=g) * 2.5 + 198.7).to("cuda:0")
    ids = torch.randint(0, V, (8, K), generator=g, dtype=torch.int32).to("cuda:0")
    t = torch.randn((8, K), generator=g).to("cuda:0")
    r = sv.spec_distill(x, ids, t, grad=not split)
    grad = r["grad"] if not split else sv.spec_distill_backward(x, ids, t, r["stats"], torch.ones(8, device="cuda:0"))["grad"]
    q = torch.softmax(x.double(), 1)
    q.scatter_(1, ids.long(), 0.0)
    grad = grad.double().scatter_(1, ids.long(), 0.0)
    off = ((grad - q).abs() / q.clamp(min=1e-30)).max().item()
    assert off < 32 * 2.0 ** -24, off / 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_an_ignored_row_whatever_its_upstream_gradient(dtype):
    """Padding rows (weight 0) under a loss scale that overflowed; and a zero upstream gradient of any weight."""
    N, V, K = 9, 3001, 12
    x, ids, t, lse = inputs(N, V, K, dtype, 31, tail=True)
    x[1], t[2], lse[3] = float("nan"), float("nan"), float("inf")
    w = torch.ones(N, device=DEV)
    w[[1, 2, 3, 4]] = 0.0
    w[4] = -0.0
    up = torch.ones(N, device=DEV)
    up[1], up[2], up[3], up[4] = float("inf"), float("nan"), float("-inf"), float("nan")
    up[6], w[7], up[7] = 0.0, float("inf"), 0.0
    finite = torch.where(torch.isfinite(w), w, 1.0)
    r = sv.spec_distill(x, ids, t, top_lse=lse, row_weight=finite)
    assert int(r["status"][0]) == 0
    back = sv.spec_distill_backward(x, ids, t, r["stats"], up, top_lse=lse, row_weight=w)
    assert int(back["status"][0]) == 0
    assert not back["grad"][[1, 2, 3, 4, 6, 7]].any()
    for b in (0, 5, 8):
        sub = slice(b, b + 1)
        check(x[sub], ids[sub], t[sub], lse[sub], 1.0, None, None, back["grad"][sub], up[sub])
