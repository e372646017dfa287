"""Distillation where the largest logit over T is far from 0: finite masks, small and large
temperatures, large logits; against the definition in 64 bits.

Tolerances, from the arithmetic (fp32, eps = 2^-24 half a step; d = |s - m| / T):
  a weight e^-d: its exponent d log2 e comes of a difference, a product and a constant that is the
  quotient of a rounded log2 e and T (4 eps relative), ex2 adds 2^-22:  (4 eps d + 2^-22) relative.
  S: the weights' errors, 4 eps E[d] + 2^-22 with E over q; its sums, at most 50 of them deep (80
  vectors a thread in batches of four, eight logits a vector, warp, row), and the 20 batches' new
  maxima, ex2's 2^-22 = 4 eps each, half of them on the mean: 50 + 40 eps, and 10 for the warps' and the row's.
  p: log p comes of a difference, a product with a rounded 1 / T and log of the sum over at most 1024
  entries (4 eps |log p| + 30 eps), expf adds 2^-22; with a log-normaliser t / T - lse is one rounding
  of its value.  So 4 eps |log p| + 2^-18 relative.
  gradient (w / T) (P q - p): the relative errors of P q and of p, 8 eps for products, then the
  output's rounding; results below fp32's normal numbers may be 0.
  loss sum p (log p - log q): p's relative error (and the sum's, of up to 1024) times |log p - log q|,
  and p (5 eps |log p| + 5 eps |log q| + S's + 30 eps).
"""
import numpy as np
import pytest
import torch

import sampling_online_softmax_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 2.0 ** -24


def exact(x, ids, t, lse, T, w):
    """(loss, m, S, gradient) and the tolerances of loss, S and gradient, in 64 bits."""
    x64, t64, T = x.double(), torch.where(ids >= 0, t.double(), -np.inf), float(np.float32(T))
    m = x64.amax(1, keepdim=True)
    d = (m - x64) / T
    e = torch.exp(-d)
    S = e.sum(1, keepdim=True)
    q = e / S
    logp = (t64 - t64.amax(1, keepdim=True)) / T
    logp = logp - torch.log(torch.exp(logp).sum(1, keepdim=True)) if lse is None else t64 / T - lse.double().unsqueeze(1)
    p = torch.exp(logp)
    logp = torch.where(p > 0, logp, 0.0)
    at = ids.clamp(min=0).long()
    logq = -d.gather(1, at) - torch.log(S)
    w64 = w.double()
    loss = w64 * torch.where(p > 0, p * (logp - logq), 0.0).sum(1)
    target = torch.zeros_like(x64).scatter_add_(1, at, p)
    P = p.sum(1, keepdim=True)
    grad = w64.unsqueeze(1) / T * (P * q - target)
    far_S = 4 * EPS * (q * torch.where(q > 0, d, 0.0)).sum(1) + 2.0 ** -22 + 100 * EPS
    far_p = 4 * EPS * logp.abs() + 2.0 ** -18
    terms = far_p * (logp - logq).abs() + 5 * EPS * (logp.abs() + logq.abs()) + far_S.unsqueeze(1) + 30 * EPS
    far_loss = w64.abs() * torch.where(p > 0, p * terms, 0.0).sum(1) + 1e-37
    far_q = 4 * EPS * torch.where(q > 0, d, 0.0) + 2.0 ** -22 + far_S.unsqueeze(1) + 8 * EPS
    far_P = torch.where(p > 0, p * far_p, 0.0).sum(1, keepdim=True)
    far_t = torch.zeros_like(x64).scatter_add_(1, at, torch.where(p > 0, p * (far_p + 8 * EPS), 0.0))
    scale = (w64.abs() / T).unsqueeze(1)
    far_grad = scale * (q * (P * far_q + far_P) + far_t) + grad.abs() * torch.finfo(x.dtype).eps / 2 * 1.01
    far_grad += 2 * torch.finfo(torch.float32).tiny * (1 + scale * (P + 1))
    return (loss, m.squeeze(1), S.squeeze(1), grad), (far_loss, far_S * S.squeeze(1), far_grad)


def check(x, ids, t, lse=None, T=1.0, w=None):
    """The loss alone, loss and gradient in one call, and the gradient alone."""
    N = x.shape[0]
    one = torch.ones(N, device=DEV)
    fused = sv.spec_distill(x, ids, t, T, top_lse=lse, row_weight=w, grad=True)
    alone = sv.spec_distill(x, ids, t, T, top_lse=lse, row_weight=w)
    back = sv.spec_distill_backward(x, ids, t, alone["stats"], one, T, top_lse=lse, row_weight=w)
    (loss, m, S, grad), (far_loss, far_S, far_grad) = exact(x, ids, t, lse, T, one if w is None else w)
    for name, r in (("fused", fused), ("alone", alone)):
        assert int(r["status"][0]) == 0, name
        assert torch.equal(r["stats"][:, 0].double(), m), name
        off = (r["stats"][:, 1].double() - S).abs()
        assert (off <= far_S).all(), (name, "S", (off / S).max().item())
        off = (r["loss"].double() - loss).abs()
        assert (off <= far_loss).all(), (name, "loss", (off / far_loss).max().item())
    assert int(back["status"][0]) == 0
    for name, g in (("fused", fused["grad"]), ("backward", back["grad"])):
        off = (g.double() - grad).abs()
        assert (off <= far_grad).all(), (name, "grad", (off / far_grad).max().item())


def teacher(x, K, T, seed, spread=1.0):
    """The K largest of the rows plus noise of `spread` T, as a teacher's."""
    g = torch.Generator().manual_seed(seed)
    values, ids = torch.topk(x.float().cpu() + torch.randn(x.shape, generator=g) * spread * T, min(K, x.shape[1]), dim=1)
    return ids.to(torch.int32).to(DEV).contiguous(), values.float().to(DEV).contiguous()


FILLS = [-1e4, -1e9, -1e10, -1e12, -1e20, -1e30]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [300, 5003, 70001])
@pytest.mark.parametrize("fill", FILLS)
def test_finite_masks(fill, V, dtype):
    """Masked by a finite number: in blocks that are a thread's first vectors, everywhere but for a few
    tokens, and whole rows."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn((8, V), generator=g) * 3
    x[1, : V // 2] = fill
    x[2, V // 2:] = fill
    x[3, ::2] = fill
    x[4][torch.rand(V, generator=g) < 0.97] = fill
    x[5, 8:] = fill
    x[6] = fill
    x[7, : V - 9] = fill
    x[7, V - 9:] = 200.0
    x = x.to(dtype).to(DEV)
    ids, t = teacher(torch.where(x > -1e3, x, torch.full_like(x, -300.0)), 5, 1.0, V)
    check(x, ids, t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1e-6, 1e-4, 1e-2, 30.0, 1e6])
def test_temperatures(T, dtype):
    """Rows around 19.7 whose logits differ by a few T or by a few steps of the type, and random ones."""
    V = 9001
    g = torch.Generator().manual_seed(3)
    step = max(float(np.float32(T)), 2.0 ** -19 if dtype == torch.float32 else 2.0 ** -3)
    x = torch.cat([19.7 - step * torch.randint(0, 7, (3, V), generator=g), torch.full((1, V), 19.7), -19.7 + step * torch.randn((3, V), generator=g),
                   torch.randn((3, V), generator=g) * 3]).to(dtype).to(DEV)
    w = torch.linspace(-1.0, 2.0, len(x)).to(DEV)
    ids, t = teacher(x, 33, T, 4)
    check(x, ids, t, T=T, w=w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [300.0, 2839.0, 1e4, 1e5, 1e6, 3e7, 1e15])
def test_large_logits(size, dtype):
    """Logits that differ by up to 8 (or by steps of the type) around +-size; rising and falling along the row,
    so that the running maximum moves in every batch; and rows of both signs."""
    V = 20011
    g = torch.Generator().manual_seed(5)
    eps = torch.finfo(dtype).eps
    step = max(1.0, size * eps / 2)
    near = step * torch.randint(0, 9, (2, V), generator=g)
    rise = torch.linspace(0.0, 8.0 * step, V)
    x = torch.stack([size + near[0], -size + near[1], size + rise, -size - rise, size - rise, -size + rise,
                     (torch.rand(V, generator=g) * 2 - 1) * size, torch.where(torch.rand(V, generator=g) < 0.5, size, -size)])
    x = x.to(dtype).to(DEV)
    ids, t = teacher(x, 17, 1.0, 6)
    check(x, ids, t)


def test_running_maxima_across_sizes():
    """A thread's maximum climbs over many orders of size, from far below 0 to far above it."""
    V = 60000
    up = torch.cat([-torch.logspace(30, 0, V // 2), torch.logspace(-2, 3.6, V // 2)])
    rows = [up, -up.flip(0), torch.linspace(-6000, 6000, V), torch.linspace(2830, 2850, V), torch.linspace(-2850, -2830, V),
            torch.linspace(-2839.2, -2839.1, V), torch.linspace(2839.1, 2839.4, V)]
    x = torch.stack(rows).to(DEV)
    ids, t = teacher(x, 9, 1.0, 7)
    check(x, ids, t)


@pytest.mark.parametrize("T", [1e-6, 1e-4, 1e-2, 0.3, 1e6])
def test_a_log_normaliser_of_large_logits(T):
    """p = exp(t / T - lse) where t / T is large and the difference a few units."""
    V, K = 5003, 40
    g = torch.Generator().manual_seed(12)
    step = max(float(np.float32(T)), 2.0 ** -19)
    x = (19.7 - step * torch.randint(0, 7, (6, V), generator=g)).to(DEV)
    ids, t = teacher(x, K, T, 13)
    t[:, 7] = torch.finfo(torch.float32).min  # (over T, nothing or -inf)
    whole = torch.logsumexp(t.double() / float(np.float32(T)), 1)
    lse = (whole + 0.3).float()
    check(x, ids, t, lse=lse, T=T)
