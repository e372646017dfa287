"""Filtered sampling at borders that whole units of weight are too coarse for."""
import numpy as np
import pytest
import torch

import sampling_online_softmax_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("V,k,u", [(1000, 0, 1 - 2.0 ** -24), (262144, 0, 0.99999), (262144, 1000, 1 - 2.0 ** -24), (262144, 5000, 1 - 2.0 ** -22)])
def test_min_p_next_to_a_long_tail(V, k, u):
    """One token ahead of a tail of equal ones whose weight, 10^-10 of its own, lies 2^-13 of itself above
    or below min-p: kept, the tail has the mass that u asks for; else the draw is the first token's."""
    B = 64
    g = torch.Generator().manual_seed(V + k)
    low = -(22.5 + torch.rand((B,), generator=g))
    w = np.exp(low.numpy().astype(np.float64))
    kept = np.arange(B) % 2 == 0
    mp = (w * np.where(kept, 1 - 2.0 ** -13, 1 + 2.0 ** -13)).astype(np.float32)
    assert ((mp <= w) == kept).all()
    x = low.unsqueeze(1).repeat(1, V)
    x[:, 7] = 0.0
    tail = (k or V) - 1
    # u W > 1 (token 7, which 7 of the tail's come before) where the tail is kept; the token is then well inside the tail
    t = float(np.float32(u)) * (1 + tail * w)
    assert ((t - 1) / w > 8).all()
    c = np.floor((t - 1) / w).astype(np.int64)  # tail tokens before the drawn one
    far = (t - 1) / w - c
    x = x.to(DEV)
    one = torch.ones(B, device=DEV)
    top_k = torch.full((B,), k, dtype=torch.int32, device=DEV)
    got = sv.spec_sample_filtered(x, one * u, one, top_k=top_k, min_p=torch.tensor(mp, device=DEV))["tokens"].tolist()
    for b in range(B):
        if not kept[b]:
            assert got[b] == 7, (b, got[b])
        else:  # whole units of the tail's weights are off by 0.8 each: a place in the tail by that share of its length
            units = w[b] * 2.0 ** min(48, 62 - (V - 1).bit_length())
            assert abs(got[b] - (c[b] + 1 + far[b])) <= 2 + tail * 0.8 / units, (b, got[b], c[b])


@pytest.mark.parametrize("V", [300, 6000, 60001])
@pytest.mark.parametrize("top", [30.0, 60.0, 85.0])
def test_min_p_far_below_the_largest(V, top):
    """The same at u = 0, down to weights of 10^-37: the first token is drawn where its weight reaches min-p."""
    B = 64
    g = torch.Generator().manual_seed(V)
    low = -(top + torch.rand((B,), generator=g))
    w = np.exp(low.numpy().astype(np.float64))
    mp = w.astype(np.float32)  # the nearest fp32, above the weight or below it
    keep = mp <= w
    assert (np.abs(mp / w - 1) > 2.0 ** -35).all() and keep.sum() > 8 and (~keep).sum() > 8
    x = torch.full((B, V), -200.0)
    x[:, 0] = low
    x[:, V // 2] = 0.0
    x = x.to(DEV)
    one = torch.ones(B, device=DEV)
    for kw in (dict(), dict(top_k=torch.full((B,), 5, dtype=torch.int32, device=DEV)), dict(top_k=torch.full((B,), 2000, dtype=torch.int32, device=DEV))):
        r = sv.spec_sample_filtered(x, one * 0.0, one, min_p=torch.tensor(mp, device=DEV), **kw)
        assert int(r["status"][0]) == 0
        assert r["tokens"].tolist() == [0 if a else V // 2 for a in keep]


@pytest.mark.parametrize("n,p", [(64, 0.5), (64, 0.25), (40, 0.625), (200, 0.5), (1000, 0.75), (3000, 0.5)])
@pytest.mark.parametrize("T", [1e-6, 1e-4, 0.01])
def test_top_p_on_the_border_between_equal_logits(T, n, p):
    """n equal tokens, of which top-p keeps n p exactly, at maxima over T of up to 10^9: the last kept one is drawn
    only if the bounds of the row's weight hold to their last place."""
    B, V = 96, 9001
    g = torch.Generator().manual_seed(n)
    m = torch.logspace(-2, 3, B)
    x = -torch.rand((B, V), generator=g) * 1000 - 100 - 2 * m.unsqueeze(1)
    at = torch.stack([torch.randperm(V, generator=g)[:n].sort().values for _ in range(B)])
    x.scatter_(1, at, m.unsqueeze(1).expand(B, n))
    x = x.to(DEV)
    one = torch.ones(B, device=DEV)
    r = sv.spec_sample_filtered(x, one * (1 - 2.0 ** -24), one * T, top_p=one * p)
    assert int(r["status"][0]) == 0
    assert r["tokens"].tolist() == at[:, int(n * p) - 1].tolist()


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 524288), (torch.float32, 262144), (torch.bfloat16, 131072), (torch.float32, 32000)])
def test_a_long_tail_of_equal_tokens(V, dtype):
    """One token far ahead of a tail of equal ones, down to a unit of weight each, whose rounding adds up:
    the drawn token's interval holds u W to within 2^-37 W + 0.8 V units of 2^-U."""
    bits = (V - 1).bit_length()
    unit = 2.0 ** -min(48, 62 - bits)
    low = [float(torch.tensor(l).to(dtype)) for l in (np.log(1.49 * unit), np.log(1.51 * unit), np.log(0.6 * unit), np.log(30.3 * unit), -21.0, -14.0, -9.3)]
    x = torch.tensor(low).unsqueeze(1).repeat(1, V)
    ahead = V // 3
    x[:, ahead] = 0.0
    x = x.to(dtype).to(DEV)
    w = np.exp(np.array(low))
    B = len(low)
    one = torch.ones(B, device=DEV)
    for u in (1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -18, 0.6, 2.0 ** -26, 2.0 ** -40):
        for kw in (dict(), dict(top_p=one * (1 - 2.0 ** -24))):
            r = sv.spec_sample_filtered(x, one * u, one, **kw)
            assert int(r["status"][0]) == 0
            for b, tok in enumerate(r["tokens"].tolist()):
                n, off = V - 1, 2.0 ** -37 * (1 + (V - 1) * w[b]) + 0.8 * V * unit
                if kw:  # the token ahead and the first n others, the fewest with that share; n may be a token and `off` off
                    n = max(0, int(np.ceil(((1 - 2.0 ** -24) * (1 + n * w[b]) - 1) / w[b])))
                    off = 2 * off + 2 * w[b]
                W = 1 + n * w[b]
                start = tok * w[b] if tok < ahead else min(n, ahead) * w[b] if tok == ahead else (tok - 1) * w[b] + 1
                end = start + (1.0 if tok == ahead else w[b])
                t = float(np.float32(u)) * W
                assert start - off <= t <= end + off, (b, u, bool(kw), tok, start, t, end, off)


@pytest.mark.parametrize("V", [100, 5000, 70001])
def test_the_smallest_weights_at_a_zero_uniform(V):
    """Weights of 2^-1075 to 2^-1074 are not 0 in 64 bits, smaller ones are: the first that is not is drawn."""
    low = np.float32([-744.5, -744.8, -745.0, -745.1, -745.2, -746.0, -800.0])
    x = torch.zeros((len(low), V))
    x[:, 0] = torch.tensor(low)
    one = torch.ones(len(low), device=DEV)
    x = x.to(DEV)
    want = [0 if w > 0 else 1 for w in np.exp(low.astype(np.float64))]
    assert want == [0, 0, 0, 0, 1, 1, 1]
    for kw in (dict(), dict(top_p=one * 0.999999), dict(top_k=torch.full((len(low),), V, dtype=torch.int32, device=DEV))):
        assert sv.spec_sample_filtered(x, one * 0.0, one, **{n: v for n, v in kw.items() if n != "top_p"})["tokens"].tolist() == want
