"""The operators on rows of logits over seeded random calls, against their definitions in 64 bits (torch):
types, lengths, alignments, spreads, ties, masks by -inf and by finite numbers, temperatures from
10^-6 to 10^6, every mixture of filters.

Tokens are equal but where u W, top-p's share or min-p lies within the stated bound of a border: 2^-37 W
+ 0.8 V units, units of 2^-min(48, 62 - ceil(log2 V)), twice over (the cut and the draw), and 2^-36 of
min-p; these rows are left out, and few.  Largest logits are equal, ids too; the log-normaliser is
fp32's: 4 roundings of its value, and its sum's 2^-19.  Distillation as in test_gpu_distill_magnitudes.py.
"""
import random

import numpy as np
import pytest
import torch

import sampling_online_softmax_gb300 as sv
import test_gpu_distill_magnitudes as distill

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def memory_given_back():
    yield
    torch.cuda.empty_cache()


def logits(rng, gen, B, V, dtype):
    """Rows of one of several kinds, at a random alignment."""
    size = 10 ** rng.uniform(-2, 1.2)
    x = torch.randn((B, V), generator=gen, device=DEV) * size
    kind = rng.choice(["plain", "plain", "ties", "levels", "ramp", "ahead", "equal"])
    if kind == "ties":
        x = (x / size * rng.choice([2, 8, 40])).round() * (size / 4)
    elif kind == "levels":
        x = torch.where(torch.rand((B, V), generator=gen, device=DEV) < 10 ** rng.uniform(-5, -0.3), 0.0, -rng.uniform(0, 30))
    elif kind == "ramp":
        x = x * 0.1 + torch.linspace(-size, size, V, device=DEV) * rng.choice([-1, 1])
    elif kind == "ahead":
        x.scatter_add_(1, torch.randint(0, V, (B, 1), generator=gen, device=DEV), torch.full((B, 1), rng.uniform(0, 25) * size, device=DEV))
    elif kind == "equal":
        x = torch.full((B, V), rng.choice([0.0, -0.0, 7.25, -100.0, 1e-30]), device=DEV)
    x = x + rng.choice([0.0, 0.0, 0.0, 30.0, -50.0, 300.0, 1e4, -1e6])
    for _ in range(rng.choice([0, 0, 1, 1, 2])):
        fill = rng.choice([-np.inf, -np.inf, -1e4, -1e9, -1e30, torch.finfo(dtype).min])
        if rng.random() < 0.5:
            x = x.masked_fill(torch.rand((B, V), generator=gen, device=DEV) < rng.choice([0.1, 0.5, 0.99]), fill)
        else:
            a, b = sorted(rng.randrange(V + 1) for _ in range(2))
            x[rng.randrange(B):, a:b] = fill
    flat = torch.zeros(B * V + 8, dtype=dtype, device=DEV)
    at = rng.randrange(8)
    flat[at:at + B * V] = x.to(dtype).reshape(-1)
    return flat[at:at + B * V].view(B, V)


def sizes(rng, most=3 << 20):
    V = max(1, int(10 ** rng.uniform(0, 5.3)))
    if rng.random() < 0.3:
        V = max(1, V // 1024 * 1024 + rng.choice([-1, 0, 1]))
    return max(1, min(int(10 ** rng.uniform(0, 3)), most // V)), V


def temperature(rng):
    return rng.choice([1.0, 1.0, rng.uniform(0.3, 1.5), rng.uniform(0.3, 1.5), rng.uniform(0.3, 1.5), 10 ** rng.uniform(-6, 6), 1e-6, 1e6])


def tokens(x, u, T, k, p, mp):
    """(tokens, whether they are clear of every border) of each row, -1 for rows that hold no logit."""
    B, V = x.shape
    x64, T64 = x.double(), T.double().unsqueeze(1)
    m = x64.amax(1, keepdim=True)
    empty = m.squeeze(1) == -np.inf
    w = torch.exp((x64 - torch.where(m == -np.inf, 0.0, m)) / torch.where(T64 == 0, 1.0, T64))
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device=DEV).unsqueeze(0)
    live = x64.gather(1, order) > -np.inf
    k = k.unsqueeze(1)
    live &= (k <= 0) | (rank < k)
    ws = torch.where(live, ws, 0.0)
    unit = 0.8 * V * 2.0 ** -min(48, 62 - max(1, (V - 1).bit_length()))
    mass = ws.cumsum(1)
    total = mass[:, -1:]
    far = 2.0 ** -37 * total + unit
    p64 = p.double().unsqueeze(1)
    keep = live & ((p64 >= 1) | (rank == 0) | (mass - ws < p64 * total))
    clear = ((p64 >= 1) | (p64 == 0) | ((mass - p64 * total).abs() > far)).all(1)
    clear |= (p64 < 1).squeeze(1) & (mass[:, 0] > (p64 * total + far).squeeze(1))  # (the first token alone has the share)
    mp64 = mp.double().unsqueeze(1)
    keep &= ws >= mp64
    clear &= ((mp64 == 0) | ~live | ((ws / torch.where(mp64 == 0, 1.0, mp64) - 1).abs() > 2.0 ** -36)  | (rank == 0)).all(1)
    keep &= (T64 > 0) | (rank == 0)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    c = torch.where(kept, w, 0.0).cumsum(1)
    W = c[:, -1:]
    t = u.double().unsqueeze(1) * W
    tok = (c <= t).sum(1).to(torch.int32)
    one = keep.sum(1) == 1
    near = ((c - t).abs() <= 2.0 ** -37 * W + unit) & (c < W) & (c > 0)
    clear &= one | (t == 0).squeeze(1) | ~(near.any(1) | (W - t <= 2.0 ** -37 * W + unit).squeeze(1))
    greedy = (T == 0) | (k.squeeze(1) == 1)
    return torch.where(empty, -1, torch.where(greedy, order[:, 0].to(torch.int32), tok)), clear | greedy | empty


def sampling_case(seed):
    rng, gen = random.Random(seed), torch.Generator(device=DEV).manual_seed(seed)
    B, V = sizes(rng)
    dtype = rng.choice([torch.float32, torch.bfloat16])
    x = logits(rng, gen, B, V, dtype)

    def per_row(pick, none, dt):
        v = [pick()] * B if rng.random() < 0.5 else [pick() if i < 40 else none for i in range(B)]
        return torch.tensor(v, dtype=dt).to(DEV)

    k = per_row(lambda: rng.choice([0, 0, -3, 1, 5, 50, 1000, 1024, 1025, 5000, V, V + 1, max(1, V // 2)]), 0, torch.int32)
    p = per_row(lambda: rng.choice([1.0, 1.0, rng.random(), rng.random(), 0.95, 0.999, 1 - 2.0 ** -20, 0.0, 1e-6]), 1.0, torch.float32)
    mp = per_row(lambda: rng.choice([0.0, 0.0, 0.0, rng.random(), 0.05, 1e-5, 10 ** rng.uniform(-38, 0), 1.0]), 0.0, torch.float32)
    T = per_row(lambda: rng.choice([0.0] + [temperature(rng) for _ in range(9)]), 0.7, torch.float32)
    u = torch.rand(B, generator=gen, device=DEV)
    u[torch.rand(B, generator=gen, device=DEV) < 0.05] = rng.choice([0.0, 1 - 2.0 ** -24, 2.0 ** -30])
    named = dict(top_k=k, top_p=p, min_p=mp)
    none = dict(top_k=torch.zeros_like(k), top_p=torch.ones_like(p), min_p=torch.zeros_like(mp))
    left = [n for n in named if rng.random() < 0.3]
    got = sv.spec_sample_filtered(x, u, T, **{n: v for n, v in named.items() if n not in left})
    want, clear = tokens(x, u, T, *(none[n] if n in left else named[n] for n in ("top_k", "top_p", "min_p")))
    assert int(got["status"][0]) == (sv.DEV_NONFINITE if (want < 0).any() else 0)
    wrong = (got["tokens"] != want) & clear
    assert not wrong.any(), (seed, dict(B=B, V=V, dtype=dtype, rows=wrong.nonzero()[:5, 0].tolist()), got["tokens"][wrong][:5].tolist(), want[wrong][:5].tolist(),
                             {n: v[wrong][:5].tolist() for n, v in dict(named, T=T, u=u).items() if n not in left})
    return B, int((~clear).sum())


def test_sampling():
    rows, open_rows = map(sum, zip(*[sampling_case(1000 + i) for i in range(1000)]))
    assert open_rows <= 0.05 * rows, (rows, open_rows)  # (rows of equal logits share their borders: whole calls of them)


def top_case(seed):
    rng, gen = random.Random(seed), torch.Generator(device=DEV).manual_seed(seed)
    B, V = sizes(rng)
    x = logits(rng, gen, B, V, rng.choice([torch.float32, torch.bfloat16]))
    k, T = rng.choice([1, 2, 8, 64, 65, rng.randrange(1, 1025), 1024]), float(np.float32(temperature(rng)))
    r = sv.spec_top_logits(x, k, temperature=T, lse=True)
    assert int(r["status"][0]) == 0
    value, order = torch.sort(x.float(), dim=1, descending=True, stable=True)
    n = min(k, V)
    value, ids = value[:, :n], torch.where(value[:, :n] > -np.inf, order[:, :n], -1).to(torch.int32)
    assert torch.equal(r["values"][:, :n], value) and torch.equal(r["ids"][:, :n], ids), (seed, B, V, k)
    assert (r["values"][:, n:] == -np.inf).all() and (r["ids"][:, n:] == -1).all()
    x64 = x.double()
    m = x64.amax(1)
    lse = m / T + torch.log(torch.exp((x64 - m.clamp(min=-3.5e38).unsqueeze(1)) / T).sum(1))
    lse = torch.where(m == -np.inf, -np.inf, lse)
    got = r["lse"].double()
    far = 4 * 2.0 ** -24 * lse.abs() + 2.0 ** -19
    top = torch.finfo(torch.float32).max
    good = (got == lse) | ((got - lse).abs() <= far) | ((lse.abs() > top * (1 - 2.0 ** -20)) & (got == torch.copysign(torch.full_like(got, np.inf), lse)))
    assert good.all(), (seed, B, V, T, got[~good][:4].tolist(), lse[~good][:4].tolist())


def test_largest_logits():
    for i in range(400):
        top_case(100000 + i)


def distill_case(seed):
    rng, gen = random.Random(seed), torch.Generator(device=DEV).manual_seed(seed)
    B, V = sizes(rng)
    T = float(np.float32(temperature(rng)))
    x = logits(rng, gen, B, V, rng.choice([torch.float32, torch.bfloat16]))
    x = torch.where((x > -np.inf).any(1, keepdim=True), x, 0.0).to(x.dtype)
    k = rng.choice([1, 3, 20, 64, 256, 257, rng.randrange(1, 1025)])
    # a teacher near the student, among its tokens that are not masked
    t = torch.where(x.float() >= x.float().amax(1, keepdim=True) - 60 * T, x.float(), -np.inf) + torch.randn(x.shape, generator=gen, device=DEV) * T
    n = min(k, V)
    v, i = torch.topk(t, n, dim=1)
    values = torch.nn.functional.pad(v, (0, k - n), value=-np.inf).contiguous()
    ids = torch.nn.functional.pad(torch.where(v > -np.inf, i, -1), (0, k - n), value=-1).to(torch.int32).contiguous()
    whole = torch.logsumexp(t.double() / T, 1)
    # (a log-normaliser that fp32 holds to a few units: p is of its error's size else)
    lse = whole.float() if rng.random() < 0.5 and ((whole.float().double() - whole).abs() < 4).all() else None
    w = torch.randn(B, generator=gen, device=DEV) if rng.random() < 0.5 else None
    try:
        distill.check(x, ids, values, lse=lse, T=T, w=w)
    except AssertionError as e:
        raise AssertionError((seed, B, V, x.dtype, k, T, lse is not None, w is not None)) from e


def test_distillation():
    for i in range(300):
        distill_case(200000 + i)
