"""The operators on the paged cache and on a verify's logits, from their definitions in 64 bits."""
import math

import torch


def tree_words(seen):
    """Rows of bits [N, N] (bool) as [N, ceil(N/32)] int32 words."""
    n = seen.shape[0]
    w = torch.nn.functional.pad(seen.long().cpu(), (0, -n % 32)).view(n, -1, 32)
    w = (w << torch.arange(32)).sum(2)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()


def tree(n, seed, chain=False):
    """(parents, bits [N, N]) of a random tree."""
    g = torch.Generator().manual_seed(seed)
    parents = [0] + [i - 1 if chain else int(torch.randint(0, i, (1,), generator=g)) for i in range(1, n)]
    seen = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        if i:
            seen[i] = seen[parents[i]]
        seen[i, i] = True
    return torch.tensor(parents, dtype=torch.int32), seen


def power_of(x):
    """The least e with max |x| <= 448 2^e over the last axis, as whole numbers (64 bits)."""
    top = x.double().abs().amax(-1)
    e = torch.frexp(top / 448.0)[1]  # top / 448 = f 2^e, 1/2 <= f < 1
    exact = top == 448.0 * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), (e - 1).double())
    return torch.where(exact, e - 1, e)


def quantised(x, fp16=False):
    """x [.., D] as an e4m3 cache gives it back (64 bits), and its scale bytes; finite rows alone."""
    x = x.double()
    e = power_of(x).clamp(-24 if fp16 else -110, 120)
    e = torch.where(x.abs().amax(-1) == 0, torch.full_like(e, -24 if fp16 else -110), e)
    y = torch.ldexp(x, -e.unsqueeze(-1))
    y = torch.where((e == (8 if fp16 else 120)).unsqueeze(-1), y.clamp(-240.0, 240.0), y)  # 256 * 2^e would be past the type's range
    unit = torch.ldexp(torch.ones_like(y), torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)  # e4m3's step: 3 bits, from 2^-6 down fixed
    return torch.ldexp(torch.round(y / unit) * unit, e.unsqueeze(-1)), (e + 127).to(torch.uint8)


def attention(q, k, v, keys, values, lens, seen, scale):
    """keys, values: per sequence [len, kv_heads, D] (64 bits).  Returns (out, lse, what bounds the kernel's error: (sum p |v|,
    the largest sum |q k| scale a row sees, the largest |s|)), each [B, N, heads, ...]."""
    B, N, H, D = q.shape
    kv = k.shape[2]
    out = torch.zeros((B, N, H, D), dtype=torch.float64)
    weight = torch.zeros((B, N, H, D), dtype=torch.float64)
    lse = torch.full((B, N, H), -math.inf, dtype=torch.float64)
    mass = torch.zeros((B, N, H), dtype=torch.float64)
    for b in range(B):
        if lens[b] < 0:
            continue
        for n in range(N):
            on = seen[n].nonzero().flatten()
            kk = torch.cat([keys[b], k[b].double().cpu()[on]])
            vv = torch.cat([values[b], v[b].double().cpu()[on]])
            if not len(kk):
                continue
            for g in range(kv):
                heads = slice(g * (H // kv), (g + 1) * (H // kv))
                x = q[b, n, heads].double().cpu()
                s = x @ kk[:, g].T * scale
                p = torch.softmax(s, 1)
                lse[b, n, heads] = torch.logsumexp(s, 1)
                out[b, n, heads] = p @ vv[:, g]
                weight[b, n, heads] = p @ vv[:, g].abs()
                mass[b, n, heads] = (x.abs() @ kk[:, g].abs().T).amax(1) * scale
    return out, lse, weight, mass


def adjusted(x, seen, tokens, prompt, total, nodes, rep, freq, pres, bias_ids, bias, allowed):
    """spec_adjust_logits on the host, in 64 bits; every list may be None."""
    x = x.double().cpu().clone()
    B, N, V = x.shape
    for b in range(B):
        p0 = 0 if prompt is None else int(prompt[b])
        t0 = (0 if tokens is None else tokens.shape[1]) if total is None else int(total[b])
        r, f, p = (d if t is None else float(t[b]) for t, d in ((rep, 1.0), (freq, 0.0), (pres, 0.0)))
        for n in range(N):
            count, was = {}, set()
            for i in range(t0):
                t = int(tokens[b, i])
                if not 0 <= t < V:
                    continue
                if i < p0:
                    was.add(t)
                else:
                    count[t] = count.get(t, 0) + 1
            if nodes is not None:
                for m in range(1, N):
                    t = int(nodes[b, m])
                    if seen[n, m] and 0 <= t < V:
                        count[t] = count.get(t, 0) + 1
            if bias_ids is not None:
                for i, t in enumerate(bias_ids[b].tolist()):
                    if 0 <= t < V:
                        x[b, n, t] += float(bias[b, i])
            for t in set(count) | was:
                y = float(x[b, n, t])
                y = y / r if y > 0 else y * r
                c = count.get(t, 0)
                x[b, n, t] = y - f * c - (p if c else 0.0)
            if allowed is not None:
                bits = (allowed[b, n].long().cpu().unsqueeze(1) >> torch.arange(32)) & 1
                x[b, n, bits.reshape(-1)[:V] == 0] = -math.inf
    return x
