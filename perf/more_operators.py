"""Workloads of the operators around a verify: attention of drafted tokens over a
paged cache, the cache's writing and reading back, and the penalties, biases and
grammar masks of the logits.

`run` computes them in plain torch operations, or, where `own` is true, through
the package's entry points.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one stream without a draft: a single token over a short context
        dict(name="attend_one", op="attend", batch=1, nodes=1, heads=32, kv_heads=8, dim=128, context=700, shared=0, dtype="bf16", cache="same", page=64, tree=False),
        # a chat batch with four drafted tokens each, the cache in 8 bits
        dict(name="attend_chain", op="attend", batch=64, nodes=5, heads=32, kv_heads=8, dim=128, context=8192, shared=0, dtype="bf16", cache="e4m3", page=64, tree=False),
        # the 64-node candidate tree
        dict(name="attend_tree", op="attend", batch=16, nodes=64, heads=32, kv_heads=8, dim=128, context=4096, shared=0, dtype="bf16", cache="same", page=32, tree=True),
        # a small model of odd sizes: seven query heads a key head, short pages, a ragged tree
        dict(name="attend_odd", op="attend", batch=7, nodes=23, heads=14, kv_heads=2, dim=64, context=1500, shared=0, dtype="f16", cache="e4m3", page=16, tree=True),
        # one long system prompt before every request of the batch
        dict(name="attend_shared", op="attend", batch=48, nodes=9, heads=32, kv_heads=8, dim=128, context=600, shared=16384, dtype="bf16", cache="same", page=64, tree=False),
        # a few very long documents
        dict(name="attend_long", op="attend", batch=3, nodes=9, heads=32, kv_heads=8, dim=128, context=131072, shared=0, dtype="bf16", cache="same", page=128, tree=False),
        # the accepted path of every tree goes into the cache, and is read back
        dict(name="cache_path", op="cache", batch=64, tokens=6, nodes=64, kv_heads=8, dim=128, dtype="bf16", cache="e4m3", page=64, path=True),
        # the same for prompts
        dict(name="cache_prompt", op="cache", batch=5, tokens=8000, nodes=8000, kv_heads=8, dim=128, dtype="bf16", cache="e4m3", page=64, path=False),
        # one stream, one row
        dict(name="adjust_one", op="adjust", batch=1, nodes=1, vocab=32000, dtype="f32", history=500, biases=8, masked=False, tree=False),
        # the target rows of four drafted tokens, penalised and under grammars
        dict(name="adjust_chain", op="adjust", batch=64, nodes=5, vocab=128256, dtype="bf16", history=4000, biases=32, masked=True, tree=False),
        # every node of the 64-node tree
        dict(name="adjust_tree", op="adjust", batch=16, nodes=64, vocab=32000, dtype="f32", history=2000, biases=0, masked=True, tree=True),
        # a large batch of long drafts
        dict(name="adjust_stress", op="adjust", batch=512, nodes=9, vocab=152064, dtype="bf16", history=1000, biases=0, masked=False, tree=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "cache", "adjust", "adjust"])
    if op == "attend":
        kv_heads, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8]), rng.choice([64, 128])
        batch, nodes = _log(rng, 1, 64), _log(rng, 1, 64)
        # no more keys and values than the long documents have, no more scores than the trees
        most = min(3 * 131072 * 8 // (batch * kv_heads), 16 * 64 * 32 * 4096 // (batch * nodes * kv_heads * group))
        context = min(_log(rng, 1, 131072), most)
        shared = _log(rng, 1, context) if batch > 1 and rng.random() < 0.3 else 0
        return dict(op=op, batch=batch, nodes=nodes, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, context=max(1, context - shared), shared=shared,
                    dtype=rng.choice(["bf16", "bf16", "f16"]), cache=rng.choice(["same", "e4m3"]), page=rng.choice([16, 32, 64, 128]), tree=rng.random() < 0.5)
    if op == "cache":
        batch, path = _log(rng, 1, 64), rng.random() < 0.5
        tokens = _log(rng, 1, 12) if path else _log(rng, 1, 40000 // batch)
        return dict(op=op, batch=batch, tokens=tokens, nodes=tokens + _log(rng, 1, 60) if path else tokens, kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f16"]), cache=rng.choice(["same", "e4m3", "e4m3"]), page=rng.choice([16, 32, 64, 128]), path=path)
    vocab, tree = _log(rng, 1000, 152064), rng.random() < 0.4
    nodes = _log(rng, 2, 64) if tree else rng.randint(1, 9)
    batch = min(_log(rng, 1, 512), max(1, 512 * 9 * 152064 // (2 * nodes * vocab)))
    return dict(op=op, batch=batch, nodes=nodes, vocab=vocab, dtype=rng.choice(["f32", "bf16"]), history=_log(rng, 1, 8000), biases=rng.choice([0, 0, _log(rng, 1, 300)]),
                masked=rng.random() < 0.5, tree=tree)


def work(case):
    c = case
    if c["op"] == "attend":
        lens = _lengths(c["batch"], c["context"])
        keys = c["shared"] + sum(lens)  # each cached key and value read once
        pairs = c["nodes"] * sum(c["shared"] + n + (c["nodes"] + 1) // 2 for n in lens)
        row = c["dim"] * 2 if c["cache"] == "same" else c["dim"] + 1
        tokens = c["batch"] * c["nodes"]
        return {"bytes": 2 * keys * c["kv_heads"] * row + tokens * 2 * c["dim"] * (2 * c["heads"] + 2 * c["kv_heads"]) + tokens * c["heads"] * 4,
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "cache":
        n = c["kv_heads"] * sum(_counts(c["batch"], c["tokens"]))
        row = c["dim"] * 2 if c["cache"] == "same" else c["dim"] + 1
        return {"bytes": 2 * n * (2 * 2 * c["dim"] + 2 * row), "flops": 2 * n * 2 * c["dim"]}
    rows, eb = c["batch"] * c["nodes"], 4 if c["dtype"] == "f32" else 2
    return {"bytes": rows * c["vocab"] * 2 * eb + (rows * ((c["vocab"] + 31) // 32) * 4 if c["masked"] else 0) + c["batch"] * (4 * c["history"] + 8 * c["biases"]) + rows * 4,
            "flops": rows * c["vocab"]}


# ----------------------------------------------------------------- the inputs
def _lengths(batch, longest):
    """Lengths of a batch: from the longest down to a third of it, ragged."""
    return [max(1, longest - (b * longest * 2) // (3 * batch) - (b * 7) % 5) for b in range(batch)]


def _counts(batch, most):
    return [max(1, most - (b * 5) % (most // 2 + 1)) for b in range(batch)]


def _tree_mask(gen, nodes, tree):
    """(mask words [N, W] int32, the same as bits [N, N]) of a random tree, or of a chain."""
    parent = [0] * nodes
    pick = torch.rand(nodes, generator=gen, device=gen.device).tolist()
    for n in range(1, nodes):
        parent[n] = int(pick[n] * min(n, 1 + n // 2)) if tree else n - 1
    seen = torch.zeros((nodes, nodes), dtype=torch.bool)
    for n in range(nodes):
        if n:
            seen[n] = seen[parent[n]]
        seen[n, n] = True
    words = torch.nn.functional.pad(seen.long(), (0, -nodes % 32)).view(nodes, -1, 32)
    words = (words << torch.arange(32)).sum(2)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return words.to(gen.device).contiguous(), seen.to(gen.device)


def _power(e):
    """2^e in float32, exactly (a power taken as a product or by exp may be a step off), for -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _e4m3(x):
    """Rows of x in 8 bits: (values as e4m3, the scale's exponent + 127)."""
    frac, exp = torch.frexp(x.float().abs().amax(-1))  # amax = frac 2^exp, frac in [1/2, 1)
    e = torch.where(frac > 0, exp - 9 + (frac > 0.875).to(exp.dtype), -110).clamp(-110, 120)
    return (x.float() * _power(-e).unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _pages(gen, batch, tokens, page):
    """A page table whose pages lie in random order: (table [B, pages a sequence], pages in all)."""
    each = (tokens + page - 1) // page
    total = batch * each + 3
    return torch.randperm(total, generator=gen, device=gen.device)[: batch * each].view(batch, each).to(torch.int32).contiguous(), total


def _new_cache(gen, c, pages, spread):
    """Keys or values of a whole cache; in 8 bits with its scales."""
    dt = _DT[c["dtype"]]
    x = torch.empty((pages, c["kv_heads"], c["page"], c["dim"]), dtype=dt, device=gen.device)
    for part in x.view(-1, c["dim"]).split(1 << 21):
        part.copy_(torch.randn(part.shape, generator=gen, device=gen.device) * spread)
    if c["cache"] == "same":
        return x, None
    q = torch.empty(x.shape, dtype=torch.uint8, device=gen.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.uint8, device=gen.device)
    for part, a, b in zip(x.view(-1, c["dim"]).split(1 << 21), q.view(-1, c["dim"]).split(1 << 21), scale.view(-1).split(1 << 21)):
        values, exps = _e4m3(part)
        a.copy_(values.view(torch.uint8))
        b.copy_(exps)
    return q.view(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 29)
    s = dict(case=dict(c), status=torch.zeros(1, dtype=torch.int32, device=dev))
    randn = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    if c["op"] == "attend":
        dt, B, N, P = _DT[c["dtype"]], c["batch"], c["nodes"], c["shared"]
        s["q"] = (randn(B, N, c["heads"], c["dim"]) * 2.0).to(dt)  # scores of a standard deviation of two
        s["k"], s["v"] = randn(B, N, c["kv_heads"], c["dim"]).to(dt), (randn(B, N, c["kv_heads"], c["dim"]) + 0.5).to(dt)
        s["table"], pages = _pages(gen, B, P + c["context"], c["page"])
        if P:  # the pages that lie whole in the prefix are the first sequence's for all
            s["table"][:, : P // c["page"]] = s["table"][:1, : P // c["page"]].clone()
        s["k_cache"], s["k_scale"] = _new_cache(gen, c, pages, 1.0)
        s["v_cache"], s["v_scale"] = _new_cache(gen, c, pages, 1.0)
        if P % c["page"]:  # the page on the border: each sequence's own copy of what is shared
            at, part = s["table"][:, P // c["page"]].long(), P % c["page"]
            for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
                if s[name] is not None:
                    x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
                    x[at, :, :part] = x[at[:1], :, :part].clone()
        s["lens"] = torch.tensor(_lengths(B, c["context"]), dtype=torch.int32, device=dev) + P
        s["longest"] = c["context"] + P
        s["mask"], s["seen"] = _tree_mask(gen, N, c["tree"])
        s["out"] = dict(out=torch.empty_like(s["q"]), lse=torch.empty((B, N, c["heads"]), device=dev))
        s["scale"] = 1.0 / math.sqrt(c["dim"])
        s["workspace"] = None
    elif c["op"] == "cache":
        dt, B, N, S = _DT[c["dtype"]], c["batch"], c["nodes"], c["tokens"]
        spread = torch.exp2(torch.randint(-3, 4, (1, 1, c["kv_heads"], 1), generator=gen, device=dev).float())  # heads differ in size
        s["k"], s["v"] = (randn(B, N, c["kv_heads"], c["dim"]) * spread).to(dt), randn(B, N, c["kv_heads"], c["dim"]).to(dt)
        s["table"], pages = _pages(gen, B, S + 500, c["page"])
        shape = (pages, c["kv_heads"], c["page"], c["dim"])
        for name in ("k", "v"):
            s[name + "_cache"] = torch.zeros(shape, dtype=dt if c["cache"] == "same" else torch.float8_e4m3fn, device=dev)
            s[name + "_scale"] = None if c["cache"] == "same" else torch.zeros(shape[:-1], dtype=torch.uint8, device=dev)
        s["start"] = torch.randint(0, 500, (B,), generator=gen, device=dev).to(torch.int32)
        s["count"] = torch.tensor(_counts(B, S), dtype=torch.int32, device=dev)
        s["select"] = None
        if c["path"]:  # as a verify of a tree names the accepted nodes: rising, -1 behind the last
            order = torch.rand((B, N), generator=gen, device=dev).argsort(1)[:, :S].sort(1).values
            s["select"] = torch.where(torch.arange(S, device=dev) < s["count"].unsqueeze(1), order, -1).to(torch.int32).contiguous()
        s["out"] = {n: torch.zeros((B, S, c["kv_heads"], c["dim"]), dtype=dt, device=dev) for n in ("k", "v")}
    else:
        B, N, V, L = c["batch"], c["nodes"], c["vocab"], c["history"]
        x = torch.empty((B, N, V), dtype=_DT[c["dtype"]], device=dev)
        for part in x.view(B * N, V).split(256):
            part.copy_(randn(*part.shape) * 4.0)
        s["logits"] = x
        # tokens as text has them: a few common ones, many rare ones
        some = lambda *shape: (V * torch.rand(shape, generator=gen, device=dev).square().square()).long().clamp(max=V - 1).to(torch.int32)  # noqa: E731
        s["tokens"], s["nodes"] = some(B, L), some(B, N)
        s["total"] = torch.tensor(_lengths(B, L), dtype=torch.int32, device=dev)
        s["prompt"] = (s["total"].float() * torch.rand(B, generator=gen, device=dev)).to(torch.int32)
        pick = lambda *v: torch.tensor(v, device=dev)[torch.randint(0, len(v), (B,), generator=gen, device=dev)].contiguous()  # noqa: E731
        s["repetition"], s["frequency"], s["presence"] = pick(1.0, 1.1, 1.3), pick(0.0, 0.2, 0.7), pick(0.0, 0.5, -0.3)
        s["bias_ids"] = s["bias"] = s["allowed"] = None
        if c["biases"]:  # (no token twice; some slots empty)
            ids = (torch.randint(0, V, (B, 1), generator=gen, device=dev) + torch.arange(c["biases"], device=dev) * (V // c["biases"])) % V
            ids[torch.rand(ids.shape, generator=gen, device=dev) < 0.2] = -1
            s["bias_ids"], s["bias"] = ids.to(torch.int32).contiguous(), (randn(B, c["biases"]) * 5.0).contiguous()
        if c["masked"]:  # a third of the rows allow few tokens, a third nearly all, a third everything
            words = torch.randint(-(1 << 31), 1 << 31, (3, B, N, (V + 31) // 32), generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
            few, most = words[0] & words[1] & words[2] & (words[0] >> 7) & (words[1] >> 9), words[0] | words[1] | words[2]
            kind = torch.randint(0, 3, (B, N, 1), generator=gen, device=dev)
            s["allowed"] = torch.where(kind == 0, few, torch.where(kind == 1, most, -1)).contiguous()
        s["mask"], s["seen"] = _tree_mask(gen, N, c["tree"])
        s["out"] = dict(logits=torch.empty_like(x))
    return s


# ------------------------------------------------------------ the plain forms
def _cached(s, name, longest, to):
    """The first `longest` cached rows of every sequence, [B, Hkv, L, D]."""
    x, scale, table = s[name + "_cache"], s[name + "_scale"], s["table"].long()
    B, P = table.shape
    _, heads, page, dim = x.shape
    rows = lambda t: t[table].transpose(1, 2).reshape(B, heads, P * page, -1)[:, :, :longest]  # noqa: E731
    if scale is None:
        return rows(x).to(to)
    return rows(x.view(torch.uint8)).view(torch.float8_e4m3fn).to(to) * _power(rows(scale.unsqueeze(-1)).int() - 127)


def _plain_attend(s):
    B, N, H, D = s["q"].shape
    heads, L = s["k"].shape[2], s["longest"]
    q = s["q"].float().view(B, N, heads, H // heads, D).permute(0, 2, 1, 3, 4).reshape(B, heads, N * (H // heads), D)
    keys = torch.cat([_cached(s, "k", L, torch.float32), s["k"].float().transpose(1, 2)], 2)
    x = torch.matmul(q, keys.transpose(2, 3)).mul_(s["scale"]).view(B, heads, N, H // heads, L + N)
    del keys
    inside = (torch.arange(L, device=x.device) < s["lens"].unsqueeze(1)).view(B, 1, 1, 1, L)
    x[..., :L].masked_fill_(~inside, float("-inf"))
    x[..., L:].masked_fill_(~s["seen"].view(1, 1, N, 1, N), float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    S = x.sum(-1, keepdim=True)
    values = torch.cat([_cached(s, "v", L, torch.float32), s["v"].float().transpose(1, 2)], 2)
    out = torch.matmul(x.view(B, heads, -1, L + N), values).view(B, heads, N, H // heads, D) / S
    lse = (m + torch.log(S)).squeeze(-1)
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, N, H, D).to(s["q"].dtype), "lse": lse.permute(0, 2, 1, 3).reshape(B, N, H)}


def _plain_cache(s):
    B, S = s["out"]["k"].shape[:2]
    i = torch.arange(S, device=s["k"].device)
    b = torch.arange(B, device=i.device).unsqueeze(1)
    page = s["k_cache"].shape[2]
    live = (i < s["count"].unsqueeze(1)).view(B, S, 1, 1)
    at = (s["start"].unsqueeze(1) + i).long()
    pages, slots = s["table"].gather(1, at // page).long(), at % page
    source = i.expand(B, S) if s["select"] is None else s["select"].clamp(min=0).long()
    result = {}
    for name in ("k", "v"):
        x, cache, scale = s[name][b, source], s[name + "_cache"], s[name + "_scale"]
        if scale is None:
            cache[pages, :, slots] = torch.where(live, x, cache[pages, :, slots])
            back = cache[pages, :, slots]
        else:
            q, e = _e4m3(x)
            cells = cache.view(torch.uint8)
            cells[pages, :, slots] = torch.where(live, q.view(torch.uint8), cells[pages, :, slots])
            scale[pages, :, slots] = torch.where(live.squeeze(-1), e, scale[pages, :, slots])
            back = cells[pages, :, slots].view(torch.float8_e4m3fn).float() * _power(scale[pages, :, slots].int().unsqueeze(-1) - 127)
        result[name] = torch.where(live, back.to(x.dtype), s["out"][name])
    return result


def _plain_adjust(s):
    B, N, V = s["logits"].shape
    dev = s["logits"].device
    x = s["logits"].float()
    if s["bias"] is not None:
        add = torch.zeros((B, V), device=dev).scatter_add_(1, s["bias_ids"].clamp(min=0).long(), torch.where(s["bias_ids"] >= 0, s["bias"], 0.0))
        x = x + add.unsqueeze(1)
    at = torch.arange(s["tokens"].shape[1], device=dev)
    live, given = at < s["total"].unsqueeze(1), at < s["prompt"].unsqueeze(1)
    count = torch.zeros((B, V), device=dev).scatter_add_(1, s["tokens"].long(), (live & ~given).float())
    in_prompt = torch.zeros((B, V), device=dev).scatter_add_(1, s["tokens"].long(), (live & given).float()) > 0
    path = s["seen"].clone()
    path[:, 0] = False  # the root is the last token of the history
    count = count.unsqueeze(1).repeat(1, N, 1).scatter_add_(2, s["nodes"].long().unsqueeze(1).expand(B, N, N), path.float().expand(B, N, N))
    row = lambda v: v.view(B, 1, 1)  # noqa: E731
    r = row(s["repetition"])
    x = torch.where((count > 0) | in_prompt.unsqueeze(1), torch.where(x > 0, x / r, x * r), x)
    x = x - row(s["frequency"]) * count
    x = x - row(s["presence"]) * (count > 0)
    if s["allowed"] is not None:
        ok = (s["allowed"].unsqueeze(-1) >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        x = x.masked_fill_(ok.view(B, N, -1)[..., :V] == 0, float("-inf"))
    return {"logits": x.to(s["logits"].dtype)}


# --------------------------------------------------------- the package's calls
def _own(s):
    import sampling_online_softmax_gb300 as sv
    op = s["case"]["op"]
    if op == "attend":
        r = sv.spec_tree_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], mask=s["mask"], shared_len=s["case"]["shared"],
                                   scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=True, out=s["out"], status=s["status"])
        return {"out": r["out"], "lse": r["lse"]}
    if op == "cache":
        sv.spec_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"], count=s["count"], select=s["select"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"], status=s["status"])
        r = sv.spec_cache_read(s["k_cache"], s["v_cache"], s["table"], s["start"], s["out"]["k"].shape[1], count=s["count"],
                               k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], status=s["status"])
        return {"k": r["k"], "v": r["v"]}
    r = sv.spec_adjust_logits(s["logits"], tokens=s["tokens"], prompt_len=s["prompt"], total_len=s["total"], node_tokens=s["nodes"], mask=s["mask"],
                              repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"],
                              allowed=s["allowed"], out=s["out"], status=s["status"])
    return {"logits": r["logits"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_attend(state) if op == "attend" else _plain_cache(state) if op == "cache" else _plain_adjust(state)


# ------------------------------------------------- the definitions, in 64 bits
def _exact_rows(cache, scale, table, n):
    """The first n cached rows of one sequence in 64 bits, [Hkv, n, D]."""
    pages = table[: (n + cache.shape[2] - 1) // cache.shape[2]].long()
    cells = cache.view(torch.uint8)[pages].view(cache.dtype) if scale is not None else cache[pages]
    x = cells.double()
    if scale is not None:
        x = x * _power64(scale[pages].int() - 127).unsqueeze(-1)
    return x.permute(1, 0, 2, 3).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def _exact_attend(s):
    out, lse = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device), None
    B, N, H, D = s["q"].shape
    lse = torch.empty((B, N, H), dtype=torch.float64, device=s["q"].device)
    group = H // s["k"].shape[2]
    for b, n in enumerate(s["lens"].tolist()):
        keys, values = (_exact_rows(s[x + "_cache"], s[x + "_scale"], s["table"][b], n) for x in ("k", "v"))
        for h in range(H):
            z = s["q"][b, :, h].double() @ torch.cat([keys[h // group], s["k"][b, :, h // group].double()]).T * s["scale"]
            z[:, n:][~s["seen"]] = -math.inf
            lse[b, :, h] = torch.logsumexp(z, 1)
            out[b, :, h] = torch.softmax(z, 1) @ torch.cat([values[h // group], s["v"][b, :, h // group].double()])
    return {"out": out, "lse": lse}


def _power64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_cache(s):
    """Every value is the multiple of its row's unit that is nearest, the even one of two."""
    result = {}
    for name in ("k", "v"):
        x = s[name].double()
        if s["select"] is not None:
            x = torch.stack([x[b, s["select"][b].clamp(min=0).long()] for b in range(x.shape[0])])
        if s["k_scale"] is not None:
            top = x.abs().amax(-1, keepdim=True)
            unit = _power64(torch.frexp(torch.where(top > 0, top, 2.0 ** -200) / 448.0)[1].clamp(-110, 120))
            unit = torch.where(top <= 224.0 * unit, (unit / 2.0).clamp(min=2.0 ** -110), unit)  # (448 times a power of two itself)
            y = x / unit
            step = _power64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
            x = torch.round(y / step) * step * unit
        live = torch.arange(x.shape[1], device=x.device) < s["count"].unsqueeze(1)
        result[name] = torch.where(live.view(*live.shape, 1, 1), x, 0.0)
    return result


def _exact_adjust(s):
    x = s["logits"].double()
    B, N, V = x.shape
    total, prompt = s["total"].tolist(), s["prompt"].tolist()
    for b in range(B):
        rep, freq, pres = (float(s[n][b]) for n in ("repetition", "frequency", "presence"))
        made = torch.bincount(s["tokens"][b, prompt[b]:total[b]].long(), minlength=V)
        was = torch.bincount(s["tokens"][b, :prompt[b]].long(), minlength=V)
        if s["bias"] is not None:
            ok = s["bias_ids"][b] >= 0
            x[b, :, s["bias_ids"][b][ok].long()] += s["bias"][b][ok].double()
        for n in range(N):
            on_path = s["seen"][n].clone()
            on_path[0] = False
            c = made + torch.bincount(s["nodes"][b][on_path].long(), minlength=V)
            row = x[b, n]
            row = torch.where((c + was) > 0, torch.where(row > 0, row / rep, row * rep), row) - freq * c.double() - pres * (c > 0).double()
            if s["allowed"] is not None:
                bits = (s["allowed"][b, n].long().unsqueeze(1) >> torch.arange(32, device=x.device)) & 1
                row = torch.where(bits.reshape(-1)[:V] == 1, row, -math.inf)
            x[b, n] = row
    return {"logits": x}


def exact(case, seed):
    if case["op"] == "adjust" and (case["batch"] * case["nodes"] * case["vocab"] > 200 << 20 or case["batch"] * case["nodes"] > 4000):
        return None
    s = prepare(case, seed)
    return _exact_attend(s) if case["op"] == "attend" else _exact_cache(s) if case["op"] == "cache" else _exact_adjust(s)
