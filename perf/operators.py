"""Workloads of the operators on rows of logits: filtered sampling, the largest
logits of a row, and distillation from a teacher's largest logits.

`run` computes them in plain torch operations, or, where `own` is true, through
the package's entry points.  Logits are random rows like the verify step's own
workloads: N(0, sigma^2), some rows with one token far above the rest.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one stream of a chat server: a single row, the usual filters
        dict(name="sample_one", op="sample", rows=1, vocab=32000, dtype="f32", filters="topk_topp", temperature=0.7, sigma=3.0, masked=0.0),
        # a batch whose requests each bring settings of their own, greedy ones and grammar-masked rows among them
        dict(name="sample_mixed", op="sample", rows=64, vocab=128256, dtype="bf16", filters="mixed", temperature=1.0, sigma=4.0, masked=0.3),
        # a large batch on nucleus sampling alone
        dict(name="sample_nucleus", op="sample", rows=512, vocab=152064, dtype="bf16", filters="topp", temperature=0.7, sigma=5.0, masked=0.0),
        # flat rows at a high temperature: thousands of tokens stay in the nucleus (odd vocabulary, unaligned rows)
        dict(name="sample_flat", op="sample", rows=48, vocab=50257, dtype="f32", filters="topp", temperature=1.2, sigma=2.0, masked=0.0),
        # the candidates of four draft heads for sixteen sequences
        dict(name="top_heads", op="top", rows=64, vocab=32000, dtype="f32", k=8, lse=False, sigma=3.0, masked=0.0),
        # a verify step's target rows, kept as a teacher's
        dict(name="top_teacher", op="top", rows=2304, vocab=129280, dtype="bf16", k=64, lse=True, sigma=4.0, masked=0.0),
        # many entries of a few ragged rows
        dict(name="top_many", op="top", rows=12, vocab=50257, dtype="bf16", k=777, lse=True, sigma=4.0, masked=0.2),
        # a micro-batch of a small draft model: loss and gradient in one call, odd sizes
        dict(name="distill_small", op="distill", rows=37, vocab=5003, dtype="bf16", k=20, tail=False, split=False, ignored=0.2, sigma=3.0),
        # a training batch: loss and gradient in one call
        dict(name="distill_train", op="distill", rows=2048, vocab=128256, dtype="bf16", k=64, tail=True, split=False, ignored=0.1, sigma=4.0),
        # the same in 32 bits, forward and backward called apart, as under an autograd graph
        dict(name="distill_apart", op="distill", rows=1024, vocab=32000, dtype="f32", k=128, tail=False, split=True, ignored=0.0, sigma=3.0),
        dict(name="distill_apart_bf16", op="distill", rows=512, vocab=152064, dtype="bf16", k=256, tail=True, split=True, ignored=0.1, sigma=4.0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "top", "distill"])
    dtype = rng.choice(["f32", "bf16"])
    vocab = _log(rng, 1000, 152064)
    sigma = round(rng.uniform(2.0, 5.0), 2)
    if op == "sample":
        rows = _log(rng, 1, 512)
        return dict(op=op, rows=rows if dtype == "bf16" else max(1, rows // 2), vocab=vocab, dtype=dtype,
                    filters=rng.choice(["topk_topp", "topp", "minp", "mixed", "none"]), temperature=round(rng.uniform(0.3, 1.4), 2),
                    sigma=sigma, masked=rng.choice([0.0, 0.0, round(rng.uniform(0.0, 0.9), 2)]))
    if op == "top":
        rows = _log(rng, 1, 2048)
        return dict(op=op, rows=rows if dtype == "bf16" else max(1, rows // 2), vocab=vocab, dtype=dtype, k=_log(rng, 1, 1000),
                    lse=rng.random() < 0.7, sigma=sigma, masked=rng.choice([0.0, round(rng.uniform(0.0, 0.5), 2)]))
    rows = _log(rng, 1, 2048)
    return dict(op=op, rows=rows if dtype == "bf16" else max(1, rows // 2), vocab=vocab, dtype=dtype, k=_log(rng, 1, 512),
                tail=rng.random() < 0.5, split=rng.random() < 0.5, ignored=rng.choice([0.0, round(rng.uniform(0.0, 0.6), 2)]), sigma=sigma)


def work(case):
    """Each logit read once, each output written once; no contraction, a few operations a logit."""
    rows, vocab, eb = case["rows"], case["vocab"], 4 if case["dtype"] == "f32" else 2
    read = rows * vocab * eb
    if case["op"] == "sample":
        return {"bytes": read + rows * 24, "flops": 2 * rows * vocab}
    if case["op"] == "top":
        return {"bytes": read + rows * (8 * case["k"] + (4 if case["lse"] else 0)), "flops": 2 * rows * vocab}
    live = rows - int(rows * case["ignored"])  # ignored rows are not read; their gradient is zero
    passes = 2 if case["split"] else 1         # a backward pass of its own reads the logits again
    teacher = rows * (8 * case["k"] + (4 if case["tail"] else 0) + 4)
    return {"bytes": passes * (live * vocab * eb + teacher) + rows * (vocab * eb + 12), "flops": 4 * rows * vocab}


# ----------------------------------------------------------------- the inputs
def _logits(gen, rows, vocab, dtype, sigma, masked):
    """Rows of N(0, sigma^2), a third of them with one token far ahead, a share of the tokens masked with -inf."""
    dev = gen.device
    x = torch.randn((rows, vocab), generator=gen, device=dev) * sigma
    at = torch.randint(0, vocab, (rows, 1), generator=gen, device=dev)
    ahead = (torch.rand((rows, 1), generator=gen, device=dev) < 0.3).float() * 4.0 * sigma
    x.scatter_add_(1, at, ahead)
    if masked:
        gone = torch.rand((rows, vocab), generator=gen, device=dev) < masked
        gone.scatter_(1, at, False)  # a token stays in every row
        x.masked_fill_(gone, float("-inf"))
    return x.to(_DT[dtype])


def _pick(gen, rows, values, dtype):
    values = torch.tensor(values, dtype=dtype, device=gen.device)
    return values[torch.randint(0, len(values), (rows,), generator=gen, device=gen.device)].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 17)
    rows, vocab = case["rows"], case["vocab"]
    s = dict(case=dict(case), status=torch.zeros(1, dtype=torch.int32, device=dev))
    if case["op"] == "sample":
        s["logits"] = _logits(gen, rows, vocab, case["dtype"], case["sigma"], case["masked"])
        s["u"] = torch.rand(rows, generator=gen, device=dev)
        full = lambda v, dt: torch.full((rows,), v, dtype=dt, device=dev)  # noqa: E731
        kind, T = case["filters"], case["temperature"]
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = full(T, torch.float32), None, None, None
        if kind == "topk_topp":
            s["top_k"], s["top_p"] = full(50, torch.int32), full(0.95, torch.float32)
        elif kind == "topp":
            s["top_p"] = full(0.9, torch.float32)
        elif kind == "minp":
            s["min_p"] = full(0.05, torch.float32)
        elif kind == "mixed":
            s["temperature"] = _pick(gen, rows, [0.0, 0.6, T, T], torch.float32)
            s["top_k"] = _pick(gen, rows, [0, 1, 20, 50, 1000], torch.int32)
            s["top_p"] = _pick(gen, rows, [1.0, 0.95, 0.8], torch.float32)
            s["min_p"] = _pick(gen, rows, [0.0, 0.0, 0.1], torch.float32)
        s["out"] = dict(tokens=torch.empty(rows, dtype=torch.int32, device=dev))
    elif case["op"] == "top":
        s["logits"] = _logits(gen, rows, vocab, case["dtype"], case["sigma"], case["masked"])
        s["out"] = dict(values=torch.empty((rows, case["k"]), device=dev), ids=torch.empty((rows, case["k"]), dtype=torch.int32, device=dev))
        if case["lse"]:
            s["out"]["lse"] = torch.empty(rows, device=dev)
    else:
        # the student's rows, and the largest logits of a teacher that the student is close to
        s["logits"] = _logits(gen, rows, vocab, case["dtype"], case["sigma"], 0.0)
        k = min(case["k"], vocab)
        values, ids, lse = [], [], []
        for part in s["logits"].split(256):
            teacher = part.float() + torch.randn(part.shape, generator=gen, device=dev)
            v, i = torch.topk(teacher, k, dim=1)
            values.append(v)
            ids.append(i.to(torch.int32))
            lse.append(torch.logsumexp(teacher, dim=1))
        s["values"], s["ids"], s["lse"] = (torch.cat(v).contiguous() for v in (values, ids, lse))
        if case["k"] > vocab:  # slots without a token
            s["values"] = torch.nn.functional.pad(s["values"], (0, case["k"] - vocab), value=float("-inf"))
            s["ids"] = torch.nn.functional.pad(s["ids"], (0, case["k"] - vocab), value=-1)
        if not case["tail"]:
            s["lse"] = None
        s["weight"] = torch.full((rows,), 1.0 / rows, device=dev)
        n = int(rows * case["ignored"])  # padding rows
        s["weight"][torch.randperm(rows, generator=gen, device=dev)[:n]] = 0.0
        s["grad_loss"] = torch.rand(rows, generator=gen, device=dev) + 0.5 if case["split"] else None
        s["out"] = dict(loss=torch.empty(rows, device=dev), stats=torch.empty((rows, 2), device=dev))
        s["grad"] = torch.empty_like(s["logits"])
        if not case["split"]:
            s["out"]["grad"] = s["grad"]
    return s


# ------------------------------------------------------------ the plain forms
def _plain_sample(s):
    # in 64 bits: a token is chosen at a border of a sum over the whole row
    x = s["logits"].double()
    rows, vocab = x.shape
    T = s["temperature"].double().unsqueeze(1)
    w = torch.exp((x - x.amax(1, keepdim=True)) / torch.where(T == 0, 1.0, T))
    order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(vocab, device=x.device).unsqueeze(0)
    if s["top_k"] is not None:
        k = s["top_k"].unsqueeze(1)
        ws = torch.where((k <= 0) | (rank < k), ws, 0.0)
    keep = ws > 0
    if s["top_p"] is not None:
        p = s["top_p"].double().unsqueeze(1)
        mass = ws.cumsum(1)
        before = torch.nn.functional.pad(mass[:, :-1], (1, 0))
        keep &= (p >= 1) | (rank == 0) | (before < p * mass[:, -1:])
    if s["min_p"] is not None:
        keep &= ws >= s["min_p"].double().unsqueeze(1)
    keep &= (T > 0) | (rank == 0)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    mass = torch.where(kept, w, 0.0).cumsum(1)
    t = s["u"].double().unsqueeze(1) * mass[:, -1:]
    return {"tokens": (mass <= t).sum(1).to(torch.int32)}


def _plain_top(s):
    x = s["logits"].float()
    k = s["case"]["k"]
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    value, order = value[:, :k], order[:, :k]
    if k > x.shape[1]:
        value = torch.nn.functional.pad(value, (0, k - x.shape[1]), value=float("-inf"))
        order = torch.nn.functional.pad(order, (0, k - x.shape[1]), value=-1)
    out = {"values": value, "ids": torch.where(value > float("-inf"), order, -1).to(torch.int32)}
    if s["case"]["lse"]:
        m = x.amax(1)
        out["lse"] = m + torch.log(torch.exp(x - m.unsqueeze(1)).sum(1))
    return out


def _plain_teacher(s):
    """(p [N, K], log p) of the teacher's entries; empty slots have p = 0."""
    valid = s["ids"] >= 0
    t = s["values"]
    if s["lse"] is not None:
        logp = t - s["lse"].unsqueeze(1)
    else:
        m = torch.where(valid, t, float("-inf")).amax(1, keepdim=True)
        logp = t - m - torch.log(torch.where(valid, torch.exp(t - m), 0.0).sum(1, keepdim=True))
    logp = torch.where(valid, logp, 0.0)
    return torch.where(valid, torch.exp(logp), 0.0), logp


def _plain_distill(s):
    """The loss w * KL(p || q) over the teacher's entries, the row statistics (max, sum), and the gradient."""
    x = s["logits"].float()
    w, ids = s["weight"].unsqueeze(1), s["ids"].clamp(min=0).long()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    S = e.sum(1, keepdim=True)
    p, logp = _plain_teacher(s)
    logq = x.gather(1, ids) - m - torch.log(S)
    live = w.squeeze(1) != 0
    loss = torch.where(live, s["weight"] * (p * (logp - logq)).sum(1), 0.0)
    stats = torch.where(w != 0, torch.cat([m, S], 1), 0.0)
    up = w if s["grad_loss"] is None else w * s["grad_loss"].unsqueeze(1)
    if s["grad_loss"] is not None:  # the backward pass on its own: from the logits and the statistics again
        e = torch.exp(x - stats[:, :1])
        p, _ = _plain_teacher(s)
    grad = e * (up * p.sum(1, keepdim=True) / S)
    grad.scatter_add_(1, ids, -up * p)
    grad = torch.where(w != 0, grad, 0.0)
    return {"loss": loss, "stats": stats, "grad": grad.to(s["logits"].dtype)}


# --------------------------------------------------------- the package's calls
def _own(s):
    import sampling_online_softmax_gb300 as sv
    c = s["case"]
    if c["op"] == "sample":
        r = sv.spec_sample_filtered(s["logits"], s["u"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                                    out=s["out"], status=s["status"])
        return {"tokens": r["tokens"]}
    if c["op"] == "top":
        r = sv.spec_top_logits(s["logits"], c["k"], lse=c["lse"], out=s["out"], status=s["status"])
        return {n: r[n] for n in ("values", "ids", "lse") if n in r}
    r = sv.spec_distill(s["logits"], s["ids"], s["values"], top_lse=s["lse"], row_weight=s["weight"], grad=not c["split"],
                        out=s["out"], status=s["status"])
    grad = r.get("grad")
    if c["split"]:
        grad = sv.spec_distill_backward(s["logits"], s["ids"], s["values"], r["stats"], s["grad_loss"], top_lse=s["lse"],
                                        row_weight=s["weight"], out=s["grad"], status=s["status"])["grad"]
    return {"loss": r["loss"], "stats": r["stats"], "grad": grad}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_sample(state) if op == "sample" else _plain_top(state) if op == "top" else _plain_distill(state)


# ------------------------------------------------- the definitions, in 64 bits
def _exact_row_sample(x, u, T, k, p, min_p):
    if T == 0:
        return int(np.argmax(x))
    order = np.argsort(-x, kind="stable")
    order = order[: int(np.isfinite(x).sum())]
    if k > 0:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / T)
    n = len(order)
    if p < 1:
        n = min(n, int(np.searchsorted(np.cumsum(w), p * w.sum(), side="left")) + 1)
    n = min(n, int((w >= min_p).sum()))
    kept = np.sort(order[:n])
    c = np.cumsum(np.exp((x[kept] - x[order[0]]) / T))
    return int(kept[min(int(np.searchsorted(c, u * c[-1], side="right")), n - 1)])


def exact(case, seed):
    s = prepare(case, seed)
    host = lambda v: None if v is None else v.double().cpu().numpy()  # noqa: E731
    rows, vocab = case["rows"], case["vocab"]
    if rows * vocab > (90 << 20 if case["op"] == "sample" else 600 << 20):
        return None
    if case["op"] == "sample":
        u, T, k, p, mp = (host(s[n]) for n in ("u", "temperature", "top_k", "top_p", "min_p"))
        at = lambda v, r, none: none if v is None else float(v[r])  # noqa: E731
        toks = [_exact_row_sample(host(s["logits"][r]), u[r], T[r], int(at(k, r, 0)), at(p, r, 1.0), at(mp, r, 0.0)) for r in range(rows)]
        return {"tokens": np.array(toks, dtype=np.int32)}
    if case["op"] == "top":
        k = min(case["k"], vocab)
        values = torch.cat([torch.topk(v.double(), k, dim=1).values for v in s["logits"].split(128)])
        out = {"values": torch.nn.functional.pad(values, (0, case["k"] - k), value=-math.inf), "ids": None}
        if case["lse"]:
            out["lse"] = torch.cat([torch.logsumexp(v.double(), 1) for v in s["logits"].split(128)])
        return out
    loss, stats, grads = [], [], []
    for r in range(0, rows, 128):
        x, ids, t = s["logits"][r:r + 128].double(), s["ids"][r:r + 128].long(), s["values"][r:r + 128].double()
        w = s["weight"][r:r + 128].double()
        t = torch.where(ids >= 0, t, -math.inf)
        logp = t - (s["lse"][r:r + 128].double().unsqueeze(1) if s["lse"] is not None else torch.logsumexp(t, 1, keepdim=True))
        p = torch.exp(logp)
        logq = torch.log_softmax(x, 1)
        terms = torch.where(p > 0, p * (logp - logq.gather(1, ids.clamp(min=0))), 0.0)
        loss.append(w * terms.sum(1))
        top = x.max(1).values
        stats.append(torch.stack([top, torch.exp(torch.logsumexp(x, 1) - top)], 1) * (w != 0).unsqueeze(1))
        up = w if s["grad_loss"] is None else w * s["grad_loss"][r:r + 128].double()
        target = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), p)
        grads.append((up.unsqueeze(1) * (torch.exp(logq) * p.sum(1, keepdim=True) - target)).float())
    return {"loss": torch.cat(loss), "stats": torch.cat(stats), "grad": torch.cat(grads)}
