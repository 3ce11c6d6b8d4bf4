"""What the single-plane serving operators are measured on: the write of new tokens
into a paged cache, the attention of a chunk of new tokens over it (prompts, chunks
of prompts, draft blocks under verification, single tokens; sliding window with
first tokens that stay visible), and the draw of a token from given random numbers.

A looped model's prelude and coda layers run once per token, so they keep one
key/value plane per position; these operators serve those layers, and the draw
feeds the draft and the acceptance step.

``run`` computes each operator in plain torch where ``own`` is false, and through the
package's public entry points where it is true.  ``exact`` is the definition in 64
bits, written apart from the plain form.
"""
import math
import random

import torch

own = False


# --------------------------------------------------------------------------- cases
def _attn(name, **kw):
    case = dict(name=name, op="attn", dtype="bf16", heads=32, kv_heads=32, d=128, page=64, nseq=1, ctx_lo=0, ctx_hi=0,
                new_lo=1, new_hi=1, chunk=0, window=0, sinks=0, token_major=False, mix=0)
    case.update(kw)
    return case


def _append(name, **kw):
    case = dict(name=name, op="append", dtype="bf16", kv_heads=8, d=128, page=16, nseq=64, ctx_lo=0, ctx_hi=0, new_lo=1,
                new_hi=1, token_major=False, mix=0)
    case.update(kw)
    return case


def _sample(name, **kw):
    case = dict(name=name, op="sample", rows=1, vocab=32000, dtype="f32", temperature=True, top_k=True, top_p=True,
                min_p=True, spread=3.0)
    case.update(kw)
    return case


def listed():
    return [
        # one sequence, one token: the latency of a single-user decode step in a 55-head layer
        _attn("decode 1x1024 h55 d96", heads=55, kv_heads=55, d=96, ctx_lo=1024, ctx_hi=1024),
        # draft blocks of 8 tokens of 64 ragged sequences under verification, grouped heads, small pages
        _attn("verify 64xk8 ragged h32/8", kv_heads=8, page=16, nseq=64, ctx_lo=512, ctx_hi=4096, new_lo=8, new_hi=8, mix=3),
        # long contexts, one token each: the cache's bytes are all that counts
        _attn("decode 16x32768 h32/8", kv_heads=8, nseq=16, ctx_lo=32768, ctx_hi=32768),
        # a whole prompt with nothing before it, every head with its own keys
        _attn("prompt 2048 h55 d96", heads=55, kv_heads=55, d=96, new_lo=2048, new_hi=2048),
        # a chunk of a long prompt: the largest call
        _attn("chunk 2048 at 32768 h32/8", kv_heads=8, ctx_lo=32768, ctx_hi=32768, new_lo=2048, new_hi=2048),
        # a serving batch: one chunk of a prompt among decode steps, window and first tokens, token-major pages
        _attn("mixed 24 window 1024+4 d64", heads=32, kv_heads=4, d=64, page=32, nseq=24, ctx_lo=100, ctx_hi=6000, new_lo=1,
              new_hi=2, chunk=509, window=1024, sinks=4, token_major=True, mix=5),
        # the 32-bit form on the smallest layer: launch latency
        _attn("tiny f32 h2 d16", dtype="f32", heads=2, kv_heads=2, d=16, page=16, ctx_lo=48, ctx_hi=48, new_lo=4, new_hi=4),
        # accepted draft tokens of a batch, written into small pages
        _append("append 64 ragged <=8", ctx_lo=512, ctx_hi=4096, new_lo=1, new_hi=8, mix=7),
        # prompts written into the pages of a 55-head layer
        _append("append 3 prompts h55 d96", kv_heads=55, d=96, page=64, nseq=3, ctx_lo=0, ctx_hi=77, new_lo=1500, new_hi=4000,
                mix=9),
        # one token for one user, all filters on
        _sample("draw 1x32000"),
        # a batch with nucleus and minimum probability over 16-bit logits, odd vocabulary
        _sample("draw 48x65537 bf16", rows=48, vocab=65537, dtype="bf16", top_k=False),
        # a large batch, every row with its own settings
        _sample("draw 256x131072", rows=256, vocab=131072),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


#: bounds on a drawn case: scores of the padded batch (the plain form holds them), pairs times width, cache elements
_MOST_SCORES, _MOST_MULS, _MOST_CACHE = 2.2e9, 1.2e12 / 4, 16 * 32768 * 8 * 128


def draw(rng):
    op = rng.choice(("attn", "attn", "attn", "append", "sample", "sample"))
    if op == "sample":
        vocab = _log_int(rng, 300, 200000)
        rows = _log_int(rng, 1, min(256, max(1, 256 * 131072 // vocab)))
        case = _sample("", rows=rows, vocab=vocab, dtype=rng.choice(("f32", "bf16")), temperature=rng.random() < 0.9,
                       top_k=rng.random() < 0.6, top_p=rng.random() < 0.7, min_p=rng.random() < 0.4,
                       spread=round(rng.uniform(1.0, 5.0), 2))
        del case["name"]
        return case
    dtype = rng.choice(("bf16", "bf16", "bf16", "bf16", "f32"))
    d = rng.choice((64, 96, 128, 128)) if dtype == "bf16" and rng.random() < 0.85 else rng.choice((16, 32, 80, 128))
    page = rng.choice((16, 32, 64, 128))
    kv_heads = rng.choice((1, 2, 4, 5, 8, 16, 32))
    mix = rng.randrange(1 << 20)
    if op == "append":
        nseq = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, min(4096, 8192 * 16 // (nseq * kv_heads))))
        case = _append("", dtype=dtype, kv_heads=kv_heads, d=d, page=page, nseq=nseq, ctx_lo=rng.randrange(0, 100),
                       ctx_hi=rng.randrange(100, 600), new_lo=rng.randint(0, hi), new_hi=hi, token_major=rng.random() < 0.5,
                       mix=mix)
        del case["name"]
        return case
    while True:
        group = rng.choice((1, 1, 2, 3, 4, 8))
        heads = kv_heads * group
        kind = rng.choice(("decode", "verify", "chunk", "mixed"))
        nseq = _log_int(rng, 1, 64) if kind != "chunk" else rng.randint(1, 3)
        ctx_hi = _log_int(rng, 1, 32768 if dtype == "bf16" else 4096)
        ctx_lo = rng.randint(0, ctx_hi)
        new_lo, new_hi, chunk = 1, 1, 0
        if kind == "verify":
            new_lo, new_hi = 1, rng.randint(2, 16)
        elif kind == "chunk":
            new_hi = _log_int(rng, 17, 2048 if dtype == "bf16" else 400)
            new_lo = rng.randint(0, new_hi)
        elif kind == "mixed":
            chunk = _log_int(rng, 17, 1024 if dtype == "bf16" else 200)
        window = rng.choice((0, 0, _log_int(rng, 1, 4096)))
        sinks = rng.choice((0, 4, rng.randrange(1, 100))) if window else 0
        longest = max(new_hi, chunk)
        scores = nseq * heads * longest * (ctx_hi + longest)
        if heads <= 64 and heads * longest <= 1 << 17 and scores <= _MOST_SCORES and scores * d <= _MOST_MULS \
                and nseq * ctx_hi * kv_heads * d <= _MOST_CACHE:
            break
    case = _attn("", dtype=dtype, heads=heads, kv_heads=kv_heads, d=d, page=page, nseq=nseq, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                 new_lo=new_lo, new_hi=new_hi, chunk=chunk, window=window, sinks=sinks, token_major=rng.random() < 0.4,
                 mix=mix)
    del case["name"]
    return case


# --------------------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens in the cache before the call, and new tokens, of each sequence."""
    rng = random.Random(case["mix"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["nseq"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["nseq"])]
    if case.get("chunk"):
        new[rng.randrange(case["nseq"])] = case["chunk"]
    if sum(new) == 0:
        new[0] = 1
    return ctx, new


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pages(case, ctx, new, gen):
    """Key and value pages full of values, and a page table that scatters the sequences over them."""
    page, hk, d = case["page"], case["kv_heads"], case["d"]
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    total, width = sum(need) + 3, max(need)
    shape = (total, page, hk, d) if case["token_major"] else (total, hk, page, d)
    k, v = (torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)) for _ in range(2))
    if case["token_major"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    rows = torch.zeros((len(need), width), dtype=torch.int64)
    at = 0
    for i, n in enumerate(need):
        rows[i, :n] = torch.arange(at, at + n)
        at += n
    return k, v, order[rows.cuda()].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "sample":
        n, vocab = case["rows"], case["vocab"]
        rand = lambda: torch.rand(n, generator=gen, device="cuda")  # noqa: E731
        z = torch.randn((n, vocab), generator=gen, device="cuda") * case["spread"]
        # a few tokens that the model is sure of, by row more or less
        at = torch.randint(0, vocab, (n, 12), generator=gen, device="cuda")
        z.scatter_add_(1, at, rand()[:, None] * 4 * case["spread"] * torch.rand((n, 12), generator=gen, device="cuda"))
        state = {"op": "sample", "logits": z if case["dtype"] == "f32" else z.bfloat16(), "u": rand()}
        state["temperature"] = torch.where(rand() < 0.15, 0.0, 0.6 + 0.6 * rand()) if case["temperature"] else None
        state["top_k"] = torch.where(rand() < 0.3, 0, (1 + 199 * rand().square()).to(torch.int32)).to(torch.int32) if case["top_k"] else None
        state["top_p"] = torch.where(rand() < 0.2, 1.0, 0.7 + 0.29 * rand()) if case["top_p"] else None
        state["min_p"] = torch.where(rand() < 0.4, 0.0, 0.1 * rand()) if case["min_p"] else None
        return state
    ctx, new = _lengths(case)
    k, v, table = _pages(case, ctx, new, gen)
    row0 = [0]
    for n in new:
        row0.append(row0[-1] + n)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    state = {"op": case["op"], "k_pages": k, "v_pages": v, "table": table, "ctx": ints(ctx), "row0": ints(row0)}
    rows, dt = row0[-1], _dtype(case)
    if case["op"] == "append":
        state["k"], state["v"] = (torch.randn((rows, case["kv_heads"], case["d"]), generator=gen, device="cuda", dtype=dt)
                                  for _ in range(2))
        return state
    # heads attend more and less sharply
    sharp = 0.5 + 1.5 * torch.rand((1, case["heads"], 1), generator=gen, device="cuda")
    state["q"] = (torch.randn((rows, case["heads"], case["d"]), generator=gen, device="cuda") * sharp).to(dt)
    state["o"] = torch.empty_like(state["q"])
    state["lse"] = torch.empty((rows, case["heads"]), device="cuda")
    state.update(window=case["window"], sinks=case["sinks"], max_new=max(new), max_len=max(c + n for c, n in zip(ctx, new)))
    return state


# --------------------------------------------------------------------------- plain forms
def _rows_of(row0, rows):
    """Sequence and place in its chunk of each of the call's rows."""
    r = torch.arange(rows, device=row0.device)
    seq = torch.searchsorted(row0[1:].long(), r, right=True)
    return seq, r - row0.long()[seq]


def _plain_append(s):
    k_pages, v_pages = s["k_pages"], s["v_pages"]
    page = k_pages.shape[2]
    seq, j = _rows_of(s["row0"], s["k"].shape[0])
    pos = s["ctx"].long()[seq] + j
    at = s["table"].long()[seq, pos // page]
    k_pages[at, :, pos % page] = s["k"]
    v_pages[at, :, pos % page] = s["v"]
    return {"k_pages": k_pages, "v_pages": v_pages}


def _plain_attn(s):
    q, table, ctx = s["q"], s["table"].long(), s["ctx"].long()
    rows, heads, d = q.shape
    hk, page = s["k_pages"].shape[1:3]
    nseq, n, length = table.shape[0], s["max_new"], s["max_len"]
    k, v = (p[table].permute(0, 2, 1, 3, 4).reshape(nseq, hk, -1, d)[:, :, :length].float() for p in (s["k_pages"], s["v_pages"]))
    # the batch padded to its longest chunk, the heads of a group beside each other
    at = (s["row0"][:-1].long()[:, None] + torch.arange(n, device=q.device)).clamp(max=rows - 1)
    qp = q[at].float().reshape(nseq, n, hk, heads // hk, d).permute(0, 2, 3, 1, 4).reshape(nseq, hk, -1, d)
    pos = (ctx[:, None] + torch.arange(n, device=q.device))[:, :, None]
    key = torch.arange(length, device=q.device)
    seen = key <= pos
    if s["window"]:
        seen &= (key > pos - s["window"]) | (key < s["sinks"])
    p = torch.matmul(qp, k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(nseq, hk, heads // hk, n, length)
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen.any(1)[:, None, :, None], 0)
    o = torch.matmul(p.view(nseq, hk, -1, length), v).view(nseq, hk, heads // hk, n, d) / total
    lse = (top + total.log()).squeeze(-1)
    seq, j = _rows_of(s["row0"], rows)
    return {"o": o.permute(0, 3, 1, 2, 4)[seq, j].reshape(rows, heads, d).to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2)[seq, j].reshape(rows, heads)}


def _plain_sample(s):
    # 64 bits: the draw and the nucleus compare running sums with a border
    z = s["logits"].double()
    n, vocab = z.shape
    col = lambda t, off: torch.full((n, 1), off, device=z.device, dtype=torch.float64) if t is None else t.double()[:, None]  # noqa: E731
    temp, k, p, low = col(s["temperature"], 1.0), col(s["top_k"], 0), col(s["top_p"], 1.0), col(s["min_p"], 0.0)
    greedy = temp == 0
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    w = ((z - z[:, :1]) / torch.where(greedy, 1.0, temp)).exp()
    place = torch.arange(vocab, device=z.device)
    keep = (place < torch.where(k > 0, k, vocab)) & (place < torch.where(greedy, 1, vocab))
    w = w * keep
    before = w.cumsum(1) - w
    keep &= (p >= 1) | (before < p * w.sum(1, keepdim=True))
    keep &= (w >= low) | (place == 0)
    w = torch.zeros_like(w).scatter_(1, order, w * keep)
    run_ = w.cumsum(1)
    token = (run_ <= s["u"].double()[:, None] * run_[:, -1:]).sum(1)
    return {"token": token.to(torch.int32), "logprob": (w.gather(1, token[:, None]) / run_[:, -1:]).log()[:, 0].float()}


def run(state):
    if own:
        from depth_planed_kv_b200 import ripe
        if state["op"] == "append":
            ripe.ripe_paged_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["table"], state["ctx"],
                                   state["row0"])
            return {"k_pages": state["k_pages"], "v_pages": state["v_pages"]}
        if state["op"] == "attn":
            ripe.ripe_paged_attn(state["q"], state["k_pages"], state["v_pages"], state["table"], state["ctx"], state["row0"],
                                 state["o"], state["lse"], max_ntok=state["max_new"], window=state["window"],
                                 sinks=state["sinks"])
            return {"o": state["o"], "lse": state["lse"]}
        token, logprob = ripe.ripe_sample(state["logits"], state["u"], state["temperature"], state["top_k"], state["top_p"],
                                          state["min_p"])
        return {"token": token, "logprob": logprob}
    return {"append": _plain_append, "attn": _plain_attn, "sample": _plain_sample}[state["op"]](state)


# --------------------------------------------------------------------------- floors
def _seen(pos, window, sinks):
    """Keys that the token at `pos` sees."""
    if not window or window > pos:
        return pos + 1
    return window + min(sinks, pos + 1 - window)


def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 28), "flops": 4 * case["rows"] * case["vocab"]}
    size = 2 if case["dtype"] == "bf16" else 4
    ctx, new = _lengths(case)
    if case["op"] == "append":
        return {"bytes": 4 * sum(new) * case["kv_heads"] * case["d"] * size, "flops": 0}
    window, sinks = case["window"], case["sinks"]
    pairs = keys = 0
    for c, n in zip(ctx, new):
        pairs += sum(_seen(c + j, window, sinks) for j in range(n))
        if n:
            first = max(0, c + 1 - window) if window else 0  # the oldest key in any token's window
            keys += c + n - first + min(sinks, first)
    rows = sum(new)
    return {"bytes": 2 * keys * case["kv_heads"] * case["d"] * size + rows * case["heads"] * (2 * case["d"] * size + 4),
            "flops": 4 * pairs * case["heads"] * case["d"]}


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "sample":
        return {"token": None, "logprob": _exact_logprob(s)}
    ctx, new = _lengths(case)
    heads, hk, d, page = case["heads"], case["kv_heads"], case["d"], case["page"]
    group = heads // hk
    out, lse = [], []
    for i, (c, n) in enumerate(zip(ctx, new)):
        if not n:
            continue
        ids = s["table"][i, :-(-(c + n) // page)].long()
        r = int(s["row0"][i])
        place = torch.arange(c, c + n, device="cuda").view(-1, 1)
        key = torch.arange(c + n, device="cuda").view(1, -1)
        hidden = key > place
        if case["window"]:
            hidden |= (place - key >= case["window"]) & (key >= case["sinks"])
        o_heads, l_heads = [], []
        for h in range(hk):
            kk = s["k_pages"][ids, h].reshape(-1, d)[:c + n].double()
            vv = s["v_pages"][ids, h].reshape(-1, d)[:c + n].double()
            qq = s["q"][r:r + n, h * group:(h + 1) * group].double()
            for g in range(group):
                score = (qq[:, g] @ kk.T) / d ** 0.5
                score[hidden] = -math.inf
                l_heads.append(torch.logsumexp(score, 1))
                o_heads.append(torch.exp(score - l_heads[-1][:, None]) @ vv)
        out.append(torch.stack(o_heads, 1))
        lse.append(torch.stack(l_heads, 1))
    return {"o": torch.cat(out), "lse": torch.cat(lse)}


def _exact_append(case, s):
    """The pages with each sequence's new tokens in the slots behind its context."""
    ctx, new = _lengths(case)
    page, out = case["page"], {}
    for name in ("k", "v"):
        flat = s[name + "_pages"].double().transpose(1, 2).reshape(-1, case["kv_heads"], case["d"])  # [page * slot][head][d]
        for i, (c, n) in enumerate(zip(ctx, new)):
            slots = (s["table"][i].long()[:, None] * page + torch.arange(page, device="cuda")).view(-1)[c:c + n]
            r = int(s["row0"][i])
            flat[slots] = s[name][r:r + n].double()
        out[name + "_pages"] = flat.view(-1, page, case["kv_heads"], case["d"]).transpose(1, 2)
    return out


def _exact_logprob(s):
    """Natural logarithm of the drawn token's share of what the filters keep, row by row."""
    got = []
    for r in range(s["logits"].shape[0]):
        z = s["logits"][r].double()
        pick = lambda key, off: off if s[key] is None else float(s[key][r])  # noqa: E731
        temp, k, p, low, u = pick("temperature", 1.0), int(pick("top_k", 0)), pick("top_p", 1.0), pick("min_p", 0.0), float(s["u"][r])
        if temp == 0:
            got.append(0.0)
            continue
        y = z / temp
        y = y - y.max()
        order = torch.argsort(y, descending=True, stable=True)
        if k:
            order = order[:k]
        w = torch.exp(y[order])
        if p < 1:
            ahead = torch.cat((w.new_zeros(1), torch.cumsum(w, 0)[:-1]))
            order = order[ahead < p * w.sum()]
        order = order[(y[order] >= math.log(low)) | (y[order] == 0)] if low > 0 else order
        order = torch.sort(order).values
        w = torch.exp(y[order])
        c = torch.cumsum(w, 0)
        at = int(torch.searchsorted(c, u * c[-1], right=True))
        got.append(float(torch.log(w[at] / c[-1])))
    return torch.tensor(got, dtype=torch.float64, device="cuda")
