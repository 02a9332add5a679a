"""The paged-cache operators of the decode window, as cases to be timed and compared.

A layer's decode window projects q, k and v, normalises and rotates the heads and writes k and v into pages
(append), then attends over the pages (attend).  At long contexts it scores every page by its mean key (scores),
selects some of them (topk) and attends over those alone (blocks).  ``run`` computes each operator in elementary
torch operations, or, where ``own`` is set, through bf16_hyper_connection_amd.paged.

Page layouts: keys [page][kv head][D / 8][P][8], values [page][kv head][P / 8][D][8], mean keys [page][kv head][D].
"""

import math

import torch

own = False

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    attn_q = {"heads": 48, "kv_heads": 8, "head_dim": 256, "page": 64}    # 12288 rows, the skinny matvec's projection
    common = {"heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64}    # a usual grouped geometry
    return [
        # the smallest step of a decode loop: one token's heads, where latency counts
        {"name": "append, one token", "op": "append", "seqs": 1, "tokens": 1, "ctx": 1000, **attn_q,
         "type": "f32", "rope": 64, "pairs": False, "norm": True},
        # prompts of unlike lengths going into the cache behind earlier tokens, rotation over whole heads
        {"name": "append, prompts", "op": "append", "seqs": 3, "tokens": 2900, "ctx": 4500, **common,
         "type": "bf16", "rope": 128, "pairs": True, "norm": True},
        # one short conversation, one token
        {"name": "attend, one short", "op": "attend", "seqs": 1, "tokens": 1, "ctx": 700, **common, "type": "f32"},
        # verify windows of up to six tokens over a few conversations of odd lengths
        {"name": "attend, windows", "op": "attend", "seqs": 4, "tokens": 6, "ctx": 9001, **attn_q, "type": "f32"},
        # a serving batch of single tokens over lengths from a thousand to eight thousand
        {"name": "attend, batch", "op": "attend", "seqs": 64, "tokens": 1, "ctx": 8192, **common, "type": "bf16"},
        # the longest context: two tokens over 420,000 positions
        {"name": "attend, long", "op": "attend", "seqs": 1, "tokens": 2, "ctx": 420000, **attn_q, "type": "f32"},
        # mean keys of 420,000 positions, a window of four tokens
        {"name": "scores, long", "op": "scores", "seqs": 1, "tokens": 4, "ctx": 420000, **attn_q},
        # a serving batch of single tokens
        {"name": "scores, batch", "op": "scores", "seqs": 32, "tokens": 1, "ctx": 32768, **common},
        # selection among the 6,562 pages of 420,000 positions
        {"name": "topk, long", "op": "topk", "seqs": 1, "tokens": 4, "ctx": 420000, **attn_q,
         "sel": 64, "first": 1, "last": 2},
        # selection for a batch of single tokens
        {"name": "topk, batch", "op": "topk", "seqs": 32, "tokens": 1, "ctx": 32768, **common,
         "sel": 32, "first": 1, "last": 2},
        # attention over 64 of those 6,562 pages, a window of four tokens
        {"name": "blocks, long", "op": "blocks", "seqs": 1, "tokens": 4, "ctx": 420000, **attn_q, "type": "f32",
         "sel": 64, "first": 1, "last": 2},
        # the same for a batch of single tokens
        {"name": "blocks, batch", "op": "blocks", "seqs": 32, "tokens": 1, "ctx": 32768, **common, "type": "bf16",
         "sel": 32, "first": 1, "last": 2},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "scores", "topk", "blocks"])
    kv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "seqs": _log(rng, 1, 64), "kv_heads": kv, "heads": kv * rng.choice([1, 2, 4, 5, 6, 8, 12, 16]),
            "head_dim": rng.choice([64, 128, 256]), "page": rng.choice([32, 64, 128])}
    row = kv * case["head_dim"]
    if op == "append":
        case["tokens"] = max(1, min(_log(rng, 1, 3000), 9000 // case["seqs"]))
        case["ctx"] = case["tokens"] + _log(rng, 1, 2000)
        case.update(type=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.8, pairs=rng.random() < 0.5,
                    rope=rng.choice([0, 16, case["head_dim"] // 2, case["head_dim"]]))
        return case
    case["tokens"] = rng.randint(1, 16) if rng.random() < 0.6 else 1
    # no more cached values than the longest listed case has, shared among the sequences
    most = min(420000, 420000 * 2048 // (row * case["seqs"]), 10 ** 8 // (case["seqs"] * case["tokens"] * case["heads"]))
    if op in ("scores", "topk", "blocks"):
        most = min(most, 420000 // case["seqs"])
    low = 4 * case["page"] + 16 if op == "scores" else 64
    if op in ("topk", "blocks"):
        case.update(sel=_log(rng, 4, max(4, min(128, most // (2 * case["page"])))), first=rng.randint(0, 2),
                    last=rng.randint(1, 2))
        low = 2 * case["page"] * case["sel"] if op == "topk" else low  # something to choose from
    case["ctx"] = max(case["tokens"], _log(rng, low, max(most, low + 1)))
    if op in ("attend", "blocks"):
        case["type"] = rng.choice(["f32", "bf16"])
    if op == "blocks":
        case["sel"] = max(4, min(case["sel"], (1 << 24) // (case["seqs"] * case["tokens"] * row * case["page"] // 16)))
    return case


def _lengths(case):
    """New tokens and cached positions (the new ones included) of each sequence: spread, odd, the first the longest."""
    B, T, ctx = case["seqs"], case["tokens"], case["ctx"]
    tokens = [T - (T - 1) * b // max(B - 1, 1) for b in range(B)]
    cached = [max(tokens[b], ctx - (ctx - ctx // 8) * b // max(B - 1, 1)) for b in range(B)]
    return tokens, cached


def _positions(case):
    """The position of every new token, sequence by sequence."""
    tokens, cached = _lengths(case)
    return [c - t + i for t, c in zip(tokens, cached) for i in range(t)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    B, P, D, H, KV = case["seqs"], case["page"], case["head_dim"], case["heads"], case["kv_heads"]
    tokens, cached = _lengths(case)
    N, most = sum(tokens), -(-max(cached) // P)
    need = [-(-c // P) for c in cached]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=host).tolist()
    table = torch.full((B, most), -1, dtype=torch.int32)
    for b in range(B):
        at = sum(need[:b])
        table[b, :need[b]] = torch.tensor(order[at:at + need[b]], dtype=torch.int32)
    starts = [sum(tokens[:b]) for b in range(B + 1)]

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype) * std

    state = {"case": case, "q_start": torch.tensor(starts, dtype=torch.int32, device=dev),
             "ctx_len": torch.tensor(cached, dtype=torch.int32, device=dev), "table": table.to(dev),
             "max_tokens": max(tokens), "max_ctx": max(cached)}
    filled = case["op"] in ("append", "attend", "blocks")  # scores and topk read no keys or values
    make = normal if filled else lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=dev)
    state["k_pages"] = make(pages, KV, D // 8, P, 8)
    state["v_pages"] = make(pages, KV, P // 8, D, 8)
    state["k_means"] = normal(pages, KV, D, std=P ** -0.5)
    if case["op"] == "append":
        # one projection's rows: q, k and v of a token side by side
        qkv = normal(N, (H + 2 * KV) * D, dtype=_DTYPE[case["type"]])
        state["q"] = qkv[:, :H * D].view(N, H, D)
        state["k"] = qkv[:, H * D:(H + KV) * D].view(N, KV, D)
        state["v"] = qkv[:, (H + KV) * D:].view(N, KV, D)
        if case["norm"]:
            state["q_norm"] = torch.rand(D, generator=g, device=dev) + 0.5
            state["k_norm"] = torch.rand(D, generator=g, device=dev) + 0.5
        if case["rope"]:
            half = case["rope"] // 2
            rate = 1e6 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
            angle = torch.arange(state["max_ctx"], dtype=torch.float64, device=dev)[:, None] * rate
            state["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    elif case["op"] in ("attend", "blocks", "scores"):
        state["q"] = normal(N, H, D, std=2.5)  # scores of standard deviation 2.5 after the scale
    if case["op"] in ("scores", "topk"):
        state["scores"] = torch.zeros(N, KV, most, device=dev)
    if case["op"] == "topk":
        # rounded to a grid, so that some pages are level
        state["scores"] = (torch.randn(N, KV, most, generator=g, device=dev) * 64).round() / 16
    if case["op"] == "blocks":
        # what a selection gives: the first and the last pages of each token and others between, ascending, -1 behind
        sel = torch.full((N, KV, case["sel"]), -1, dtype=torch.int32)
        for n, p in enumerate(_positions(case)):
            last = p // P
            ends = set(range(case["first"])) | set(range(last + 1 - case["last"], last + 1))
            rest = [j for j in range(last + 1) if j not in ends]
            for h in range(KV):
                take = list(range(last + 1))
                if last + 1 > case["sel"]:
                    at = torch.randperm(len(rest), generator=host)[:case["sel"] - len(ends)].tolist()
                    take = sorted(ends | {rest[i] for i in at})
                sel[n, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
        state["sel"] = sel.to(dev)
    return state


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "attend": _attend, "scores": _scores, "topk": _topk, "blocks": _blocks}[
        state["case"]["op"]](state)


def _run_own(state):
    from bf16_hyper_connection_amd import paged
    case = state["case"]
    if "cache" not in state:
        state["cache"] = paged.PagedCache(state["k_pages"], state["v_pages"], state["k_means"])
        state["batch"] = paged.Batch(state["q_start"], state["ctx_len"], state["table"], state["max_tokens"],
                                     state["max_ctx"])
    cache, batch = state["cache"], state["batch"]
    if case["op"] == "append":
        q = cache.append(batch, state["q"], state["k"], state["v"], q_norm=state.get("q_norm"),
                         k_norm=state.get("k_norm"), eps=1e-6, rope=state.get("rope"), interleaved=case["pairs"])
        return {"q": q, "k_pages": state["k_pages"], "v_pages": state["v_pages"], "k_means": state["k_means"]}
    if case["op"] == "attend":
        return cache.attend(batch, state["q"], out_dtype=_DTYPE[case["type"]])
    if case["op"] == "scores":
        return cache.block_scores(batch, state["q"], scores=state["scores"])
    if case["op"] == "topk":
        return cache.block_topk(batch, state["scores"], case["sel"], n_first=case["first"], n_last=case["last"])
    return cache.attend_blocks(batch, state["q"], state["sel"], out_dtype=_DTYPE[case["type"]])


# ---- the plain forms ----

def _tokens(state):
    """Of every new token: its sequence, its index in the window and its position."""
    start, N = state["q_start"].long(), state["q_start"].shape[0] - 1
    total = state["q"].shape[0] if "q" in state else state["scores"].shape[0]
    n = torch.arange(total, device=start.device)
    seq = torch.searchsorted(start, n, right=True).clamp(max=N) - 1
    i = n - start[seq]
    return seq, i, state["ctx_len"].long()[seq] - (start[seq + 1] - start[seq]) + i


def _norm_rotate(x, weight, rope, pairs, pos):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
    if rope is not None:
        r = rope.shape[1]
        cos, sin = rope[pos, None, :r // 2], rope[pos, None, r // 2:]
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
        turned = (a * cos - b * sin, b * cos + a * sin)
        turned = torch.stack(turned, -1).flatten(-2) if pairs else torch.cat(turned, -1)
        x = torch.cat([turned, x[..., r:]], -1)
    return x.to(torch.bfloat16)


def _append(state):
    case, P = state["case"], state["case"]["page"]
    kp, vp, means = state["k_pages"], state["v_pages"], state["k_means"]
    seq, _, pos = _tokens(state)
    rope, pairs = state.get("rope"), case["pairs"]
    q = _norm_rotate(state["q"], state.get("q_norm"), rope, pairs, pos)
    k = _norm_rotate(state["k"], state.get("k_norm"), rope, pairs, pos)
    page, slot = state["table"].long()[seq, pos // P], pos % P
    kp[page, :, :, slot, :] = k.unflatten(-1, (-1, 8))
    vp[page, :, slot // 8, :, slot % 8] = state["v"].to(torch.bfloat16)
    # the pages that the window may have completed
    start = state["q_start"].long()
    ctx = state["ctx_len"].long()
    first = (ctx - (start[1:] - start[:-1])) // P
    j = first[:, None] + torch.arange((state["max_tokens"] - 1) // P + 2, device=kp.device)
    done = ((j + 1) * P <= ctx[:, None]).flatten()
    j = j.clamp(max=state["table"].shape[1] - 1)
    at = torch.where(done, state["table"].long().gather(1, j).flatten(), 0)
    mean = kp[at].float().mean(3).flatten(2).to(torch.bfloat16)
    more = torch.cat([means, means[:1]])  # one more row takes what is not complete
    more[torch.where(done, at, means.shape[0])] = mean
    means.copy_(more[:-1])
    return {"q": q, "k_pages": kp, "v_pages": vp, "k_means": means}


def _window(state, x):
    """x [N][...] as [B][T][...], rows past a sequence's window repeated from others."""
    start = state["q_start"].long()
    at = start[:-1, None] + torch.arange(state["max_tokens"], device=start.device)
    return x[at.clamp(max=x.shape[0] - 1)]


def _softmax_of(s):
    """exp(s - max) and its sum along the last axis, rows of -inf alone giving zeros and a sum of one."""
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(m), 0, m))
    total = e.sum(-1, keepdim=True)
    return e, torch.where(total == 0, 1, total)


def _attend(state):
    case = state["case"]
    B, T, KV, D, P = case["seqs"], state["max_tokens"], case["kv_heads"], case["head_dim"], case["page"]
    at = state["table"].long().clamp(min=0)
    L = at.shape[1] * P
    k = state["k_pages"][at].permute(0, 2, 3, 5, 1, 4).reshape(B, KV, D, L).float()       # b h (d8 8) (j P)
    v = state["v_pages"][at].permute(0, 2, 1, 3, 5, 4).reshape(B, KV, L, D).float()       # b h (j P8 8) d
    q = _window(state, state["q"]).float().view(B, T, KV, -1, D).permute(0, 2, 1, 3, 4)   # b h t g d
    s = (q.reshape(B, KV, -1, D) @ k).view(B, KV, T, -1, L) * (D ** -0.5)
    start = state["q_start"].long()
    pos = state["ctx_len"].long()[:, None] - (start[1:] - start[:-1])[:, None] + torch.arange(T, device=q.device)
    seen = torch.arange(L, device=q.device) <= pos[:, None, :, None, None]
    e, total = _softmax_of(s.masked_fill(~seen, -math.inf))
    out = (e.view(B, KV, -1, L) @ v).view(B, KV, T, -1, D) / total
    seq, i, _ = _tokens(state)
    return out.permute(0, 2, 1, 3, 4)[seq, i].flatten(1, 2).to(_DTYPE[case["type"]])


def _scores(state):
    case = state["case"]
    B, T, KV, D, P = case["seqs"], state["max_tokens"], case["kv_heads"], case["head_dim"], case["page"]
    at = state["table"].long().clamp(min=0)
    mean = state["k_means"][at].permute(0, 2, 3, 1).float()                               # b h d j
    q = _window(state, state["q"]).float().view(B, T, KV, -1, D).permute(0, 2, 1, 3, 4)   # b h t g d
    s = (q.reshape(B, KV, -1, D) @ mean).view(B, KV, T, -1, at.shape[1]).amax(3)          # b h t j
    seq, i, pos = _tokens(state)
    before = torch.arange(at.shape[1], device=s.device) < (pos // P)[:, None, None]
    return torch.where(before, s.permute(0, 2, 1, 3)[seq, i], state["scores"])


def _topk(state):
    case, scores = state["case"], state["scores"]
    _, _, pos = _tokens(state)
    last = (pos // case["page"])[:, None, None]
    j = torch.arange(scores.shape[2], device=scores.device).expand_as(scores)
    ends = (j < case["first"]) | (j > last - case["last"])
    rank = torch.where(j > last, 0, torch.where(ends, 2, 1))
    by_score = torch.sort(scores.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf), dim=-1,
                          descending=True, stable=True).indices
    by_rank = torch.sort(rank.gather(-1, by_score), dim=-1, descending=True, stable=True)
    take = by_score.gather(-1, by_rank.indices)[..., :case["sel"]]
    take = torch.where(by_rank.values[..., :case["sel"]] > 0, take, 1 << 40).sort(-1).values
    out = torch.full((*scores.shape[:2], case["sel"]), -1, dtype=torch.int32, device=scores.device)
    out[..., :take.shape[-1]] = torch.where(take == 1 << 40, -1, take).int()
    return out


def _blocks(state):
    case = state["case"]
    KV, D, P = case["kv_heads"], case["head_dim"], case["page"]
    sel, q = state["sel"].long(), state["q"]
    N, L = q.shape[0], sel.shape[2] * P
    seq, _, pos = _tokens(state)
    j = sel.clamp(min=0)
    at = state["table"].long()[seq[:, None, None], j].clamp(min=0)
    head = torch.arange(KV, device=q.device)[None, :, None]
    k = state["k_pages"][at, head].permute(0, 1, 3, 5, 2, 4).reshape(N, KV, D, L).float()
    v = state["v_pages"][at, head].permute(0, 1, 2, 3, 5, 4).reshape(N, KV, L, D).float()
    s = (q.view(N, KV, -1, D).float() @ k) * (D ** -0.5)
    cell = (j[..., None] * P + torch.arange(P, device=q.device)).flatten(2)
    seen = (cell <= pos[:, None, None]) & (sel >= 0).repeat_interleave(P, 2)
    e, total = _softmax_of(s.masked_fill(~seen[:, :, None], -math.inf))
    return ((e @ v) / total).reshape(N, -1, D).to(_DTYPE[case["type"]])


# ---- what a pass cannot do without ----

def work(case):
    tokens, cached = _lengths(case)
    N, H, KV, D, P = sum(tokens), case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    io = N * H * D * (2 + (4 if case.get("type") == "f32" else 2))  # q read, out written
    if case["op"] == "append":
        values = N * (H + 2 * KV) * D
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": values * (size + 2) + N * case["rope"] * 4, "flops": values * 7}
    if case["op"] == "attend":
        # a window's tokens see the positions before them; each cached position is read once
        pairs = sum(t * c - t * (t - 1) // 2 for t, c in zip(tokens, cached))
        return {"bytes": sum(cached) * KV * D * 4 + io, "flops": pairs * H * D * 4}
    if case["op"] == "blocks":
        seen = sum(min(case["sel"] * P, p + 1) for p in _positions(case))
        return {"bytes": seen * KV * D * 4 + io, "flops": seen * H * D * 4}
    before = sum(p // P for p in _positions(case))
    if case["op"] == "scores":
        means = sum(c // P for c in cached)
        return {"bytes": means * KV * D * 2 + N * H * D * 2 + before * KV * 4, "flops": before * H * D * 2}
    return {"bytes": before * KV * 4 + N * KV * case["sel"] * 4, "flops": before * KV}


# ---- the definitions in 64 bits, token by token ----

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "topk":
        return None  # whole numbers: the plain form is exact
    P, KV, D = case["page"], case["kv_heads"], case["head_dim"]
    tokens, cached = _lengths(case)
    table = state["table"].cpu().tolist()
    group = case["heads"] // KV
    if case["op"] == "append":

        def turned(x, weight, pos):
            x = x.double()
            if weight is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.double()
            if not case["rope"]:
                return x
            half = case["rope"] // 2
            row = state["rope"][pos].double()[:, None]
            at = torch.arange(half, device=x.device)
            first, second = (2 * at, 2 * at + 1) if case["pairs"] else (at, at + half)
            y = x.clone()
            y[..., first] = x[..., first] * row[..., :half] - x[..., second] * row[..., half:]
            y[..., second] = x[..., second] * row[..., :half] + x[..., first] * row[..., half:]
            return y

        kp, vp, means = state["k_pages"].double(), state["v_pages"].double(), state["k_means"].double()
        q = torch.zeros_like(state["q"], dtype=torch.float64, memory_format=torch.contiguous_format)
        n = 0
        for b, (t, c) in enumerate(zip(tokens, cached)):
            pos = torch.arange(c - t, c, device=q.device)
            q[n:n + t] = turned(state["q"][n:n + t], state.get("q_norm"), pos)
            k, v = turned(state["k"][n:n + t], state.get("k_norm"), pos), state["v"][n:n + t].double()
            for j in range((c - t) // P, (c - 1) // P + 1):
                low, high = max(c - t, j * P), min(c, (j + 1) * P)
                page, rows = table[b][j], slice(low - (c - t), high - (c - t))
                slots = slice(low - j * P, high - j * P)
                kp[page, :, :, slots] = k[rows].unflatten(-1, (D // 8, 8)).permute(1, 2, 0, 3)
                whole = vp[page].transpose(2, 3).reshape(-1, P, D).clone()
                whole[:, slots] = v[rows].transpose(0, 1)
                vp[page] = whole.unflatten(1, (P // 8, 8)).transpose(2, 3)
                if high == (j + 1) * P:
                    means[page] = kp[page].to(torch.bfloat16).double().mean(2).flatten(1)
            n += t
        return {"q": q, "k_pages": kp, "v_pages": vp, "k_means": means}
    q = state["q"].double()
    if case["op"] == "scores":
        out, n = state["scores"].double(), 0
        for b, (t, c) in enumerate(zip(tokens, cached)):
            mean = state["k_means"][state["table"][b, :max(c // P, 1)].long()].double()   # j h d
            for i in range(t):
                last = (c - t + i) // P
                heads = q[n].view(KV, group, D)
                if last:
                    out[n, :, :last] = torch.einsum("hgd,jhd->hgj", heads, mean[:last]).amax(1)
                n += 1
        return out
    out, n = torch.zeros_like(q), 0
    sel = state["sel"].cpu().tolist() if case["op"] == "blocks" else None
    if sel is not None and len(sel) * KV > 6000:
        return None  # too many small products
    for b, (t, c) in enumerate(zip(tokens, cached)):
        for h in range(KV):
            if sel is None:
                at = torch.tensor(table[b][:-(-c // P)], device=q.device)
                k = state["k_pages"][at, h].double().transpose(1, 2).reshape(-1, D)
                v = state["v_pages"][at, h].double().transpose(2, 3).reshape(-1, D)
            for i in range(t):
                pos = c - t + i
                if sel is None:
                    keys, values = k[:pos + 1], v[:pos + 1]
                else:
                    js = [j for j in sel[n + i][h] if j >= 0]
                    at = torch.tensor([table[b][j] for j in js], device=q.device)
                    cell = (torch.tensor(js, device=q.device)[:, None] * P + torch.arange(P, device=q.device)).flatten()
                    keys = state["k_pages"][at, h].double().transpose(1, 2).reshape(-1, D)[cell <= pos]
                    values = state["v_pages"][at, h].double().transpose(2, 3).reshape(-1, D)[cell <= pos]
                heads = q[n + i, h * group:(h + 1) * group]
                out[n + i, h * group:(h + 1) * group] = torch.softmax(heads @ keys.T / math.sqrt(D), -1) @ values
        n += t
    return out
