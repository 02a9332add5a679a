"""The paged cache in 8 bits, and attention over a sliding window, as cases to be timed and compared.

A cache of half the bytes: keys and values are held as int8 or E4M3 codes with an FP32 scale for each position and kv
head, quantised as they are appended (append) and read back as rows (read); attention runs over the codes (attend, and
blocks over listed pages).  Attention over a sliding window and a few first positions (window) runs over either cache.
``run`` computes each operator in elementary torch operations, or, where ``own`` is set, through
bf16_hyper_connection_amd.paged.

Page layouts in 8 bits: keys [page][kv head][D / 16][P][16], values [page][kv head][P / 16][D][16], scales of each
[page][kv head][P]; in BF16 the same with 8 in the place of 16 and no scales.  Mean keys [page][kv head][D].
"""

import math

import torch

own = False

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_CODES = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_TOP = {"int8": 127.0, "e4m3": 448.0}  # the largest code


def listed():
    attn_q = {"heads": 48, "kv_heads": 8, "head_dim": 256, "page": 64}    # 12288 rows, the skinny matvec's projection
    common = {"heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64}    # a usual grouped geometry
    return [
        # the smallest step of a decode loop: one token's heads, where latency counts
        {"name": "append, one token, e4m3", "op": "append", "cache": "e4m3", "seqs": 1, "tokens": 1, "ctx": 1000,
         **attn_q, "type": "f32", "rope": 64, "pairs": False, "norm": True},
        # prompts of unlike lengths going into the cache behind earlier tokens, rotation over whole heads
        {"name": "append, prompts, e4m3", "op": "append", "cache": "e4m3", "seqs": 3, "tokens": 2900, "ctx": 4500,
         **common, "type": "bf16", "rope": 128, "pairs": True, "norm": True},
        # verify windows of a batch, written and read back as attention will see them
        {"name": "append and read, int8", "op": "append", "cache": "int8", "seqs": 32, "tokens": 6, "ctx": 5000,
         **attn_q, "type": "f32", "rope": 64, "pairs": False, "norm": True},
        # whole sequences read back as BF16 rows
        {"name": "read, sequences, int8", "op": "read", "cache": "int8", "seqs": 8, "tokens": 8192, "ctx": 8192,
         **common, "type": "bf16"},
        # one short conversation, one token
        {"name": "attend, one short, int8", "op": "attend", "cache": "int8", "seqs": 1, "tokens": 1, "ctx": 700,
         **common, "type": "f32"},
        # verify windows of up to six tokens over a few conversations of odd lengths
        {"name": "attend, windows, int8", "op": "attend", "cache": "int8", "seqs": 4, "tokens": 6, "ctx": 9001,
         **attn_q, "type": "f32"},
        # a serving batch of single tokens over lengths from a thousand to eight thousand
        {"name": "attend, batch, int8", "op": "attend", "cache": "int8", "seqs": 64, "tokens": 1, "ctx": 8192,
         **common, "type": "bf16"},
        # the longest context: two tokens over 420,000 positions
        {"name": "attend, long, e4m3", "op": "attend", "cache": "e4m3", "seqs": 1, "tokens": 2, "ctx": 420000,
         **attn_q, "type": "f32"},
        # a serving batch whose layer sees the last 4,096 positions and the first four; pages between are given back
        {"name": "window, batch, bf16", "op": "window", "cache": "bf16", "seqs": 64, "tokens": 1, "ctx": 32768,
         **common, "type": "bf16", "window": 4096, "first": 4},
        # prompts going through such a layer
        {"name": "window, prompts, bf16", "op": "window", "cache": "bf16", "seqs": 2, "tokens": 2048, "ctx": 4096,
         **common, "type": "bf16", "window": 1024, "first": 4},
        # a verify window far into a long context
        {"name": "window, long, int8", "op": "window", "cache": "int8", "seqs": 1, "tokens": 4, "ctx": 420000,
         **attn_q, "type": "f32", "window": 8192, "first": 64},
        # attention over 64 of 6,562 pages, a window of four tokens
        {"name": "blocks, long, int8", "op": "blocks", "cache": "int8", "seqs": 1, "tokens": 4, "ctx": 420000,
         **attn_q, "type": "f32", "sel": 64, "ends": 2},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attend", "attend", "window", "window", "blocks"])
    kv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "cache": rng.choice(["int8", "e4m3"]), "seqs": _log(rng, 1, 64), "kv_heads": kv,
            "heads": kv * rng.choice([1, 2, 4, 5, 6, 8, 12, 16]), "head_dim": rng.choice([64, 128, 256]),
            "page": rng.choice([64, 128, 256])}
    if op in ("read", "window") and rng.random() < 0.4:
        case.update(cache="bf16", page=rng.choice([32, 64, 128]))
    row = kv * case["head_dim"]
    if op == "append":
        case["tokens"] = max(1, min(_log(rng, 1, 3000), 9000 // case["seqs"]))
        case["ctx"] = case["tokens"] + _log(rng, 1, 2000)
        case.update(type=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.8, pairs=rng.random() < 0.5,
                    rope=rng.choice([0, 16, case["head_dim"] // 2, case["head_dim"]]))
        return case
    case["type"] = rng.choice(["f32", "bf16"])
    if op == "read":
        case["tokens"] = max(1, min(_log(rng, 1, 20000), 65536 * 1024 // (row * case["seqs"])))
        case["ctx"] = case["tokens"] + rng.choice([0, _log(rng, 1, 500)])
        return case
    case["tokens"] = rng.randint(1, 16) if rng.random() < 0.6 else 1
    if op == "window":
        if rng.random() < 0.25:  # prompts
            case["seqs"] = rng.randint(1, 3)
            case["tokens"] = min(_log(rng, 64, 2048), (1 << 25) // (case["seqs"] * case["heads"] * 512))
        case["window"] = _log(rng, 16, min(8192, max(64, 10 ** 8 // (case["seqs"] * case["tokens"] * case["heads"]))))
        case["first"] = rng.choice([0, 1, 4, rng.randint(5, 200)])
        most = max(case["tokens"], min(100000, 10 ** 8 // row))
        case["ctx"] = max(case["tokens"], _log(rng, 64, most))
        return case
    # no more cached values than the longest listed case has, shared among the sequences
    most = min(420000, 420000 * 2048 // (row * case["seqs"]), 10 ** 8 // (case["seqs"] * case["tokens"] * case["heads"]))
    if op == "blocks":
        most = min(most, 420000 // case["seqs"])
        case.update(sel=_log(rng, 4, max(4, min(128, most // (2 * case["page"])))), ends=rng.randint(1, 2))
        case["sel"] = max(4, min(case["sel"], (1 << 24) // (case["seqs"] * case["tokens"] * row * case["page"] // 16)))
    case["ctx"] = max(case["tokens"], _log(rng, 64, max(most, 65)))
    return case


def _lengths(case):
    """New tokens and cached positions (the new ones included) of each sequence: spread, odd, the first the longest."""
    B, T, ctx = case["seqs"], case["tokens"], case["ctx"]
    tokens = [T - (T - 1) * b // max(B - 1, 1) for b in range(B)]
    if case["op"] == "read":
        tokens = [max(1, T - T * b // (2 * B)) for b in range(B)]
    cached = [max(tokens[b], ctx - (ctx - ctx // 8) * b // max(B - 1, 1)) for b in range(B)]
    return tokens, cached


def _kept(case):
    """Of each sequence the pages that are held: all, or those that a window or its first positions still touch."""
    P, kept = case["page"], []
    for t, c in zip(*_lengths(case)):
        pages = list(range(-(-c // P)))
        if case["op"] == "window":
            low = max(0, c - t + 1 - case["window"])
            pages = [j for j in pages if j * P < case["first"] or (j + 1) * P > low]
        kept.append(pages)
    return kept


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    B, P, D, H, KV = case["seqs"], case["page"], case["head_dim"], case["heads"], case["kv_heads"]
    tokens, cached = _lengths(case)
    N, most = sum(tokens), -(-max(cached) // P)
    kept = _kept(case)
    pages = sum(len(k) for k in kept) + 3
    order = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(kept):
        table[b, torch.tensor(k)] = order[at:at + len(k)]
        at += len(k)
    starts = [sum(tokens[:b]) for b in range(B + 1)]

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype) * std

    def codes(*shape):
        if case["cache"] == "bf16":
            return normal(*shape)
        x = torch.randn(shape, generator=g, device=dev).mul_(_TOP[case["cache"]] / 3.2)
        x = x.clamp_(-_TOP[case["cache"]], _TOP[case["cache"]])
        return (x.round_() if case["cache"] == "int8" else x).to(_CODES[case["cache"]])

    each = 8 if case["cache"] == "bf16" else 16
    state = {"case": case, "q_start": torch.tensor(starts, dtype=torch.int32, device=dev),
             "ctx_len": torch.tensor(cached, dtype=torch.int32, device=dev), "table": table.to(dev),
             "max_tokens": max(tokens), "max_ctx": max(cached), "n_tokens": N,
             "k_pages": codes(pages, KV, D // each, P, each), "v_pages": codes(pages, KV, P // each, D, each),
             "k_means": normal(pages, KV, D, std=P ** -0.5)}
    if each == 16:  # largest values of 2.4 to 4.8 standard deviations
        for name in ("k_scales", "v_scales"):
            state[name] = (torch.rand(pages, KV, P, generator=g, device=dev) + 1) * (2.4 / _TOP[case["cache"]])
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
    elif case["op"] != "read":
        state["q"] = normal(N, H, D, std=2.5)  # scores of standard deviation 2.5 after the scale
    if case["op"] == "blocks":
        # what a selection gives: the first page and the last ones of each token, others between, ascending, -1 behind
        sel = torch.full((N, KV, case["sel"]), -1, dtype=torch.int32)
        for n, p in enumerate(_positions(case)):
            last = p // P
            ends = {0} | set(range(max(0, last + 1 - case["ends"]), last + 1))
            rest = [j for j in range(last + 1) if j not in ends]
            for h in range(KV):
                take = list(range(last + 1))
                if last + 1 > case["sel"]:
                    at = torch.randperm(len(rest), generator=host)[:case["sel"] - len(ends)].tolist()
                    take = sorted(ends | {rest[i] for i in at})
                sel[n, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
        state["sel"] = sel.to(dev)
    return state


def _positions(case):
    """The position of every new token, sequence by sequence."""
    tokens, cached = _lengths(case)
    return [c - t + i for t, c in zip(tokens, cached) for i in range(t)]


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "read": _read, "attend": _attend, "window": _window, "blocks": _blocks}[
        state["case"]["op"]](state)


def _run_own(state):
    from bf16_hyper_connection_amd import paged
    case = state["case"]
    if "cache" not in state:
        state["cache"] = paged.PagedCache(state["k_pages"], state["v_pages"], state["k_means"],
                                          k_scales=state.get("k_scales"), v_scales=state.get("v_scales"))
        state["batch"] = paged.Batch(state["q_start"], state["ctx_len"], state["table"], state["max_tokens"],
                                     state["max_ctx"])
    cache, batch, dtype = state["cache"], state["batch"], _DTYPE[case["type"]]
    if case["op"] == "append":
        q = cache.append(batch, state["q"], state["k"], state["v"], q_norm=state.get("q_norm"),
                         k_norm=state.get("k_norm"), eps=1e-6, rope=state.get("rope"), interleaved=case["pairs"])
        out = {"q": q, "k_scales": state["k_scales"], "v_scales": state["v_scales"], "k_means": state["k_means"]}
        if case["cache"] == "e4m3":
            return {**out, "k_pages": state["k_pages"], "v_pages": state["v_pages"]}
        out["k"], out["v"] = cache.read(batch, state["n_tokens"], out_dtype=torch.bfloat16)
        return out
    if case["op"] == "read":
        return cache.read(batch, state["n_tokens"], out_dtype=dtype)
    if case["op"] == "attend":
        return cache.attend(batch, state["q"], out_dtype=dtype)
    if case["op"] == "window":
        return cache.attend_window(batch, state["q"], case["window"], n_first=case["first"], out_dtype=dtype)
    return cache.attend_blocks(batch, state["q"], state["sel"], out_dtype=dtype)


# ---- the plain forms ----

def _tokens(state):
    """Of every new token: its sequence, its index in the window and its position."""
    start = state["q_start"].long()
    n = torch.arange(state["n_tokens"], device=start.device)
    seq = torch.searchsorted(start, n, right=True).clamp(max=start.shape[0] - 1) - 1
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
    return x


def _quantised(x, cache):
    """Codes of the cache's type and the scale of each head: the largest value is the largest code."""
    scale = x.abs().amax(-1) / _TOP[cache]
    y = torch.where(scale[..., None] > 0, x / scale[..., None], 0).clamp(-_TOP[cache], _TOP[cache])
    return (y.round() if cache == "int8" else y).to(_CODES[cache]), scale


def _raw(codes):
    """Codes as bytes, which every indexing takes."""
    return codes if codes.dtype == torch.bfloat16 else codes.view(torch.uint8)


def _append(state):
    case, P, D, KV = state["case"], state["case"]["page"], state["case"]["head_dim"], state["case"]["kv_heads"]
    kp, vp, ks, vs, means = (state[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales", "k_means"))
    seq, _, pos = _tokens(state)
    rope, pairs = state.get("rope"), case["pairs"]
    q = _norm_rotate(state["q"], state.get("q_norm"), rope, pairs, pos).to(torch.bfloat16)
    k, k_scale = _quantised(_norm_rotate(state["k"], state.get("k_norm"), rope, pairs, pos), case["cache"])
    v, v_scale = _quantised(state["v"].float(), case["cache"])
    page, slot = state["table"].long()[seq, pos // P], pos % P
    _raw(kp)[page, :, :, slot, :] = _raw(k).unflatten(-1, (-1, 16))
    _raw(vp)[page, :, slot // 16, :, slot % 16] = _raw(v)
    ks[page, :, slot] = k_scale
    vs[page, :, slot] = v_scale
    # the pages that the window may have completed
    start = state["q_start"].long()
    ctx = state["ctx_len"].long()
    first = (ctx - (start[1:] - start[:-1])) // P
    j = first[:, None] + torch.arange((state["max_tokens"] - 1) // P + 2, device=kp.device)
    done = ((j + 1) * P <= ctx[:, None]).flatten()
    j = j.clamp(max=state["table"].shape[1] - 1)
    at = torch.where(done, state["table"].long().gather(1, j).flatten(), 0)
    mean = (_raw(kp)[at].view(kp.dtype).float() * ks[at][:, :, None, :, None]).mean(3).flatten(2).to(torch.bfloat16)
    more = torch.cat([means, means[:1]])  # one more row takes what is not complete
    more[torch.where(done, at, means.shape[0])] = mean
    means.copy_(more[:-1])
    out = {"q": q, "k_scales": ks, "v_scales": vs, "k_means": means}
    if case["cache"] == "e4m3":
        return {**out, "k_pages": kp, "v_pages": vp}
    stand = torch.bfloat16
    return {**out, "k": (k.float() * k_scale[..., None]).to(stand), "v": (v.float() * v_scale[..., None]).to(stand)}


def _read(state):
    case, P, D, KV = state["case"], state["case"]["page"], state["case"]["head_dim"], state["case"]["kv_heads"]
    seq, _, pos = _tokens(state)
    page, slot = state["table"].long()[seq, pos // P], pos % P
    each = state["k_pages"].shape[-1]
    kp, vp = _raw(state["k_pages"]), _raw(state["v_pages"])
    k = kp[page, :, :, slot, :].reshape(-1, KV, D).view(state["k_pages"].dtype).float()
    v = vp[page, :, slot // each, :, slot % each].view(state["k_pages"].dtype).float()
    if "k_scales" in state:
        k = k * state["k_scales"][page, :, slot][..., None]
        v = v * state["v_scales"][page, :, slot][..., None]
    return k.to(_DTYPE[case["type"]]), v.to(_DTYPE[case["type"]])


def _softmax_of(s):
    """exp(s - max) and its sum along the last axis, rows of -inf alone giving zeros and a sum of one."""
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(m), 0, m))
    total = e.sum(-1, keepdim=True)
    return e, torch.where(total == 0, 1, total)


def _over(state, at, seen):
    """Attention of each sequence's window over the pages at [B][n], seen [B][T][n P]."""
    case = state["case"]
    B, T, KV, D, P = case["seqs"], state["max_tokens"], case["kv_heads"], case["head_dim"], case["page"]
    L, dtype = at.shape[1] * P, state["k_pages"].dtype
    start = state["q_start"].long()
    k = _raw(state["k_pages"])[at].view(dtype).permute(0, 2, 3, 5, 1, 4).float()   # b h (d8 8) (j P)
    v = _raw(state["v_pages"])[at].view(dtype).permute(0, 2, 1, 3, 5, 4).float()   # b h (j P8 8) d
    k, v = k.reshape(B, KV, D, L), v.reshape(B, KV, L, D)
    if "k_scales" in state:
        k = k * state["k_scales"][at].permute(0, 2, 1, 3).reshape(B, KV, 1, L)
        v = v * state["v_scales"][at].permute(0, 2, 1, 3).reshape(B, KV, L, 1)
    rows = start[:-1, None] + torch.arange(T, device=start.device)  # past a sequence's window repeated from others
    q = state["q"][rows.clamp(max=state["n_tokens"] - 1)].float().view(B, T, KV, -1, D).permute(0, 2, 1, 3, 4)
    s = (q.reshape(B, KV, -1, D) @ k).view(B, KV, T, -1, L) * (D ** -0.5)
    e, total = _softmax_of(s.masked_fill(~seen[:, None, :, None], -math.inf))
    out = (e.view(B, KV, -1, L) @ v).view(B, KV, T, -1, D) / total
    seq, i, _ = _tokens(state)
    return out.permute(0, 2, 1, 3, 4)[seq, i].flatten(1, 2).to(_DTYPE[case["type"]])


def _window_positions(state):
    start, T = state["q_start"].long(), state["max_tokens"]
    return (state["ctx_len"].long() - (start[1:] - start[:-1]))[:, None] + torch.arange(T, device=start.device)


def _attend(state):
    at = state["table"].long().clamp(min=0)
    cell = torch.arange(at.shape[1] * state["case"]["page"], device=at.device)
    return _over(state, at, cell <= _window_positions(state)[..., None])


def _window(state):
    case, P, table = state["case"], state["case"]["page"], state["table"].long()
    pos = _window_positions(state)[..., None]
    # the pages of the first positions, then those that the sequence's windows touch
    firsts = min(-(-case["first"] // P), table.shape[1])
    low = (pos[:, 0] + 1 - case["window"]).clamp(min=0) // P
    more = min((case["window"] + state["max_tokens"] - 2) // P + 2, table.shape[1])
    j = torch.cat([torch.arange(firsts, device=table.device).expand(table.shape[0], -1),
                   low + torch.arange(more, device=table.device)], 1)
    once = (torch.arange(firsts + more, device=table.device) < firsts) | ((j >= firsts) & (j < table.shape[1]))
    cell = (j[..., None] * P + torch.arange(P, device=table.device)).flatten(1)[:, None]
    seen = (cell <= pos) & ((cell > pos - case["window"]) | (cell < case["first"]))
    seen &= once.repeat_interleave(P, 1)[:, None]
    return _over(state, table.gather(1, j.clamp(max=table.shape[1] - 1)).clamp(min=0), seen)


def _blocks(state):
    case = state["case"]
    KV, D, P = case["kv_heads"], case["head_dim"], case["page"]
    sel, q, dtype = state["sel"].long(), state["q"], state["k_pages"].dtype
    N, L = q.shape[0], sel.shape[2] * P
    seq, _, pos = _tokens(state)
    j = sel.clamp(min=0)
    at = state["table"].long()[seq[:, None, None], j].clamp(min=0)
    head = torch.arange(KV, device=q.device)[None, :, None]
    k = _raw(state["k_pages"])[at, head].view(dtype).permute(0, 1, 3, 5, 2, 4).float()
    v = _raw(state["v_pages"])[at, head].view(dtype).permute(0, 1, 2, 3, 5, 4).float()
    k = k.reshape(N, KV, D, L) * state["k_scales"][at, head].reshape(N, KV, 1, L)
    v = v.reshape(N, KV, L, D) * state["v_scales"][at, head].reshape(N, KV, L, 1)
    s = (q.view(N, KV, -1, D).float() @ k) * (D ** -0.5)
    cell = (j[..., None] * P + torch.arange(P, device=q.device)).flatten(2)
    seen = (cell <= pos[:, None, None]) & (sel >= 0).repeat_interleave(P, 2)
    e, total = _softmax_of(s.masked_fill(~seen[:, :, None], -math.inf))
    return ((e @ v) / total).reshape(N, -1, D).to(_DTYPE[case["type"]])


# ---- what a pass cannot do without ----

def work(case):
    tokens, cached = _lengths(case)
    N, H, KV, D, P = sum(tokens), case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    cell = KV * (D * 2 if case["cache"] == "bf16" else D + 4)  # bytes of a position's keys, or of its values
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "append":
        bytes_ = N * (H + 2 * KV) * D * size + N * H * D * 2 + 2 * N * cell + N * case["rope"] * 4
        if case["cache"] == "int8":
            bytes_ += 2 * N * KV * D * 2
        return {"bytes": bytes_, "flops": N * (H + 2 * KV) * D * 8}
    if case["op"] == "read":
        return {"bytes": 2 * N * (cell + KV * D * size), "flops": 2 * N * KV * D}
    io = N * H * D * (2 + size)  # q read, out written
    if case["op"] == "attend":
        # a window's tokens see the positions before them; each cached position is read once
        pairs = sum(t * c - t * (t - 1) // 2 for t, c in zip(tokens, cached))
        return {"bytes": 2 * sum(cached) * cell + io, "flops": pairs * H * D * 4}
    if case["op"] == "blocks":
        seen = sum(min(case["sel"] * P, p + 1) for p in _positions(case))
        return {"bytes": 2 * seen * cell + io, "flops": seen * H * D * 4}
    W, F = case["window"], case["first"]
    pairs = sum(min(p + 1, W) + min(max(p + 1 - W, 0), F) for p in _positions(case))
    held = 0
    for t, c in zip(tokens, cached):
        low = max(0, c - t + 1 - W)
        held += c - low + min(low, F)
    return {"bytes": 2 * held * cell + io, "flops": pairs * H * D * 4}


# ---- the definitions in 64 bits, sequence by sequence ----

def _nearest(x, cache):
    """The code nearest to each value, ties to even, in 64 bits."""
    if cache == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def exact(case, seed):
    state = prepare(case, seed)
    P, KV, D = case["page"], case["kv_heads"], case["head_dim"]
    tokens, cached = _lengths(case)
    table = state["table"].cpu().tolist()
    group = case["heads"] // KV
    dtype = state["k_pages"].dtype

    def keys_of(pages, h):
        """Keys of a kv head in these pages, [positions][D], and the values."""
        at = torch.tensor(pages, device=state["table"].device)
        k = _raw(state["k_pages"])[at, h].view(dtype).double().transpose(1, 2).reshape(-1, D)
        v = _raw(state["v_pages"])[at, h].view(dtype).double().transpose(2, 3).reshape(-1, D)
        if "k_scales" in state:
            k = k * state["k_scales"][at, h].double().reshape(-1, 1)
            v = v * state["v_scales"][at, h].double().reshape(-1, 1)
        return k, v

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

        kp, vp = state["k_pages"].double(), state["v_pages"].double()
        ks, vs, means = (state[n].double() for n in ("k_scales", "v_scales", "k_means"))
        q = torch.zeros_like(state["q"], dtype=torch.float64, memory_format=torch.contiguous_format)
        stand = {"k": [], "v": []}
        n = 0
        for b, (t, c) in enumerate(zip(tokens, cached)):
            pos = torch.arange(c - t, c, device=q.device)
            q[n:n + t] = turned(state["q"][n:n + t], state.get("q_norm"), pos)
            k, v = turned(state["k"][n:n + t], state.get("k_norm"), pos), state["v"][n:n + t].double()
            k_top, v_top = (x.abs().amax(-1) / _TOP[case["cache"]] for x in (k, v))
            k_codes, v_codes = k / k_top[..., None], v / v_top[..., None]
            k_near = _nearest(k_codes, case["cache"])
            if case["cache"] == "int8":
                stand["k"].append(k_near * k_top[..., None])
                stand["v"].append(_nearest(v_codes, "int8") * v_top[..., None])
            for j in range((c - t) // P, (c - 1) // P + 1):
                low, high = max(c - t, j * P), min(c, (j + 1) * P)
                page, rows = table[b][j], slice(low - (c - t), high - (c - t))
                slots = slice(low - j * P, high - j * P)
                if high == (j + 1) * P:
                    whole = kp[page].transpose(1, 2).reshape(KV, P, D) * ks[page][..., None]
                    whole[:, slots] = (k_near * k_top[..., None])[rows].transpose(0, 1)
                    means[page] = whole.mean(1)
                ks[page, :, slots], vs[page, :, slots] = k_top[rows].T, v_top[rows].T
                kp[page, :, :, slots] = k_codes[rows].unflatten(-1, (D // 16, 16)).permute(1, 2, 0, 3)
                whole = vp[page].transpose(2, 3).reshape(-1, P, D).clone()
                whole[:, slots] = v_codes[rows].transpose(0, 1)
                vp[page] = whole.unflatten(1, (P // 16, 16)).transpose(2, 3)
            n += t
        out = {"q": q, "k_scales": ks, "v_scales": vs, "k_means": means}
        if case["cache"] == "e4m3":
            return {**out, "k_pages": kp, "v_pages": vp}  # before their rounding to codes
        return {**out, "k": torch.cat(stand["k"]), "v": torch.cat(stand["v"])}
    if case["op"] == "read":
        parts = []
        for b, (t, c) in enumerate(zip(tokens, cached)):
            heads = [keys_of(table[b][:-(-c // P)], h) for h in range(KV)]
            parts.append([torch.stack([x[i][c - t:c] for x in heads], 1) for i in (0, 1)])
        return tuple(torch.cat([p[i] for p in parts]) for i in (0, 1))
    q = state["q"].double()
    if sum(tokens) * KV > 40000:
        return None  # too many small products
    out, n = torch.zeros_like(q), 0
    sel = state["sel"].cpu().tolist() if case["op"] == "blocks" else None
    kept = _kept(case)
    for b, (t, c) in enumerate(zip(tokens, cached)):
        cells = torch.cat([torch.arange(j * P, (j + 1) * P, device=q.device) for j in kept[b]])
        for h in range(KV):
            if sel is None:
                k, v = keys_of([table[b][j] for j in kept[b]], h)
            for i in range(t):
                pos = c - t + i
                if sel is not None:
                    js = [j for j in sel[n + i][h] if j >= 0]
                    keys, values = keys_of([table[b][j] for j in js], h)
                    at = torch.cat([torch.arange(j * P, (j + 1) * P, device=q.device) for j in js]) <= pos
                    keys, values = keys[at], values[at]
                elif case["op"] == "window":
                    at = (cells <= pos) & ((cells > pos - case["window"]) | (cells < case["first"]))
                    keys, values = k[at], v[at]
                else:
                    keys, values = k[:pos + 1], v[:pos + 1]
                heads = q[n + i, h * group:(h + 1) * group]
                out[n + i, h * group:(h + 1) * group] = torch.softmax(heads @ keys.T / math.sqrt(D), -1) @ values
        n += t
    return out
