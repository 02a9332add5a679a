"""FP64 CPU reference of the paged key-value cache: append, attention, page scores and page selection.

TEST INFRASTRUCTURE. Only ``tests/`` may import or call this module. It shares
no code with the HIP path and imports nothing from it.

A batch is (q_start, ctx_len, table): sequence b's new tokens are the rows
q_start[b] .. q_start[b + 1] - 1, the i-th of T_b at position
ctx_len[b] - T_b + i; position p lives in slot p % page of page
table[b][p // page] (a number outside the cache: nowhere).  Pages are given
decoded, keys and values [n_pages][kv_heads][page][D] (``decode_keys``,
``decode_values`` undo the stored orders [D / 8][page][8] and
[page / 8][D][8]).
"""

import numpy as np

from .reference import bf16_bits_to_f64


def decode_keys(bits):
    """uint16 [n][h][D / 8][page][8] -> float64 [n][h][page][D]."""
    n, h, c, page, _ = bits.shape
    return bf16_bits_to_f64(np.ascontiguousarray(bits.transpose(0, 1, 3, 2, 4)).reshape(n, h, page, c * 8))


def decode_values(bits):
    """uint16 [n][h][page / 8][D][8] -> float64 [n][h][page][D]."""
    n, h, o, d, _ = bits.shape
    return bf16_bits_to_f64(np.ascontiguousarray(bits.transpose(0, 1, 2, 4, 3)).reshape(n, h, o * 8, d))


def tokens(q_start, ctx_len):
    """(row, sequence, position) of every new token."""
    out = []
    for b in range(len(ctx_len)):
        t = int(q_start[b + 1]) - int(q_start[b])
        out += [(int(q_start[b]) + i, b, int(ctx_len[b]) - t + i) for i in range(t)]
    return out


def norm_rotate(x, weight, eps, rope_row, pairs):
    """One head's values x [D] normalised (weight None: as they are) and rotated by a table row (None: not)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x * np.asarray(weight, np.float64) / np.sqrt(np.mean(x * x) + eps)
    if rope_row is None or len(rope_row) == 0:
        return x.copy()
    half = len(rope_row) // 2
    cos, sin = np.asarray(rope_row[:half], np.float64), np.asarray(rope_row[half:], np.float64)
    y = x.copy()
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if pairs else (j, j + half)
        y[a] = x[a] * cos[j] - x[b] * sin[j]
        y[b] = x[b] * cos[j] + x[a] * sin[j]
    return y


def append(batch, page, n_pages, q, k, v, q_norm, k_norm, eps, rope, pairs):
    """(q_out [rows][heads][D] or None per row, writes): q_out rows of tokens at negative positions are zeros;
    writes maps (page number, slot) to (k [h][D], v [h][D])."""
    q_start, ctx_len, table = batch
    q_out, writes = {}, {}
    for n, b, p in tokens(q_start, ctx_len):
        if p < 0:
            q_out[n] = np.zeros(q[n].shape)
            continue
        row = None if rope is None else rope[p]
        q_out[n] = np.stack([norm_rotate(x, q_norm, eps, row, pairs) for x in q[n]])
        at = int(table[b][p // page])
        if 0 <= at < n_pages:
            writes[at, p % page] = (np.stack([norm_rotate(x, k_norm, eps, row, pairs) for x in k[n]]),
                                    np.asarray(v[n], np.float64))
    return q_out, writes


def completed(batch, page, n_pages):
    """Pages whose last slot a new token fills."""
    q_start, ctx_len, table = batch
    done = [int(table[b][p // page]) for _, b, p in tokens(q_start, ctx_len) if p >= 0 and p % page == page - 1]
    return [j for j in done if 0 <= j < n_pages]


def _softmax_rows(s):
    e = np.exp(s - s.max(axis=-1, keepdims=True))
    return e / e.sum(axis=-1, keepdims=True)


def attend(batch, keys, values, q, scale, sel=None):
    """out[row] = [heads][D] for every new token; ``sel`` [rows][kv_heads][n_sel] lists pages (None: all)."""
    q_start, ctx_len, table = batch
    n_pages, kv_heads, page, D = keys.shape
    out = {}
    for n, b, p in tokens(q_start, ctx_len):
        heads = q[n].shape[0]
        group = heads // kv_heads
        out[n] = np.zeros((heads, D))
        for h in range(kv_heads):
            listed = range(p // page + 1) if sel is None else [int(j) for j in sel[n][h]]
            ks, vs = [], []
            for j in listed:
                if j < 0 or j * page > p or not 0 <= int(table[b][j]) < n_pages:
                    continue
                seen = min(page, p + 1 - j * page)
                ks.append(keys[int(table[b][j]), h, :seen])
                vs.append(values[int(table[b][j]), h, :seen])
            if p < 0 or not ks:
                continue
            kk, vv = np.concatenate(ks), np.concatenate(vs)
            out[n][h * group:(h + 1) * group] = _softmax_rows(
                scale * (np.asarray(q[n][h * group:(h + 1) * group], np.float64) @ kk.T)) @ vv
    return out


def block_scores(batch, means, page, q):
    """scores[row] = [kv_heads][p // page], means float64 [n_pages][kv_heads][D]."""
    q_start, ctx_len, table = batch
    n_pages, kv_heads, D = means.shape
    out = {}
    for n, b, p in tokens(q_start, ctx_len):
        before = max(p, 0) // page
        group = q[n].shape[0] // kv_heads
        s = np.full((kv_heads, before), -np.inf)
        for j in range(before):
            at = int(table[b][j])
            if 0 <= at < n_pages:
                for h in range(kv_heads):
                    s[h, j] = np.max(np.asarray(q[n][h * group:(h + 1) * group], np.float64) @ means[at, h])
        out[n] = s
    return out


def block_topk(batch, page, scores, n_sel, n_first, n_last):
    """sel[row] = [kv_heads][n_sel] from scores [rows][kv_heads][pages]."""
    q_start, ctx_len, _ = batch
    out = {}
    for n, _, p in tokens(q_start, ctx_len):
        count = p // page + 1 if p >= 0 else 0
        rows = []
        for h in range(scores.shape[1]):
            take = list(range(count))
            if count > n_sel:
                ends = list(range(n_first)) + list(range(count - n_last, count))

                def order(j, s=scores[n, h]):
                    x = float(s[j])
                    return (-x if x == x else np.inf, j)  # highest first, NaN as -inf, then the lowest index
                between = sorted(range(n_first, count - n_last), key=order)
                take = sorted(ends + between[:n_sel - len(ends)])
            rows.append(take + [-1] * (n_sel - len(take)))
        out[n] = np.array(rows, dtype=np.int32)
    return out
