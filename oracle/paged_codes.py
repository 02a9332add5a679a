"""FP64 CPU reference of the paged cache's other forms: 8-bit codes with a scale for each position and kv head, reading
a cache back, and attention over a sliding window with a few first positions.

TEST INFRASTRUCTURE. Only ``tests/`` may import or call this module. It shares
no code with the HIP path and imports nothing from it.

A head of values x stands as codes and a scale: scale = max |x| / TOP, code = the code nearest to x / scale (ties to the
one whose last bit is zero).  A head that holds a value that is not finite has the scale NaN and codes of zero; zeros
have the scale 0.  Stored orders: keys [n][h][D / 16][page][16], values [n][h][page / 16][D][16], scales [n][h][page].
Batches are as in ``paged``.
"""

import numpy as np

from .paged import tokens

TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_table():
    """What each of the 256 E4M3 codes stands for: bias 7, 3 mantissa bits, no infinities, NaN at 0x7F and 0xFF."""
    out = np.zeros(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = np.nan if (e, m) == (15, 7) else 2.0 ** -9 * m if e == 0 else 2.0 ** (e - 10) * (8 + m)
        out[c] = -x if c & 128 else x
    return out


def code_values(codes, kind):
    """Bytes (uint8) as the numbers they stand for, without the scale."""
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else e4m3_table()[codes]


def nearest(x, kind):
    """The value of the code nearest to each x, ties to the even code, held to -TOP .. TOP."""
    x = np.asarray(x, np.float64)
    if kind == "int8":
        return np.clip(np.rint(x), -127, 127)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)


def quantise(x, kind):
    """(x / scale before rounding, scale) of heads x [...][D]; NaN scales and zeros as the definition says."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = np.max(np.abs(x), axis=-1)
        scale = np.where(np.isfinite(x).all(-1), top / TOP[kind], np.nan)
        ratio = np.where(scale[..., None] > 0, x / scale[..., None], 0.0)
    return ratio, scale


def to_bytes(values, kind):
    """Numbers that are codes (``nearest``'s) as their bytes."""
    if kind == "int8":
        return values.astype(np.int8).view(np.uint8)
    table = e4m3_table()
    mags = table[:127]  # ascending, 0x00 .. 0x7E
    at = np.searchsorted(mags, np.abs(values))
    return (at + 128 * (np.signbit(values) & (at > 0))).astype(np.uint8)


def store_keys(x):
    """[n][h][page][D] -> [n][h][D / 16][page][16]."""
    n, h, page, D = x.shape
    return np.ascontiguousarray(x.reshape(n, h, page, D // 16, 16).transpose(0, 1, 3, 2, 4))


def store_values(x):
    """[n][h][page][D] -> [n][h][page / 16][D][16]."""
    n, h, page, D = x.shape
    return np.ascontiguousarray(x.reshape(n, h, page // 16, 16, D).transpose(0, 1, 2, 4, 3))


def load_keys(x):
    """[n][h][D / 16][page][16] -> [n][h][page][D]."""
    n, h, c, page, _ = x.shape
    return np.ascontiguousarray(x.transpose(0, 1, 3, 2, 4)).reshape(n, h, page, c * 16)


def load_values(x):
    """[n][h][page / 16][D][16] -> [n][h][page][D]."""
    n, h, o, D, _ = x.shape
    return np.ascontiguousarray(x.transpose(0, 1, 2, 4, 3)).reshape(n, h, o * 16, D)


def read(batch, cells):
    """Rows [kv_heads][D] of every token's position, from cells [n_pages][kv_heads][page][D]."""
    q_start, ctx_len, table = batch
    n_pages, kv_heads, page, D = cells.shape
    out = {}
    for n, b, p in tokens(q_start, ctx_len):
        at = int(table[b][p // page]) if p >= 0 else -1
        out[n] = cells[at, :, p % page] if 0 <= at < n_pages else np.zeros((kv_heads, D))
    return out


def attend_window(batch, keys, values, q, scale, window, n_first):
    """out[row] = [heads][D]: the token at position p sees positions p - window + 1 .. p and 0 .. n_first - 1."""
    q_start, ctx_len, table = batch
    n_pages, kv_heads, page, D = keys.shape
    out = {}
    for n, b, p in tokens(q_start, ctx_len):
        heads = q[n].shape[0]
        group = heads // kv_heads
        out[n] = np.zeros((heads, D))
        if p < 0:
            continue
        cells = np.arange(p + 1)
        cells = cells[(cells > p - window) | (cells < n_first)]
        pages = np.asarray(table[b])[cells // page]
        held = (pages >= 0) & (pages < n_pages)
        cells, pages = cells[held], pages[held]
        if len(cells) == 0:
            continue
        for h in range(kv_heads):
            s = scale * (np.asarray(q[n][h * group:(h + 1) * group], np.float64) @ keys[pages, h, cells % page].T)
            e = np.exp(s - s.max(-1, keepdims=True))
            out[n][h * group:(h + 1) * group] = e / e.sum(-1, keepdims=True) @ values[pages, h, cells % page]
    return out
