"""Seeded caches and batches of the paged-cache tests, as numpy arrays (BF16 as uint16 bits) and on the device."""

from dataclasses import dataclass

import numpy as np
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from bf16_hyper_connection_amd import paged

NAN_BITS = 0x7FD5  # a BF16 NaN: what lies in cells that no visible position owns


def bf16(a):
    """float32 rounded to BF16 bits."""
    return gen.f32_to_bf16_bits(np.asarray(a, np.float32))


def store_keys(x):
    """[n][h][page][D] -> [n][h][D / 8][page][8]."""
    n, h, page, D = x.shape
    return np.ascontiguousarray(x.reshape(n, h, page, D // 8, 8).transpose(0, 1, 3, 2, 4))


def store_values(x):
    """[n][h][page][D] -> [n][h][page / 8][D][8]."""
    n, h, page, D = x.shape
    return np.ascontiguousarray(x.reshape(n, h, page // 8, 8, D).transpose(0, 1, 2, 4, 3))


@dataclass
class Scene:
    page: int
    q_start: np.ndarray
    ctx_len: np.ndarray
    table: np.ndarray
    k_bits: np.ndarray   # stored order
    v_bits: np.ndarray
    means: np.ndarray    # BF16 bits [n][h][D]

    @property
    def batch(self):
        return self.q_start, self.ctx_len, self.table

    @property
    def n_tokens(self):
        return int(self.q_start[-1])


def scene(seed, kv_heads, head_dim, page, windows, spare=2, table_extra=1, visible=None):
    """``windows``: (new tokens, cached positions with them) of each sequence.  Visible cells (or the first
    ``visible[b]`` of a sequence) hold N(0, 1) keys and values, all others NaN; page order is shuffled."""
    g = gen.rng(91, seed)
    B = len(windows)
    need = [-(-max(c, 0) // page) for _, c in windows]
    n_pages = max(sum(need) + spare, 1)
    width = max(max(need), 1) + table_extra
    order = g.permutation(n_pages)
    table = np.full((B, width), -1, np.int32)
    k = np.full((n_pages, kv_heads, page, head_dim), NAN_BITS, np.uint16)
    v = np.full((n_pages, kv_heads, page, head_dim), NAN_BITS, np.uint16)
    at = 0
    for b, (_, c) in enumerate(windows):
        left = c if visible is None else visible[b]
        for j in range(need[b]):
            pg = int(order[at])
            at += 1
            table[b, j] = pg
            m = min(page, max(left - j * page, 0))
            if m:
                k[pg, :, :m] = bf16(g.standard_normal((kv_heads, m, head_dim)))
                v[pg, :, :m] = bf16(g.standard_normal((kv_heads, m, head_dim)))
    starts = np.concatenate([[0], np.cumsum([t for t, _ in windows])]).astype(np.int32)
    means = bf16(g.standard_normal((n_pages, kv_heads, head_dim)) * page ** -0.5)
    return Scene(page, starts, np.array([c for _, c in windows], np.int32), table, store_keys(k), store_values(v),
                 means)


def queries(seed, n, heads, head_dim, std=2.0):
    return bf16(gen.rng(92, seed).standard_normal((n, heads, head_dim)) * std)


def dev_bits(a):
    """BF16 bits (uint16) as a bfloat16 device tensor."""
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16)


def host_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def dev_cache(s, means=True):
    return paged.PagedCache(dev_bits(s.k_bits), dev_bits(s.v_bits), dev_bits(s.means) if means else None)


def dev_batch(s, max_tokens=None, max_ctx=None):
    t = np.diff(s.q_start)
    return paged.Batch(torch.from_numpy(s.q_start).cuda(), torch.from_numpy(s.ctx_len).cuda(),
                       torch.from_numpy(s.table).cuda(), int(t.max()) if max_tokens is None else max_tokens,
                       int(max(s.ctx_len.max(), 0)) if max_ctx is None else max_ctx)


def decoded(s):
    return oracle.paged.decode_keys(s.k_bits), oracle.paged.decode_values(s.v_bits)


def rows_tolerance(q, keys_max, scale, length, bf16_out):
    """Relative 2-norm that a row of attention may be off.

    A dot product of D BF16 products summed in FP32 is off by at most about sqrt(D) roundings of half a step
    (2^-24) of its partial sums, which |q| |k| bounds; times the scale that is the relative error of a
    probability.  The running sums add up to sqrt(length) roundings, the exponentials and the joins 16 more; 8 of
    these deviations are allowed.  A BF16 output adds half a step, 2^-8, and its probabilities' 2^-16.
    """
    D = q.shape[-1]
    reach = float(np.sqrt((q.astype(np.float64) ** 2).sum(-1)).max()) * keys_max
    tol = 8 * 2.0 ** -24 * (abs(scale) * np.sqrt(D) * reach + np.sqrt(max(length, 1)) + 16)
    return tol + (2.0 ** -8 + 2.0 ** -16 if bf16_out else 0.0)


def check_rows(out, want, tol, label):
    """Every row's heads within ``tol`` of the reference's 2-norm; rows of zeros exactly."""
    got = out.float().double().cpu().numpy()
    for n, w in want.items():
        for hd in range(w.shape[0]):
            norm = float(np.linalg.norm(w[hd]))
            off = float(np.linalg.norm(got[n, hd] - w[hd]))
            assert off <= tol * norm, f"{label}: row {n} head {hd}: off by {off:.3e}, allowed {tol * norm:.3e}"


# Attention whose work-groups walk more pages than a wave has lanes (they load 64 entries of a table's row or a list at
# a time): name -> (kv heads, heads, head_dim, page, windows, entries of a list or 0)
LONG_RUNS = {
    "a sequence whole": (8, 16, 64, 32, [(1, 4000)] + [(1, 7 + 31 * (i % 9)) for i in range(63)], 0),
    "a sequence cut": (16, 16, 64, 32, [(1, 70), (1, 40000)], 0),
    "lists whole": (8, 8, 64, 32, [(4, 4190 + 3 * i) for i in range(8)], 130),
    "lists cut": (16, 16, 64, 32, [(1, 40000)], 1200),
}
