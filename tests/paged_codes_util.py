"""Seeded caches of codes for the paged-cache tests, as numpy arrays and on the device, beside ``paged_util``'s BF16
scenes: cells that no visible position owns hold NaN scales and, in E4M3, NaN codes."""

from dataclasses import dataclass

import numpy as np
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from bf16_hyper_connection_amd import paged
from tests import paged_util as pu

KINDS = ["int8", "e4m3"]
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16}


@dataclass
class CodeScene:
    kind: str
    page: int
    q_start: np.ndarray
    ctx_len: np.ndarray
    table: np.ndarray
    k_codes: np.ndarray   # bytes, stored order
    v_codes: np.ndarray
    k_scales: np.ndarray  # float32 [n][h][page]
    v_scales: np.ndarray
    means: np.ndarray     # BF16 bits [n][h][D]

    @property
    def batch(self):
        return self.q_start, self.ctx_len, self.table

    @property
    def n_tokens(self):
        return int(self.q_start[-1])

    def decoded(self):
        o = oracle.paged_codes
        return (o.code_values(o.load_keys(self.k_codes), self.kind) * self.k_scales[..., None].astype(np.float64),
                o.code_values(o.load_values(self.v_codes), self.kind) * self.v_scales[..., None].astype(np.float64))


def coded(s, kind, seed=0):
    """A BF16 scene's cells as codes; what its NaN cells hold may be anything."""
    o, g = oracle.paged_codes, gen.rng(111, seed)
    out = []
    for cells, store in ((oracle.paged.decode_keys(s.k_bits), o.store_keys),
                         (oracle.paged.decode_values(s.v_bits), o.store_values)):
        ratio, scale = o.quantise(cells, kind)
        scale = scale.astype(np.float32)
        codes = o.to_bytes(o.nearest(ratio, kind), kind)
        codes[np.isnan(scale)] = 0x7F if kind == "e4m3" else g.integers(0, 256, codes.shape[-1], dtype=np.uint8)
        out += [store(codes), scale]
    return CodeScene(kind, s.page, s.q_start, s.ctx_len, s.table, out[0], out[2], out[1], out[3], s.means)


def scene(kind, seed, *args, **kw):
    """``paged_util.scene`` in any kind of pages: its BF16 scene, or its cells as codes."""
    s = pu.scene(seed, *args, **kw)
    return s if kind == "bf16" else coded(s, kind, seed)


def decoded(s):
    return s.decoded() if isinstance(s, CodeScene) else pu.decoded(s)


def dev_codes(a, kind):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().view(DTYPE[kind])


def dev_cache(s, means=True):
    if not isinstance(s, CodeScene):
        return pu.dev_cache(s, means)
    return paged.PagedCache(dev_codes(s.k_codes, s.kind), dev_codes(s.v_codes, s.kind),
                            pu.dev_bits(s.means) if means else None, torch.from_numpy(s.k_scales).cuda(),
                            torch.from_numpy(s.v_scales).cuda())


def host_codes(t):
    return t.view(torch.uint8).cpu().numpy()


def half_step(x, kind):
    """Half the distance of neighbouring codes at values of magnitude x."""
    if kind == "int8":
        return 0.5
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 4)


def reach(keys):
    """The longest key."""
    return float(np.sqrt(np.nansum(keys ** 2, axis=-1)).max()) if keys.size else 0.0


def attend(s, heads, seed=0, scale=None, out_dtype=torch.float32, sel=None, window=None, n_first=0, extra_rows=0,
           **bounds):
    """(out, want, tolerance) of one call on a scene.  The tolerance is that of BF16 pages: a code is exact in BF16, its
    scale's product is one more FP32 rounding of a dot product and of a probability."""
    D, KV = s.means.shape[2], s.means.shape[1]
    q = pu.queries(seed, max(s.n_tokens, 1) + extra_rows, heads, D)
    qf = oracle.bf16_bits_to_f64(q)
    keys, values = decoded(s)
    sc = D ** -0.5 if scale is None else scale
    if window is None:
        want = oracle.paged.attend(s.batch, keys, values, qf, sc, sel=sel)
    else:
        want = oracle.paged_codes.attend_window(s.batch, keys, values, qf, sc, window, n_first)
    tol = pu.rows_tolerance(qf, reach(keys), sc, int(max(s.ctx_len.max(), 1)), out_dtype == torch.bfloat16)
    cache, batch, qd = dev_cache(s), pu.dev_batch(s, **bounds), pu.dev_bits(q)
    if window is not None:
        out = cache.attend_window(batch, qd, window, n_first, scale=scale, out_dtype=out_dtype)
    elif sel is None:
        out = cache.attend(batch, qd, scale=scale, out_dtype=out_dtype)
    else:
        out = cache.attend_blocks(batch, qd, torch.from_numpy(sel).cuda(), scale=scale, out_dtype=out_dtype)
    torch.cuda.synchronize()
    return out, want, tol
