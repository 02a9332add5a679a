"""Attention over a sliding window and a few first positions, on the GPU (through the C ABI), against the FP64
reference, over BF16 pages and pages of codes."""

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from bf16_hyper_connection_amd import paged
from tests import paged_codes_util as cu
from tests import paged_util as pu
from tests.libhcr_util import ensure_built

pytestmark = pytest.mark.gpu
o = oracle.paged_codes
KINDS = ["bf16"] + cu.KINDS


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


WINDOWS = [(1, 0), (1, 1), (31, 0), (32, 4), (33, 33), (64, 0), (65, 70), (100, 200), (1000, 4), (2 ** 31 - 1, 0),
           (7, 2 ** 31 - 1)]  # positions, first ones


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,n_first", WINDOWS)
@pytest.mark.parametrize("head_dim,page,kv,group", [(64, 64, 2, 8), (128, 64, 2, 4), (256, 128, 1, 6)])
def test_single_tokens(kind, window, n_first, head_dim, page, kv, group):
    """Lengths around the ends of tiles, pages and windows; an empty sequence."""
    lens = [1, 0, 2, 31, 32, 33, 64, 65, 66, 127, 128, 129, 300, 1000, 1001, 2500]
    s = cu.scene(kind, 130, kv, head_dim, page, [(1, c) for c in lens])
    out, want, tol = cu.attend(s, kv * group, window=window, n_first=n_first)
    assert torch.all(out[1] == 0)
    pu.check_rows(out, want, tol, f"window {window} {n_first}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,n_first", [(1, 0), (3, 2), (16, 0), (40, 5), (130, 64), (5000, 1)])
@pytest.mark.parametrize("head_dim,page,kv,group", [(64, 64, 3, 7), (128, 128, 1, 5), (256, 64, 2, 6)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_windows_of_tokens(kind, window, n_first, head_dim, page, kv, group, out_dtype):
    """Several new tokens, each with a window of its own; a window longer than its sequence; no new tokens."""
    s = cu.scene(kind, 131, kv, head_dim, page, [(6, 200), (16, 16), (1, 77), (0, 50), (5, 3), (3, 3), (16, page * 3 + 1)])
    out, want, tol = cu.attend(s, kv * group, window=window, n_first=n_first, out_dtype=out_dtype)
    assert torch.all(out[23:25] == 0)  # positions -2 and -1
    pu.check_rows(out, want, tol, "windows")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T", [(128, 2, 4, 300), (64, 1, 16, 200), (256, 1, 6, 130), (128, 1, 17, 3),
                                                 (256, 1, 24, 1), (256, 1, 12, 5)])
@pytest.mark.parametrize("window,n_first", [(50, 4), (129, 0), (1, 0)])
def test_prompts(kind, head_dim, kv, group, T, window, n_first):
    """More rows than a work-group holds: each row block has tiles of its own."""
    s = cu.scene(kind, 132, kv, head_dim, 64, [(T, T + 200), (max(T // 2, 1), T), (1, 40), (T, T)])
    out, want, tol = cu.attend(s, kv * group, window=window, n_first=n_first)
    pu.check_rows(out, want, tol, "prompts")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T", [(64, 1, 16, 20), (128, 2, 10, 17), (256, 1, 24, 14)])
@pytest.mark.parametrize("window,n_first", [(50, 4), (130, 0)])
def test_ragged_prompts(kind, head_dim, kv, group, T, window, n_first):
    """Far fewer tokens than the bounds allow, over many sequences: smaller row blocks, most of them empty."""
    g = gen.rng(120, head_dim)
    s = cu.scene(kind, 143, kv, head_dim, 64,
                 [(int(t), int(t) + int(c)) for t, c in zip(g.integers(0, 4, 60), g.integers(0, 300, 60))] + [(T, 400), (T, T)])
    out, want, tol = cu.attend(s, kv * group, window=window, n_first=n_first)
    pu.check_rows(out, want, tol, "ragged prompts")


@pytest.mark.parametrize("head_dim,kv,group,T", [(128, 1, 4, 1), (64, 2, 8, 5), (256, 1, 6, 9), (128, 1, 17, 40),
                                                 (64, 1, 64, 3), (256, 1, 33, 20)])
@pytest.mark.parametrize("window,n_first", [(1, 0), (40, 5), (33, 33), (900, 70)])
def test_pages_of_32(head_dim, kv, group, T, window, n_first):
    """BF16 pages shorter than a tile of shared rows, up to many rows."""
    s = cu.scene("bf16", 140, kv, head_dim, 32, [(T, 1000), (max(T - 1, 1), T), (1, 31), (T, 2500), (0, 9)])
    out, want, tol = cu.attend(s, kv * group, window=window, n_first=n_first)
    pu.check_rows(out, want, tol, "pages of 32")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,group", [(3, 4), (9, 8)])
def test_rows_behind_the_last_and_loose_bounds(kind, T, group):
    """Bounds above what the sequences have; rows behind the last sequence's stay as they were."""
    s = cu.scene(kind, 141, 2, 128, 64, [(T, 1500), (1, 70), (T, 33)], table_extra=40)
    q = pu.queries(141, s.n_tokens + 5, 2 * group, 128)
    keys, values = cu.decoded(s)
    qf = oracle.bf16_bits_to_f64(q)
    want = o.attend_window(s.batch, keys, values, qf, 0.1, 200, 3)
    out = torch.full((s.n_tokens + 5, 2 * group, 128), 7.0, device="cuda")
    cu.dev_cache(s).attend_window(pu.dev_batch(s, max_tokens=2 * T, max_ctx=3000), pu.dev_bits(q), 200, 3, scale=0.1, out=out)
    torch.cuda.synchronize()
    pu.check_rows(out, want, pu.rows_tolerance(qf, cu.reach(keys), 0.1, 1500, False), "loose")
    assert torch.all(out[s.n_tokens:] == 7.0)


@pytest.mark.parametrize("head_dim,kv,group,T,window", [(128, 2, 4, 3, 20), (256, 1, 6, 7, 40), (64, 1, 8, 20, 10),
                                                        (128, 1, 4, 90, 33), (256, 1, 4, 4, 64)])
def test_codes_that_are_no_numbers_stay_with_the_rows_that_see_them(head_dim, kv, group, T, window):
    """E4M3 codes 0x7F and 0xFF of values at positions that only some of a window's tokens see."""
    lens = [300, 400]
    s = cu.scene("e4m3", 142, kv, head_dim, 64, [(T, c) for c in lens])
    q = pu.queries(142, s.n_tokens, kv * group, head_dim)
    keys, values = cu.decoded(s)
    qf = oracle.bf16_bits_to_f64(q)
    want = o.attend_window(s.batch, keys, values, qf, 0.1, window, 2)
    codes, spoilt = o.load_values(s.v_codes), []
    for b, c in enumerate(lens):
        spoilt.append([c - T + 1 - window, c - 1] if b == 0 else [c - T - window, c - 1])
        for i, p in enumerate(spoilt[b]):
            codes[s.table[b, p // 64], :, p % 64, 5::16] = 0x7F if i else 0xFF
    s.v_codes = o.store_values(codes)
    out = cu.dev_cache(s).attend_window(pu.dev_batch(s), pu.dev_bits(q), window, 2, scale=0.1)
    fine = {}
    for n, b, p in oracle.paged.tokens(s.q_start, s.ctx_len):
        if any(p - window < x <= p for x in spoilt[b]):
            assert torch.isnan(out[n][..., 5::16]).all(), f"row {n} sees a code that is no number"
        else:
            fine[n] = want[n]
    assert len(fine) > 0
    pu.check_rows(out, fine, pu.rows_tolerance(qf, cu.reach(keys), 0.1, 400, False), "others")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group,T", [(128, 64, 1, 4, 1), (256, 64, 2, 6, 2), (64, 128, 1, 8, 40),
                                                      (128, 256, 1, 16, 20)])
@pytest.mark.parametrize("window,n_first", [(15000, 4), (3000, 9000), (700, 0)])
def test_split_lengths(kind, head_dim, page, kv, group, T, window, n_first):
    """Windows over several work-groups, joined; first positions past the 64 pages that a wave holds."""
    s = cu.scene(kind, 133, kv, head_dim, page, [(T, 20011), (1, 5), (T, 4097), (1, 8192), (1, 0)])
    out, want, tol = cu.attend(s, kv * group, window=window, n_first=n_first)
    pu.check_rows(out, want, tol, "splits")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T", [(128, 1, 4, 1), (64, 1, 2, 3), (256, 1, 6, 4), (128, 2, 2, 70)])
def test_many_sequences(kind, head_dim, kv, group, T):
    """More sequences than a wave has lanes, some without new tokens, one long."""
    g = gen.rng(134, head_dim)
    windows = [(int(t), int(c)) for t, c in zip(g.integers(0, T + 1, 150), g.integers(0, 150, 150))]
    windows[70] = (T, 6000)
    windows[149] = (1, 33)
    s = cu.scene(kind, 134, kv, head_dim, 64, windows)
    for window, n_first in ((40, 2), (5000, 0)):
        out, want, tol = cu.attend(s, kv * group, window=window, n_first=n_first, out_dtype=torch.bfloat16)
        pu.check_rows(out, want, tol, "many")


@pytest.mark.parametrize("kind", KINDS)
def test_pages_that_no_token_sees_may_be_given_back(kind):
    """Table entries behind the window and the first positions are -1, their old pages hold NaN."""
    T, window, n_first, P = 3, 300, 70, 64
    s = cu.scene(kind, 135, 2, 128, P, [(T, 3000), (T, 500), (1, 4097)])
    whole, want, tol = cu.attend(s, 8, window=window, n_first=n_first)
    scales = s.k_scales if kind != "bf16" else None
    for b, (t, c) in enumerate([(T, 3000), (T, 500), (1, 4097)]):
        low = c - t + 1 - window
        for j in range(-(-c // P)):
            if j * P >= n_first and (j + 1) * P <= low:
                if scales is not None:
                    scales[s.table[b, j]] = np.nan
                else:
                    s.k_bits[s.table[b, j]] = pu.NAN_BITS
                s.table[b, j] = -1
    out, _, _ = cu.attend(s, 8, window=window, n_first=n_first)
    assert torch.equal(out, whole)
    pu.check_rows(out, want, tol, "given back")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T,window", [(128, 2, 4, 5, 20), (256, 1, 6, 7, 40), (64, 1, 8, 20, 10),
                                                        (128, 1, 12, 3, 100), (256, 2, 10, 3, 64), (128, 1, 4, 90, 33)])
@pytest.mark.parametrize("odd", [np.inf, -np.inf, np.nan])
def test_rows_do_not_depend_on_positions_that_others_see(kind, head_dim, kv, group, T, window, odd):
    """Keys and values that are no numbers where only a window's first tokens see them (its oldest positions), only its
    last ones (new tokens), or none: rows that do not see them are as ever, the others are no numbers."""
    lens = [300, 400]
    s = cu.scene(kind, 136, kv, head_dim, 64, [(T, c) for c in lens])
    heads = kv * group
    q = pu.queries(136, s.n_tokens, heads, head_dim)
    keys, values = cu.decoded(s)
    qf = oracle.bf16_bits_to_f64(q)
    n_first = 2
    want = o.attend_window(s.batch, keys, values, qf, 0.1, window, n_first)
    tol = pu.rows_tolerance(qf, cu.reach(keys), 0.1, 400, False)
    spoilt = []
    for b, c in enumerate(lens):
        oldest = c - T + 1 - window  # the first token alone sees it
        at = [oldest, c - 1] if b == 0 else [oldest - 1, n_first]
        at += [c] if c % 64 else []  # behind the sequence
        spoilt.append(at)
        for p in at:
            pg, slot = s.table[b, p // 64], p % 64
            if kind == "bf16":
                bits = pu.bf16([odd])[0]
                s.v_bits[pg, :, slot // 8, ::3, slot % 8] = bits
                if p != oldest:
                    s.k_bits[pg, :, :, slot, 0] = bits
            else:
                s.v_scales[pg, :, slot] = odd
                if p != oldest:
                    s.k_scales[pg, :, slot] = odd
    out = cu.dev_cache(s).attend_window(pu.dev_batch(s), pu.dev_bits(q), window, n_first, scale=0.1)
    fine = {}
    for n, b, p in oracle.paged.tokens(s.q_start, s.ctx_len):
        sees = any(x <= p and (x > p - window or x < n_first) for x in spoilt[b])
        if not sees:
            fine[n] = want[n]
        elif spoilt[b][0] <= p and spoilt[b][0] > p - window:
            assert not torch.isfinite(out[n][..., 0]).any(), f"row {n} sees a value that is no number"
    assert len(fine) > 0
    pu.check_rows(out, fine, tol, "others")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
def test_scales(kind, scale):
    s = cu.scene(kind, 137, 1, 64, 64, [(3, 130), (2, 1), (2, 900)])
    out, want, tol = cu.attend(s, 4, scale=scale, window=50, n_first=3)
    pu.check_rows(out, want, tol, f"scale {scale}")


def test_a_window_of_everything_is_attend():
    """To FP32's rounding: the products are hidden in another way."""
    s = cu.scene("bf16", 138, 2, 128, 64, [(2, 5000), (1, 77), (3, 901)])
    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    q = pu.dev_bits(pu.queries(138, s.n_tokens, 8, 128))
    a, b = cache.attend(batch, q), cache.attend_window(batch, q, 5000)
    assert torch.allclose(a, b, rtol=0, atol=2e-5 * float(a.abs().max()))


@pytest.mark.parametrize("kind", KINDS)
def test_a_graph_whose_sequences_grow(kind):
    """Lengths and pages are read when the graph runs; two graphs share a scratch on one stream."""
    KV, D, T = 2, 128, 2
    s = cu.scene(kind, 139, KV, D, 64, [(T, 9000), (T, 2000)])
    cache, batch = cu.dev_cache(s), pu.dev_batch(s, max_ctx=9000)
    q = pu.dev_bits(pu.queries(139, 2 * T, 8, D))
    need = max(cache.window_scratch_bytes(batch, 2 * T, 8, w, 4) for w in (6000, 50))
    assert need > 0
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(2 * T, 8, D, device="cuda") for _ in range(2)]
    graphs = []
    for out, w in zip(outs, (6000, 50)):
        cache.attend_window(batch, q, w, 4, out=out, scratch=scratch)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.attend_window(batch, q, w, 4, out=out, scratch=scratch)
        graphs.append(g)
    keys, values = cu.decoded(s)
    qf = oracle.bf16_bits_to_f64(pu.host_bits(q))
    tol = pu.rows_tolerance(qf, cu.reach(keys), D ** -0.5, 9000, False)
    for lens in ([100, 40], [6001, 1], [9000, 2000], [64, 0], [20000, 1999]):
        batch.ctx_len.copy_(torch.tensor(lens, dtype=torch.int32))
        for g in graphs * 2:
            g.replay()
        torch.cuda.synchronize()
        held = (s.q_start, np.minimum(lens, 9000).astype(np.int32), s.table)
        for out, w in zip(outs, (6000, 50)):
            pu.check_rows(out, o.attend_window(held, keys, values, qf, D ** -0.5, w, 4), tol, f"{lens} {w}")
            assert torch.equal(out, cache.attend_window(batch, q, w, 4))
