"""The paged cache on the GPU (through the C ABI) against the FP64 reference: append, attention over every page
and over listed pages, page scores, page selection, and a window's run of them together.

Cells that no visible position owns hold NaN, so a read behind a sequence shows.  Tolerances: see
``paged_util.rows_tolerance`` (attention); BF16 outputs half a step (2^-8 of the value) and FP32's share."""

import textwrap

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import hcr, paged
from bf16_hyper_connection_amd import inputs as gen
from tests import paged_util as pu
from tests.libhcr_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def _attend(s, heads, seed=0, scale=None, out_dtype=torch.float32, sel=None, extra_rows=0, **bounds):
    """(out, want, tolerance) of one call on a scene."""
    D, KV = s.means.shape[2], s.means.shape[1]
    q = pu.queries(seed, max(s.n_tokens, 1) + extra_rows, heads, D)
    qf = oracle.bf16_bits_to_f64(q)
    keys, values = pu.decoded(s)
    sc = D ** -0.5 if scale is None else scale
    want = oracle.paged.attend(s.batch, keys, values, qf, sc, sel=sel)
    reach = float(np.sqrt(np.nansum(keys ** 2, axis=-1)).max()) if keys.size else 0.0
    tol = pu.rows_tolerance(qf, reach, sc, int(max(s.ctx_len.max(), 1)), out_dtype == torch.bfloat16)
    cache, batch = pu.dev_cache(s), pu.dev_batch(s, **bounds)
    qd = pu.dev_bits(q)
    if sel is None:
        out = cache.attend(batch, qd, scale=scale, out_dtype=out_dtype)
    else:
        out = cache.attend_blocks(batch, qd, torch.from_numpy(sel).cuda(), scale=scale, out_dtype=out_dtype)
    torch.cuda.synchronize()
    return out, want, tol


GEOMETRIES = [(64, 32, 1, 1), (64, 64, 2, 8), (128, 64, 8, 4), (128, 128, 1, 5), (256, 64, 2, 6), (256, 32, 1, 16),
              (128, 256, 2, 3), (64, 128, 3, 7)]  # head_dim, page, kv heads, group


@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_attend_short_lengths(head_dim, page, kv, group, out_dtype):
    """One token over lengths around a tile's and a page's ends, an empty sequence (a row of zeros) among them."""
    lens = [1, 0, 2, 8, 31, 32, 33, page - 1, page, page + 1, 2 * page, 2 * page + 31, 5 * page + 7]
    s = pu.scene(1, kv, head_dim, page, [(1, c) for c in lens])
    out, want, tol = _attend(s, kv * group, out_dtype=out_dtype)
    assert torch.all(out[1] == 0)
    pu.check_rows(out, want, tol, "short")


@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
def test_attend_windows(head_dim, page, kv, group):
    """Windows of 1..16 tokens, causal among themselves; a window longer than its sequence has rows that see
    nothing; a sequence without new tokens."""
    s = pu.scene(2, kv, head_dim, page, [(6, 200), (16, 16), (1, 77), (0, 50), (5, 3), (3, 3), (16, page * 3 + 1)])
    out, want, tol = _attend(s, kv * group)
    assert torch.all(out[23:25] == 0)  # positions -2 and -1
    pu.check_rows(out, want, tol, "windows")


@pytest.mark.parametrize("head_dim,kv,group,T", [(256, 1, 16, 16), (128, 1, 64, 3), (64, 2, 16, 40), (128, 2, 5, 13),
                                                 (256, 1, 33, 1), (128, 1, 17, 1)])
def test_attend_many_rows(head_dim, kv, group, T):
    """More rows than one work-group holds, ragged tiles of 16."""
    s = pu.scene(3, kv, head_dim, 64, [(T, 300), (max(T - 2, 1), 150)])
    out, want, tol = _attend(s, kv * group)
    pu.check_rows(out, want, tol, "rows")


@pytest.mark.parametrize("head_dim,page,kv,group,T", [(128, 64, 1, 4, 1), (256, 64, 2, 6, 2), (64, 32, 1, 8, 4),
                                                      (128, 256, 1, 16, 5), (256, 64, 1, 8, 8)])
def test_attend_split_lengths(head_dim, page, kv, group, T):
    """Long and short sequences in one call: splits that only some sequences reach, joined."""
    s = pu.scene(4, kv, head_dim, page, [(T, 20011), (1, 5), (T, 4097), (1, 8192), (1, 0)])
    out, want, tol = _attend(s, kv * group)
    pu.check_rows(out, want, tol, "splits")


@pytest.mark.parametrize("head_dim,kv,group,T", [(128, 1, 4, 1), (64, 1, 2, 3), (256, 1, 6, 4)])
def test_attend_runs_over_many_short_sequences(head_dim, kv, group, T):
    """More sequences than a wave has lanes, one of them long: runs that hold several sequences, begin and end
    inside one, or skip sequences without new tokens."""
    g = gen.rng(99, head_dim)
    windows = [(int(t), int(c)) for t, c in zip(g.integers(0, T + 1, 150), g.integers(0, 90, 150))]
    windows[70] = (T, 6000)
    windows[149] = (1, 33)
    s = pu.scene(12, kv, head_dim, 32, windows)
    out, want, tol = _attend(s, kv * group)
    pu.check_rows(out, want, tol, "runs")


@pytest.mark.parametrize("head_dim,kv,group,most", [(128, 2, 2, 500), (64, 2, 1, 2000), (256, 2, 1, 300),
                                                    (128, 2, 9, 400)])
def test_attend_many_sequences(head_dim, kv, group, most):
    """A work-group a sequence, more of them than the chip holds at once."""
    g = gen.rng(100, head_dim)
    s = pu.scene(13, kv, head_dim, 64, [(1, int(c)) for c in g.integers(0, most, 270)] + [(2, most)])
    out, want, tol = _attend(s, kv * group, out_dtype=torch.bfloat16)
    pu.check_rows(out, want, tol, "many")


def test_lengths_and_rows_beyond_the_bounds_are_cut():
    """ctx_len above max_ctx counts as max_ctx, rows past n_tokens and past max_tokens do not exist."""
    s = pu.scene(14, 2, 128, 64, [(2, 640), (3, 200)])
    q = pu.queries(14, 4, 4, 128)
    keys, values = pu.decoded(s)
    cut = (np.array([0, 2, 4], np.int32), np.array([600, 200], np.int32), s.table)  # the second: rows 2 and 3
    want = oracle.paged.attend(cut, keys, values, oracle.bf16_bits_to_f64(q), 0.1)
    batch = pu.dev_batch(s, max_tokens=2, max_ctx=600)
    out = pu.dev_cache(s).attend(batch, pu.dev_bits(q), scale=0.1)
    pu.check_rows(out, want, pu.rows_tolerance(oracle.bf16_bits_to_f64(q), 20.0, 0.1, 640, False), "cut")
    batch.q_start.copy_(torch.tensor([-3, 2 ** 31 - 1, 1], dtype=torch.int32))  # no sequence has rows
    again = torch.full_like(out, 3.0)
    pu.dev_cache(s).attend(batch, pu.dev_bits(q), scale=0.1, out=again)
    assert torch.all(again == 3.0)


@pytest.mark.parametrize("head_dim,kv,group,T", [(128, 2, 4, 5), (256, 1, 6, 7), (64, 1, 8, 20), (128, 1, 12, 3),
                                                 (256, 2, 10, 3), (256, 1, 16, 9)])
@pytest.mark.parametrize("odd", [np.inf, -np.inf, np.nan])
def test_attend_rows_do_not_depend_on_later_tokens(head_dim, kv, group, T, odd):
    """A window's last tokens have keys and values that are no numbers: the rows before them are as ever, their own
    are no numbers either."""
    windows = [(T, 300), (T, 64), (T, T), (T, 5003)]
    s = pu.scene(15, kv, head_dim, 64, windows)
    heads = kv * group
    q = pu.queries(15, s.n_tokens, heads, head_dim)
    keys, values = pu.decoded(s)
    qf = oracle.bf16_bits_to_f64(q)
    want = oracle.paged.attend(s.batch, keys, values, qf, 0.1)
    tol = pu.rows_tolerance(qf, float(np.sqrt(np.nansum(keys ** 2, axis=-1)).max()), 0.1, 5003, False)
    bits = pu.bf16([odd])[0]
    for b, (_, ctx) in enumerate(windows):
        for at, store in ((ctx - 2, s.v_bits), (ctx - 1, s.k_bits)):
            page = s.table[b, at // 64]
            if store is s.v_bits:
                store[page, :, at % 64 // 8, ::3, at % 8] = bits
            else:
                store[page, :, :, at % 64, 0] = bits
    out = pu.dev_cache(s).attend(pu.dev_batch(s), pu.dev_bits(q), scale=0.1)
    early = {n: w for n, w in want.items() if n % T < T - 2}
    pu.check_rows(out, early, tol, "early")
    finite = torch.isfinite(out).all(-1)
    late = torch.arange(s.n_tokens, device="cuda") % T >= T - 2
    assert finite[~late].all() and not finite[late].any()


@pytest.mark.parametrize("scale", [0.1, 0.125, 0.3, -0.1, -0.7])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_a_product_of_minus_infinity_weighs_nothing(scale, out_dtype):
    s = pu.scene(16, 1, 64, 32, [(2, 70), (1, 33)])
    q = pu.queries(16, s.n_tokens, 4, 64)
    q[..., 0] = pu.bf16([2.0])[0]
    low = np.float32(-np.inf if scale > 0 else np.inf)
    for b, at in ((0, 5), (0, 66), (1, 0)):
        s.k_bits[s.table[b, at // 32], 0, 0, at % 32, 0] = pu.bf16([low])[0]
    keys, values = pu.decoded(s)
    keys = np.where(np.isinf(keys), np.sign(low) * 1e30, keys)  # far enough
    qf = oracle.bf16_bits_to_f64(q)
    want = oracle.paged.attend(s.batch, keys, values, qf, scale)
    out = pu.dev_cache(s).attend(pu.dev_batch(s), pu.dev_bits(q), scale=scale, out_dtype=out_dtype)
    pu.check_rows(out, want, pu.rows_tolerance(qf, 20.0, scale, 70, out_dtype == torch.bfloat16), "infinite")


def test_attend_of_a_padded_batch():
    """A few sequences far apart among many without new tokens, some of those with a length."""
    windows = [(0, 0 if i % 3 else 90) for i in range(260)]
    for i, w in ((3, (1, 1500)), (70, (2, 40)), (71, (1, 900)), (190, (2, 1300)), (259, (1, 33))):
        windows[i] = w
    s = pu.scene(17, 1, 128, 64, windows)
    out, want, tol = _attend(s, 4)
    pu.check_rows(out, want, tol, "padded")


def test_attend_with_loose_bounds():
    """Bounds above what the sequences have (as a captured graph keeps them), rows behind the last sequence's."""
    s = pu.scene(5, 2, 128, 64, [(2, 100), (1, 700)], table_extra=40)
    q = pu.queries(5, 9, 8, 128)
    keys, values = pu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, oracle.bf16_bits_to_f64(q), 0.1)
    out = torch.full((9, 8, 128), 7.0, device="cuda")
    cache = pu.dev_cache(s)
    cache.attend(pu.dev_batch(s, max_tokens=6, max_ctx=3000), pu.dev_bits(q), scale=0.1, out=out)
    torch.cuda.synchronize()
    pu.check_rows(out, want, pu.rows_tolerance(oracle.bf16_bits_to_f64(q), 20.0, 0.1, 700, False), "loose")
    assert torch.all(out[3:] == 7.0)


def test_attend_skips_pages_outside_the_cache():
    """Table entries below 0 or past the last page own no positions."""
    s = pu.scene(6, 2, 64, 32, [(2, 300), (1, 64), (1, 40)])
    s.table[0, 3], s.table[0, 5] = -1, s.k_bits.shape[0]
    s.table[0, 9] = 2 ** 31 - 1
    s.table[1, :] = -5  # nothing at all: zeros
    out, want, tol = _attend(s, 8)
    assert torch.all(out[2] == 0)
    pu.check_rows(out, want, tol, "bad pages")


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
def test_attend_scales(scale):
    s = pu.scene(7, 1, 64, 64, [(3, 130)])
    out, want, tol = _attend(s, 4, scale=scale)
    pu.check_rows(out, want, tol, f"scale {scale}")


def test_attend_large_scores():
    """Scores in the thousands: one probability, the others vanish; the maximum moves many times."""
    s = pu.scene(8, 1, 128, 64, [(2, 3000)])
    out, want, tol = _attend(s, 8, scale=40.0)
    pu.check_rows(out, want, tol, "large scores")


def test_attend_past_2_31_elements():
    """Pages behind 2^31 elements of each array."""
    KV, D, P = 8, 256, 256
    per = KV * D * P
    n = 2 ** 31 // per + 4
    cache = paged.PagedCache.allocate(n, KV, D, P)
    s = pu.scene(9, KV, D, P, [(2, 700)], spare=0, table_extra=0)
    numbers = [n - 1, n - 2, 1]
    for j, pg in enumerate(numbers):
        cache.k_pages[pg] = pu.dev_bits(s.k_bits[s.table[0, j]])
        cache.v_pages[pg] = pu.dev_bits(s.v_bits[s.table[0, j]])
    q = pu.queries(9, 2, 16, D)
    keys, values = pu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, oracle.bf16_bits_to_f64(q), D ** -0.5)
    batch = pu.dev_batch(s)
    batch.block_table[0, :3] = torch.tensor(numbers, dtype=torch.int32)
    out = cache.attend(batch, pu.dev_bits(q))
    torch.cuda.synchronize()
    pu.check_rows(out, want, pu.rows_tolerance(oracle.bf16_bits_to_f64(q), 22.0, D ** -0.5, 700, False), "far pages")


@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_attend_blocks(head_dim, page, kv, group, out_dtype):
    """Listed pages in any order, -1 among them, pages past the token, one listed twice, none at all."""
    s = pu.scene(10, kv, head_dim, page, [(3, 9 * page + 5), (1, 20), (2, 4 * page), (3, 2)])
    g = gen.rng(93, head_dim, page)
    sel = g.integers(-1, 12, size=(s.n_tokens, kv, 7)).astype(np.int32)
    sel[1, 0] = [0, 9, 9, -1, 3, 2 ** 30, -7]
    sel[2, :] = -1
    out, want, tol = _attend(s, kv * group, out_dtype=out_dtype, sel=sel)
    assert torch.all(out[2] == 0)
    pu.check_rows(out, want, tol, "blocks")


def test_attend_blocks_many_tokens():
    """More sequences than a wave has lanes, a list for each of their tokens; rows behind the last one's."""
    g = gen.rng(101, 1)
    windows = [(int(t), int(c)) for t, c in zip(g.integers(0, 4, 90), g.integers(1, 300, 90))]
    s = pu.scene(15, 2, 64, 32, windows)
    sel = g.integers(-1, 10, size=(s.n_tokens + 3, 2, 5)).astype(np.int32)
    out, want, tol = _attend(s, 6, sel=sel, extra_rows=3)
    pu.check_rows(out, want, tol, "tokens")


def test_attend_blocks_long_list():
    """A list that is split over work-groups and joined."""
    s = pu.scene(11, 1, 128, 64, [(2, 12000)])
    sel = np.stack([np.sort(gen.rng(94, n).permutation(187)[:150])[None] for n in range(2)]).astype(np.int32)
    sel[1, 0, 140:] = -1
    out, want, tol = _attend(s, 4, sel=sel)
    pu.check_rows(out, want, tol, "long list")


# ---- append

def _append(s, heads, dtype, rope_dim, pairs, norm, seed=0, fused=True, rows=None):
    D, KV, P, n_pages = s.means.shape[2], s.means.shape[1], s.page, s.k_bits.shape[0]
    n = s.n_tokens if rows is None else rows
    g = gen.rng(95, seed)
    qkv = (g.standard_normal((n, (heads + 2 * KV) * D)) * 3).astype(np.float32)
    if dtype == torch.bfloat16:
        qkv = oracle.bf16_bits_to_f64(pu.bf16(qkv)).astype(np.float32)
    split = [qkv[:, :heads * D].reshape(n, heads, D), qkv[:, heads * D:(heads + KV) * D].reshape(n, KV, D),
             qkv[:, (heads + KV) * D:].reshape(n, KV, D)]
    wq, wk = (g.uniform(0.5, 1.5, (2, D)).astype(np.float32)) if norm else (None, None)
    top = int(max(s.ctx_len.max(), 1))
    rope = None
    if rope_dim:
        angle = np.arange(top)[:, None] * 1e4 ** (-np.arange(rope_dim // 2) / (rope_dim / 2))
        rope = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    eps = 1e-6
    q_want, writes = oracle.paged.append(s.batch, P, n_pages, *split, wq, wk, eps, rope, pairs)

    cache, batch = pu.dev_cache(s), pu.dev_batch(s)
    whole = torch.from_numpy(qkv).cuda().to(dtype)
    if fused:
        q = whole[:, :heads * D].view(n, heads, D)
        k = whole[:, heads * D:(heads + KV) * D].view(n, KV, D)
        v = whole[:, (heads + KV) * D:].view(n, KV, D)
    else:
        q, k, v = (torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dtype) for x in split)

    def dev(a):
        return None if a is None else torch.from_numpy(a).cuda()
    q_out = torch.full((n, heads, D), 5.0, device="cuda", dtype=torch.bfloat16)
    cache.append(batch, q, k, v, q_norm=dev(wq), k_norm=dev(wk), eps=eps, rope=dev(rope), interleaved=pairs,
                 q_out=q_out)
    torch.cuda.synchronize()

    got = q_out.float().double().cpu().numpy()
    for m in range(n):
        if m not in q_want:
            assert np.all(got[m] == 5.0), f"row {m} is behind the last sequence's"
            continue
        # half a BF16 step, and FP32: D + 8 roundings of the row's largest value at most
        room = 2.0 ** -8 * np.abs(q_want[m]) + (D + 8) * 2.0 ** -24 * np.abs(q_want[m]).max()
        assert np.all(np.abs(got[m] - q_want[m]) <= room), f"q row {m}"

    k_got, v_got = pu.host_bits(cache.k_pages), pu.host_bits(cache.v_pages)
    k_new, v_new = oracle.paged.decode_keys(k_got), oracle.paged.decode_values(v_got)
    touched = np.zeros((n_pages, P), bool)
    for (pg, slot), (kw, vw) in writes.items():
        touched[pg, slot] = True
        room = 2.0 ** -8 * np.abs(kw) + (D + 8) * 2.0 ** -24 * np.abs(kw).max()
        assert np.all(np.abs(k_new[pg, :, slot] - kw) <= room), f"key of page {pg} slot {slot}"
        assert np.array_equal(v_new[pg, :, slot], oracle.bf16_bits_to_f64(pu.bf16(vw))), f"value {pg} {slot}"
    # every other cell is as it was, bit for bit
    for before, after, order in ((s.k_bits, k_got, (0, 3, 1, 2, 4)), (s.v_bits, v_got, (0, 2, 4, 1, 3))):
        x, y = before.transpose(order), after.transpose(order)
        if order[1] == 2:
            x, y = (z.reshape(n_pages, P, *z.shape[3:]) for z in (x, y))
        assert np.array_equal(x[~touched], y[~touched])
    done = set(oracle.paged.completed(s.batch, P, n_pages))
    means = pu.host_bits(cache.k_means)
    for pg in range(n_pages):
        if pg not in done:
            assert np.array_equal(means[pg], s.means[pg]), f"mean of page {pg}"
            continue
        # the mean of the stored keys: P FP32 roundings of its partial sums, half a BF16 step
        want = k_new[pg].mean(axis=1)
        room = 2.0 ** -8 * np.abs(want) + P * 2.0 ** -24 * np.abs(k_new[pg]).max()
        assert np.all(np.abs(oracle.bf16_bits_to_f64(means[pg]) - want) <= room), f"mean of page {pg}"
    return cache, batch, q_out


@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_windows(head_dim, page, kv, group, dtype, pairs):
    """Windows that begin and end inside pages and octets, that complete pages, and a padded sequence."""
    windows = [(1, 1), (1, page), (1, page + 1), (7, page + 3), (16, 16), (1, 0), (3, 1), (9, 2 * page), (0, 5)]
    s = pu.scene(20, kv, head_dim, page, windows, visible=[c - t for t, c in windows])
    _append(s, kv * group, dtype, head_dim // 4, pairs, True)


@pytest.mark.parametrize("rope_dim", [0, 16, 48, 128])
@pytest.mark.parametrize("norm", [True, False])
def test_append_rotations(rope_dim, norm):
    s = pu.scene(21, 2, 128, 64, [(5, 70), (2, 300)], visible=[65, 298])
    _append(s, 10, torch.float32, rope_dim, False, norm, fused=False)
    _append(s, 10, torch.float32, rope_dim, True, norm)


@pytest.mark.parametrize("head_dim,page", [(128, 64), (64, 256), (256, 128), (128, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_prompts(head_dim, page, dtype):
    """Prompts over many pages behind earlier tokens, of unlike lengths."""
    windows = [(600, 641), (130, 130), (1, 900), (257, 300)]
    s = pu.scene(22, 2, head_dim, page, windows, visible=[c - t for t, c in windows])
    _append(s, 6, dtype, head_dim, False, True)


def test_append_leaves_pages_outside_the_cache_and_rows_behind():
    s = pu.scene(23, 1, 64, 32, [(40, 100), (2, 10)], visible=[60, 8])
    s.table[0, 2] = s.k_bits.shape[0] + 3
    s.table[1, 0] = -1
    _append(s, 2, torch.float32, 32, False, True, rows=50)


# ---- scores and selection

@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES + [(128, 64, 1, 16), (64, 32, 2, 24), (128, 64, 1, 64)])
def test_block_scores(head_dim, page, kv, group):
    s = pu.scene(30, kv, head_dim, page, [(4, 70 * 32 + 3), (1, page), (2, page + 1), (3, 2), (1, 40 * 32)])
    s.table[0, 1] = -1
    q = pu.queries(30, s.n_tokens, kv * group, head_dim)
    means, qf = oracle.bf16_bits_to_f64(s.means), oracle.bf16_bits_to_f64(q)
    want = oracle.paged.block_scores(s.batch, means, page, qf)
    width = -(-int(s.ctx_len.max()) // page)
    scores = torch.full((s.n_tokens, kv, width), 9.0, device="cuda")
    pu.dev_cache(s).block_scores(pu.dev_batch(s), pu.dev_bits(q), scores=scores)
    got = scores.double().cpu().numpy()
    # FP32 sums of head_dim exact products: head_dim half steps of the sum of magnitudes
    room = head_dim * 2.0 ** -24 * float(np.abs(qf).sum(-1).max() * np.abs(means).max())
    for n, w in want.items():
        m = w.shape[1]
        assert np.array_equal(np.isinf(w), np.isinf(got[n, :, :m]))
        fine = np.isfinite(w)
        assert np.all(np.abs(got[n, :, :m][fine] - w[fine]) <= room), f"row {n}"
        assert np.all(got[n, :, m:] == 9.0), f"row {n}: entries from the token's own page on"


def _scores_of(kind, n, kv, pages):
    g = gen.rng(96, pages)
    if kind == "normal":
        return g.standard_normal((n, kv, pages)).astype(np.float32)
    if kind == "level":
        return np.full((n, kv, pages), 0.25, np.float32)
    if kind == "few":
        return g.integers(-2, 3, size=(n, kv, pages)).astype(np.float32) * np.float32(0.5)
    x = g.standard_normal((n, kv, pages)).astype(np.float32)  # odd values
    for value in (np.nan, np.inf, -np.inf, -0.0, 0.0, 1e-45, -1e-45, np.finfo(np.float32).min):
        x[g.random(x.shape) < 0.1] = value
    return x


def test_block_topk_of_ragged_windows():
    """Rows of more sequences than a wave has lanes, windows of 0 to 5 tokens."""
    g = gen.rng(102, 1)
    page, kv = 32, 3
    tokens = g.integers(0, 6, 100)
    starts = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    lens = (tokens + g.integers(0, 2500, 100)).astype(np.int32)
    table = np.zeros((100, 80), np.int32)
    n = int(starts[-1])
    scores = g.standard_normal((n + 2, kv, 80)).astype(np.float32)
    want = oracle.paged.block_topk((starts, lens, table), page, scores, 9, 2, 1)
    cache = paged.PagedCache.allocate(1, kv, 64, page)
    batch = paged.Batch(torch.from_numpy(starts).cuda(), torch.from_numpy(lens).cuda(),
                        torch.from_numpy(table).cuda(), 5, 2560)
    sel = torch.full((n + 2, kv, 9), 77, dtype=torch.int32, device="cuda")
    cache.block_topk(batch, torch.from_numpy(scores).cuda(), 9, n_first=2, n_last=1, sel=sel)
    got = sel.cpu().numpy()
    assert all(np.array_equal(got[r], w) for r, w in want.items()) and np.all(got[n:] == 77)


@pytest.mark.parametrize("n_seqs", [63, 64, 65, 128, 4096, 4097, 9000])
def test_rows_of_many_sequences(n_seqs):
    """Every row finds its sequence, runs of sequences without new tokens among them; rows behind the last."""
    g = gen.rng(103, n_seqs)
    page, kv = 32, 1
    tokens = g.integers(0, 3, n_seqs) * (g.random(n_seqs // 50 + 1).repeat(50)[:n_seqs] < 0.6)
    tokens[-1] = 1
    starts = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    lens = (tokens + g.integers(0, 500, n_seqs)).astype(np.int32)
    n = int(starts[-1])
    scores = g.standard_normal((n + 2, kv, 16)).astype(np.float32)
    table = np.zeros((n_seqs, 16), np.int32)
    want = oracle.paged.block_topk((starts, lens, table), page, scores, 4, 1, 1)
    cache = paged.PagedCache.allocate(1, kv, 64, page)
    batch = paged.Batch(torch.from_numpy(starts).cuda(), torch.from_numpy(lens).cuda(),
                        torch.from_numpy(table).cuda(), 2, 512)
    sel = torch.full((n + 2, kv, 4), 77, dtype=torch.int32, device="cuda")
    cache.block_topk(batch, torch.from_numpy(scores).cuda(), 4, n_first=1, n_last=1, sel=sel)
    got = sel.cpu().numpy()
    assert len(want) == n and all(np.array_equal(got[r], w) for r, w in want.items()) and np.all(got[n:] == 77)


@pytest.mark.parametrize("kind", ["normal", "level", "few", "odd"])
@pytest.mark.parametrize("ctx", [1, 33, 700, 20000, 300000])
@pytest.mark.parametrize("n_sel,n_first,n_last", [(16, 1, 2), (3, 1, 2), (1, 0, 1), (100, 0, 3)])
def test_block_topk(kind, ctx, n_sel, n_first, n_last):
    page, kv = 32, 2
    windows = [(2, ctx), (1, max(ctx // 3, 1)), (1, 0)]
    starts = np.array([0, 2, 3, 4], np.int32)
    lens = np.array([c for _, c in windows], np.int32)
    width = -(-ctx // page) + 1
    table = np.zeros((3, width), np.int32)
    scores = _scores_of(kind, 5, kv, width)
    want = oracle.paged.block_topk((starts, lens, table), page, scores, n_sel, n_first, n_last)
    cache = paged.PagedCache.allocate(1, kv, 64, page)
    batch = paged.Batch(torch.from_numpy(starts).cuda(), torch.from_numpy(lens).cuda(),
                        torch.from_numpy(table).cuda(), 2, ctx)
    sel = torch.full((5, kv, n_sel), 77, dtype=torch.int32, device="cuda")
    cache.block_topk(batch, torch.from_numpy(scores).cuda(), n_sel, n_first=n_first, n_last=n_last, sel=sel)
    got = sel.cpu().numpy()
    for n, w in want.items():
        assert np.array_equal(got[n], w), f"row {n}"
    assert np.all(got[4] == 77)


# ---- together, as a decode window uses them

def _window_state(seed, kv, group, D, page, windows):
    s = pu.scene(seed, kv, D, page, windows, visible=[c - t for t, c in windows])
    g = gen.rng(97, seed)
    hidden = 512
    rows = (kv * group + 2 * kv) * D
    w = gen.matvec_weights(seed, rows=rows, cols=hidden)
    x = g.standard_normal((s.n_tokens, hidden)).astype(np.float32)
    top = int(s.ctx_len.max())
    angle = np.arange(top)[:, None] * 1e4 ** (-np.arange(D // 4) / (D / 4))
    rope = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    return s, w, x, rope, g.uniform(0.5, 1.5, (2, D)).astype(np.float32)


def test_a_window_through_projection_append_selection_and_attention():
    """The matvec's output appended, scored, selected and attended; each step against the reference on what the
    GPU's step before gave, and a selection of every page equal to attention over all of them."""
    kv, group, D, page = 2, 4, 128, 64
    s, w, x, rope, norms = _window_state(40, kv, group, D, page, [(3, 1500), (1, 130)])
    for b in range(2):  # means of the pages that were complete before
        for j in range(int(s.ctx_len[b]) // page):
            pg = s.table[b, j]
            s.means[pg] = pu.bf16(np.nan_to_num(pu.decoded(s)[0][pg].mean(axis=1)))
    heads = kv * group
    y = hcr.matvec_bf16(torch.from_numpy(w.view(np.int16)).cuda(), torch.from_numpy(x).cuda())
    q, k, v = (t.view(s.n_tokens, -1, D) for t in y.split([heads * D, kv * D, kv * D], dim=1))
    cache, batch = pu.dev_cache(s), pu.dev_batch(s)
    qn = cache.append(batch, q, k, v, q_norm=torch.from_numpy(norms[0]).cuda(),
                      k_norm=torch.from_numpy(norms[1]).cuda(), rope=torch.from_numpy(rope).cuda())
    scores = cache.block_scores(batch, qn)
    sel = cache.block_topk(batch, scores, 6, n_first=1, n_last=2)
    out = cache.attend_blocks(batch, qn, sel)
    dense = cache.attend(batch, qn)
    every = cache.attend_blocks(batch, qn, cache.block_topk(batch, scores, 24))
    torch.cuda.synchronize()

    yq = y.double().cpu().numpy().reshape(s.n_tokens, -1, D)
    q_want, writes = oracle.paged.append(s.batch, page, s.k_bits.shape[0], yq[:, :heads], yq[:, heads:heads + kv],
                                         yq[:, heads + kv:], norms[0], norms[1], 1e-6, rope, False)
    qg = qn.float().double().cpu().numpy()
    for n, want in q_want.items():
        assert np.all(np.abs(qg[n] - want) <= 2.0 ** -8 * np.abs(want) + (D + 8) * 2.0 ** -24 * np.abs(want).max())
    keys = oracle.paged.decode_keys(pu.host_bits(cache.k_pages))
    values = oracle.paged.decode_values(pu.host_bits(cache.v_pages))
    for (pg, slot), (kw, _) in writes.items():
        assert np.all(np.abs(keys[pg, :, slot] - kw) <= 2.0 ** -8 * np.abs(kw) + (D + 8) * 2.0 ** -24 * np.abs(kw).max())
    means = oracle.bf16_bits_to_f64(pu.host_bits(cache.k_means))
    sg = scores.double().cpu().numpy()
    room = D * 2.0 ** -24 * float(np.abs(qg).sum(-1).max() * np.abs(means).max())
    for n, want in oracle.paged.block_scores(s.batch, means, page, qg).items():
        assert np.all(np.abs(sg[n, :, :want.shape[1]] - want) <= room)
    picked = sel.cpu().numpy()
    for n, want in oracle.paged.block_topk(s.batch, page, scores.cpu().numpy(), 6, 1, 2).items():
        assert np.array_equal(picked[n], want)
    reach = float(np.sqrt(np.nansum(keys ** 2, axis=-1)).max())
    tol = pu.rows_tolerance(qg, reach, D ** -0.5, 1500, False)
    pu.check_rows(out, oracle.paged.attend(s.batch, keys, values, qg, D ** -0.5, sel=picked), tol, "selected")
    all_pages = oracle.paged.attend(s.batch, keys, values, qg, D ** -0.5)
    pu.check_rows(dense, all_pages, tol, "every page")
    pu.check_rows(every, all_pages, tol, "every page listed")


def _decode_step(cache, batch, y, heads, norms, rope):
    kv, D = cache.kv_heads, cache.head_dim
    q, k, v = (t.view(y.shape[0], -1, D) for t in y.split([heads * D, kv * D, kv * D], dim=1))
    qn = cache.append(batch, q, k, v, q_norm=norms[0], k_norm=norms[1], rope=rope)
    scores = torch.zeros(y.shape[0], kv, -(-batch.max_ctx // cache.page), device="cuda")
    cache.block_scores(batch, qn, scores=scores)
    sel = cache.block_topk(batch, scores, 5)
    return cache.attend_blocks(batch, qn, sel), cache.attend(batch, qn, out_dtype=torch.bfloat16), qn, sel


@pytest.mark.parametrize("other_stream", [False, True])
def test_captured_window_follows_its_lengths(other_stream):
    """One captured window replayed while the sequences grow: every replay equals the eager calls bit for bit.
    The padded third sequence joins in later; two graphs over one cache run in turn."""
    kv, group, D, page, most = 2, 4, 128, 32, 6000
    heads = kv * group
    s = pu.scene(41, kv, D, page, [(1, 5100), (1, 95), (1, 64)], visible=[5099, 94, 63], spare=40, table_extra=30)
    free = [p for p in range(s.k_bits.shape[0]) if p not in set(s.table[s.table >= 0].tolist())]
    for b in range(3):  # pages to grow into
        at = int((s.table[b] >= 0).sum())
        for j in range(3):
            s.table[b, at + j] = free.pop()
    g = gen.rng(98, 1)
    norms = [torch.from_numpy(g.uniform(0.5, 1.5, D).astype(np.float32)).cuda() for _ in range(2)]
    angle = np.arange(most)[:, None] * 1e4 ** (-np.arange(D // 2) / (D / 2))
    rope = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    graph_cache, eager_cache = pu.dev_cache(s), pu.dev_cache(s)
    graph_cache.k_means.zero_(), eager_cache.k_means.zero_()
    table = torch.from_numpy(s.table).cuda()
    ctx = torch.tensor([5100, 95, 0], dtype=torch.int32, device="cuda")
    starts = torch.from_numpy(s.q_start).cuda()
    batch = paged.Batch(starts, ctx, table, 1, min(most, s.table.shape[1] * page))
    y = torch.zeros(3, (heads + 2 * kv) * D, device="cuda")
    stream = torch.cuda.Stream() if other_stream else torch.cuda.current_stream()
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for _ in range(2):
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            outs.append(_decode_step(graph_cache, batch, y, heads, norms, rope))
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(graph)
    for step in range(8):
        y.copy_(torch.from_numpy(g.standard_normal(tuple(y.shape)).astype(np.float32)))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graphs[step % 2].replay()
        torch.cuda.synchronize()
        want = _decode_step(eager_cache, batch, y, heads, norms, rope)
        torch.cuda.synchronize()
        for got, w in zip(outs[step % 2], want):
            assert torch.equal(got, w), f"step {step}"
            assert torch.isfinite(got.float()).all()
        for a, b in ((graph_cache.k_pages, eager_cache.k_pages), (graph_cache.v_pages, eager_cache.v_pages),
                     (graph_cache.k_means, eager_cache.k_means)):
            assert np.array_equal(pu.host_bits(a), pu.host_bits(b)), f"step {step}"
        ctx[:2] += 1
        ctx[2] = 62 + step if step >= 2 else 0
        torch.cuda.synchronize()


def test_calls_are_bitwise_reproducible():
    s = pu.scene(42, 2, 128, 64, [(4, 9000), (2, 333)])
    cache, batch = pu.dev_cache(s), pu.dev_batch(s)
    q = pu.dev_bits(pu.queries(42, s.n_tokens, 12, 128))
    first = cache.attend(batch, q)
    for _ in range(5):
        assert torch.equal(first, cache.attend(batch, q))


def test_two_streams_with_their_own_scratch():
    """Two attention calls at once on two streams, each with scratch and outputs of its own."""
    s = pu.scene(43, 2, 256, 64, [(2, 15000)])
    cache, batch = pu.dev_cache(s), pu.dev_batch(s)
    qs = [pu.dev_bits(pu.queries(44 + i, 2, 12, 256)) for i in range(2)]
    want = [cache.attend(batch, q) for q in qs]
    need = cache.scratch_bytes(batch, 2, 12)
    assert need > 0
    scratch = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(2, 12, 256, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, q, o, sc in zip(streams, qs, outs, scratch):
            cache.attend(batch, q, out=o, scratch=sc, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_append_of_one_token_takes_any_stride():
    """A single row's token stride is never used (torch leaves it as it comes), nor a single head's."""
    s = pu.scene(45, 1, 64, 32, [(1, 20)], visible=[19])
    y = torch.randn(6 * 64 + 3, device="cuda")
    odd = [y.as_strided((1, n, 64), (387, 64 if n > 1 else 5, 1), at * 64) for n, at in ((4, 0), (1, 4), (1, 5))]
    even = [y[at * 64:(at + n) * 64].clone().view(1, n, 64) for n, at in ((4, 0), (1, 4), (1, 5))]
    assert odd[0].stride(0) == 387 and odd[1].stride(1) == 5
    caches = [pu.dev_cache(s) for _ in range(2)]
    got = [c.append(pu.dev_batch(s), *p) for c, p in zip(caches, (odd, even))]
    assert torch.equal(got[0], got[1])
    for a, b in ((caches[0].k_pages, caches[1].k_pages), (caches[0].v_pages, caches[1].v_pages)):
        assert np.array_equal(pu.host_bits(a), pu.host_bits(b))


def test_a_batch_keeps_its_tensors_and_bounds():
    s = pu.scene(46, 1, 64, 32, [(1, 20)])
    batch = pu.dev_batch(s)
    for name, value in (("max_ctx", 30), ("max_tokens", 2), ("ctx_len", batch.ctx_len.clone()), ("n_seqs", 0)):
        with pytest.raises(AttributeError):
            setattr(batch, name, value)


def test_the_decode_step_of_the_documentation():
    """The binding's example as it stands, over a few sequences."""
    code = textwrap.dedent(paged.__doc__.split("::\n\n")[1])
    starts = torch.tensor([0, 1, 4, 8], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([1, 300, 32768], dtype=torch.int32, device="cuda")
    table = torch.arange(3 * 512, dtype=torch.int32, device="cuda").view(3, 512)
    angles = torch.randn(32768, 64, device="cuda")
    names = dict(q_start=starts, ctx_len=lengths, block_table=table, y=torch.randn(8, 48, 128, device="cuda"),
                 wq=torch.ones(128, device="cuda"), wk=torch.ones(128, device="cuda"), angles=angles)
    allocate = paged.PagedCache.allocate

    def zeroed(**kw):
        cache = allocate(**kw)
        for t in (cache.k_pages, cache.v_pages, cache.k_means):
            t.zero_()
        return cache
    paged.PagedCache.allocate = zeroed
    try:
        exec(code, names)
    finally:
        paged.PagedCache.allocate = allocate
    out = names["out"]
    assert out.shape == (8, 32, 128) and torch.isfinite(out).all()
    # the first token's only position: its value times p and 1 / p, p near 1.  Three roundings of the parts' sums, two
    # of the reciprocal and one of the product, half a step (2^-24) each
    value = names["y"][0, 40:].bfloat16().float().repeat_interleave(4, 0)
    assert torch.all((out[0] - value).abs() <= 6 * 2.0 ** -24 * value.abs())


@pytest.mark.parametrize("max_ctx,columns", [(0, 0), (0, 3), (90, 3)])
def test_a_batch_of_empty_sequences(max_ctx, columns):
    """Padded sequences alone, lengths of zero and below, a table without columns: zeros, -1 and untouched pages."""
    kv, D, page, n = 2, 128, 32, 5
    cache = paged.PagedCache.allocate(4, kv, D, page)
    before = [t.view(torch.int16).clone() for t in (cache.k_pages, cache.v_pages, cache.k_means)]
    batch = paged.Batch(torch.tensor([0, 1, 3, 5], dtype=torch.int32, device="cuda"),
                        torch.tensor([0, -7, 0], dtype=torch.int32, device="cuda"),
                        torch.zeros(3, columns, dtype=torch.int32, device="cuda"), 2, max_ctx)
    y = torch.randn(n, 8 + 2 * kv, D, device="cuda")
    rope = torch.randn(max(max_ctx, 1), 64, device="cuda")
    q = cache.append(batch, y[:, :8], y[:, 8:8 + kv], y[:, 8 + kv:], rope=rope)
    assert torch.all(q == 0)
    q = y[:, :8].bfloat16()
    assert torch.all(cache.attend(batch, q) == 0)
    sel = torch.zeros(n, kv, 3, dtype=torch.int32, device="cuda")
    assert torch.all(cache.attend_blocks(batch, q, sel, out_dtype=torch.bfloat16) == 0)
    scores = cache.block_scores(batch, q)
    assert torch.all(scores == -torch.inf)
    assert torch.all(cache.block_topk(batch, scores, 3) == -1)
    for t, b in zip((cache.k_pages, cache.v_pages, cache.k_means), before):
        assert torch.equal(t.view(torch.int16), b)


def test_the_binding_refuses():
    """Shapes, types, strides and devices that do not fit, before any pointer is taken; the library's own codes."""
    s = pu.scene(47, 2, 64, 32, [(2, 3000), (1, 20)])
    cache, batch = pu.dev_cache(s), pu.dev_batch(s)
    q = pu.dev_bits(pu.queries(47, 3, 4, 64))
    f = torch.zeros(3, 8, 64, device="cuda")
    sel = torch.zeros(3, 2, 4, dtype=torch.int32, device="cuda")
    scores = torch.zeros(3, 2, 94, device="cuda")
    refused = [
        lambda: cache.attend(batch, q.float()),
        lambda: cache.attend(batch, q.half()),
        lambda: cache.attend(batch, q[..., :32]),
        lambda: cache.attend(batch, q.transpose(0, 1)),
        lambda: cache.attend(batch, q.cpu()),
        lambda: cache.attend(batch, q, out=torch.zeros(3, 4, 64, device="cuda", dtype=torch.float16)),
        lambda: cache.attend(batch, q, out=torch.zeros(2, 4, 64, device="cuda")),
        lambda: cache.attend(batch, q, out_dtype=torch.float64),
        lambda: cache.attend(batch, q, scratch=torch.zeros(8)),
        lambda: cache.attend_blocks(batch, q, sel.long()),
        lambda: cache.attend_blocks(batch, q, sel[:2]),
        lambda: cache.attend_blocks(batch, q, sel[:, :1]),
        lambda: cache.append(batch, f[:, :4].half(), f[:, 4:6].half(), f[:, 6:].half()),
        lambda: cache.append(batch, f[:, :4], f[:, 4:6].bfloat16(), f[:, 6:]),
        lambda: cache.append(batch, f[:, :4], f[:, 4:7], f[:, 6:]),
        lambda: cache.append(batch, f[:, :4], f[:, 4:6], f.permute(0, 2, 1)[:, :2]),
        lambda: cache.append(batch, f[:, :4], f[:, 4:6], f[:, 6:], q_norm=torch.ones(32, device="cuda")),
        lambda: cache.append(batch, f[:, :4], f[:, 4:6], f[:, 6:], rope=torch.ones(64, device="cuda")),
        lambda: cache.block_scores(batch, q, scores=scores.double()),
        lambda: cache.block_topk(batch, scores[:, :1], 4),
        lambda: cache.block_topk(batch, scores, 4, sel=sel[:, :, :2]),
    ]
    for call in refused:
        with pytest.raises(ValueError):
            call()
    coded = [
        (lambda: cache.attend(batch, q, scratch=torch.zeros(16, dtype=torch.uint8, device="cuda")), hcr.HCR_ESCRATCH),
        (lambda: cache.attend(batch, q, scale=float("nan")), hcr.HCR_EINVAL),
        (lambda: cache.attend(batch, q, out=q), hcr.HCR_EALIAS),
        (lambda: cache.attend(batch, pu.dev_bits(pu.queries(47, 3, 5, 64))), hcr.HCR_EINVAL),
        (lambda: cache.attend_blocks(batch, q, sel[:, :, :0].contiguous()), hcr.HCR_EINVAL),
        (lambda: cache.append(batch, f[:, :4], f[:, 4:6], f[:, 6:], rope=torch.ones(600, 32, device="cuda")),
         hcr.HCR_EINVAL),
        (lambda: cache.append(batch, f[:, :4], f[:, 4:6], f[:, 6:], eps=-1.0), hcr.HCR_EINVAL),
        (lambda: cache.block_scores(batch, q, scores=scores[:, :, :20].contiguous()), hcr.HCR_EINVAL),
        (lambda: cache.block_topk(batch, scores, 2), hcr.HCR_EINVAL),
        (lambda: cache.block_topk(batch, scores, 0), hcr.HCR_EINVAL),
        (lambda: pu.dev_cache(s, means=False).block_scores(batch, q), hcr.HCR_EINVAL),
    ]
    for call, code in coded:
        with pytest.raises(hcr.HCRError) as e:
            call()
        assert e.value.rc == code


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pairs", [0, 1])
def test_append_reads_no_row_of_a_table_without_rows(dtype, pairs):
    """Bounds of zero positions allow a table of none: padded tokens alone, zeros (through C; the address is not read)."""
    kv, D, page, n = 2, 128, 32, 40
    cache = paged.PagedCache.allocate(4, kv, D, page)
    batch = paged.Batch(torch.tensor([0, 1, 39, 40], dtype=torch.int32, device="cuda"),
                        torch.zeros(3, dtype=torch.int32, device="cuda"),
                        torch.zeros(3, 0, dtype=torch.int32, device="cuda"), n, 0)
    y = torch.randn(n, 8 + 2 * kv, D, device="cuda").to(dtype)
    table = torch.full((1, D), float("nan"), device="cuda")
    q_out = torch.full((n, 8, D), 5.0, dtype=torch.bfloat16, device="cuda")
    rows = [paged.hcr_rows(y[:, h:].data_ptr(), y.stride(0), D) for h in (0, 8, 8 + kv)]
    rc = paged.lib().hcr_cache_append(cache.handle, batch._of(n), 8, paged._TYPES[dtype], *rows, None, None, 1e-6,
                                      table.data_ptr(), 0, D, pairs, q_out.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == hcr.HCR_OK and torch.all(q_out == 0)
