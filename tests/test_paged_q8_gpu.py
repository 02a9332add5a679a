"""The paged cache of codes on the GPU (through the C ABI) against the FP64 reference: append, read-back, attention over
every page and over listed pages, and a decode loop of them together.

Cells that no visible position owns hold NaN scales (and NaN codes in E4M3).  Tolerances: attention as over BF16 pages
(``paged_codes_util.attend``); a code is at most half a step from its quotient, and FP32's share of the quotient."""

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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


GEOMETRIES = [(64, 64, 2, 8), (128, 64, 8, 4), (128, 128, 1, 5), (256, 64, 2, 6), (256, 128, 1, 16), (128, 256, 2, 3),
              (64, 128, 3, 7), (64, 256, 1, 1)]  # head_dim, page, kv heads, group


# ---- append and read-back

def _append(kind, s, heads, dtype, rope_dim, pairs, norm, seed=0, rows=None, edit=None):
    """Appends to a scene of codes and checks every array; returns (cache, batch, q)."""
    D, KV, P, n_pages = s.means.shape[2], s.means.shape[1], s.page, s.k_codes.shape[0]
    n = s.n_tokens if rows is None else rows
    g = gen.rng(112, seed)
    qkv = (g.standard_normal((n, (heads + 2 * KV) * D)) * 3).astype(np.float32)
    if dtype == torch.bfloat16:
        qkv = oracle.bf16_bits_to_f64(pu.bf16(qkv)).astype(np.float32)
    split = [qkv[:, :heads * D].reshape(n, heads, D), qkv[:, heads * D:(heads + KV) * D].reshape(n, KV, D),
             qkv[:, (heads + KV) * D:].reshape(n, KV, D)]  # views
    if edit:
        edit(*split)
    wq, wk = (g.uniform(0.5, 1.5, (2, D)).astype(np.float32)) if norm else (None, None)
    rope = None
    if rope_dim:
        angle = np.arange(int(max(s.ctx_len.max(), 1)))[:, None] * 1e4 ** (-np.arange(rope_dim // 2) / (rope_dim / 2))
        rope = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    q_want, writes = oracle.paged.append(s.batch, P, n_pages, *split, wq, wk, 1e-6, rope, pairs)

    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    whole = torch.from_numpy(qkv).cuda().to(dtype)
    q, k, v = (whole[:, a * D:b * D].view(n, -1, D) for a, b in ((0, heads), (heads, heads + KV), (heads + KV, heads + 2 * KV)))

    def dev(a):
        return None if a is None else torch.from_numpy(a).cuda()
    q_out = torch.full((n, heads, D), 5.0, device="cuda", dtype=torch.bfloat16)
    cache.append(batch, q, k, v, q_norm=dev(wq), k_norm=dev(wk), rope=dev(rope), interleaved=pairs, q_out=q_out)
    torch.cuda.synchronize()

    got = q_out.float().double().cpu().numpy()
    for m in range(n):
        if m not in q_want:
            assert np.all(got[m] == 5.0), f"row {m} is behind the last sequence's"
            continue
        room = 2.0 ** -8 * np.abs(q_want[m]) + (D + 8) * 2.0 ** -24 * np.abs(q_want[m]).max()
        assert np.all(np.abs(got[m] - q_want[m]) <= room), f"q row {m}"

    touched = np.zeros((n_pages, P), bool)
    for pg, slot in writes:
        touched[pg, slot] = True
    after = {"k": (cu.host_codes(cache.k_pages), cache.k_scales.cpu().numpy()),
             "v": (cu.host_codes(cache.v_pages), cache.v_scales.cpu().numpy())}
    for name, load, before, at in (("k", o.load_keys, (s.k_codes, s.k_scales), 0),
                                   ("v", o.load_values, (s.v_codes, s.v_scales), 1)):
        codes, scales = load(after[name][0]), after[name][1]
        values = o.code_values(codes, kind)
        # FP32's share: of the values the norm's and rotation's D + 8 roundings (values as they are: none), of the scale
        # one division, of a quotient another
        share = ((D + 8) if name == "k" else 0) * 2.0 ** -24 + 2.0 ** -23
        for (pg, slot), both in writes.items():
            ratio, scale = o.quantise(both[at], kind)
            assert np.array_equal(np.isnan(scale), np.isnan(scales[pg, :, slot])), f"{name} scale {pg} {slot}"
            off = np.abs(scales[pg, :, slot] - scale)
            assert not np.any(off > scale * share), f"{name} scale of page {pg} slot {slot}"
            room = cu.half_step(np.abs(ratio) + o.TOP[kind] * 2 * share, kind) + o.TOP[kind] * 2 * share
            assert np.all(np.abs(values[pg, :, slot] - ratio) <= room), f"{name} codes of page {pg} slot {slot}"
        # every other cell is as it was, bit for bit
        old_codes, old_scales = load(before[0]).transpose(0, 2, 1, 3)[~touched], before[1].transpose(0, 2, 1)[~touched]
        assert np.array_equal(codes.transpose(0, 2, 1, 3)[~touched], old_codes)
        assert np.array_equal(scales.transpose(0, 2, 1)[~touched], old_scales, equal_nan=True)
    stand = o.code_values(o.load_keys(after["k"][0]), kind) * after["k"][1][..., None].astype(np.float64)
    done, means = set(oracle.paged.completed(s.batch, P, n_pages)), pu.host_bits(cache.k_means)
    for pg in range(n_pages):
        if pg not in done:
            assert np.array_equal(means[pg], s.means[pg]), f"mean of page {pg}"
            continue
        # the mean of what the stored codes stand for: a rounding of each product, P of the partial sums, half a BF16 step
        want = stand[pg].mean(axis=1)
        room = 2.0 ** -8 * np.abs(want) + (P + 1) * 2.0 ** -24 * np.abs(stand[pg]).max()
        mean = oracle.bf16_bits_to_f64(means[pg])
        assert np.array_equal(np.isnan(want), np.isnan(mean))
        assert not np.any(np.abs(mean - want) > room), f"mean of page {pg}"
    return cache, batch, q_out


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_windows(kind, head_dim, page, kv, group, dtype):
    """Windows that begin and end inside pages and groups of 16, that complete pages, and a padded sequence."""
    windows = [(1, 1), (1, page), (1, page + 1), (7, page + 3), (16, 16), (1, 0), (3, 1), (33, 2 * page), (0, 5), (17, 40)]
    s = cu.scene(kind, 50, kv, head_dim, page, windows, visible=[c - t for t, c in windows])
    _append(kind, s, kv * group, dtype, head_dim // 4, head_dim == 128, True)


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("rope_dim,norm", [(0, False), (16, True), (128, False)])
def test_append_rotations(kind, rope_dim, norm):
    s = cu.scene(kind, 51, 2, 128, 64, [(5, 70), (2, 300)], visible=[65, 298])
    _append(kind, s, 10, torch.float32, rope_dim, False, norm)
    _append(kind, s, 10, torch.float32, rope_dim, True, norm)


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page", [(128, 64), (64, 256), (256, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_prompts(kind, head_dim, page, dtype):
    """Prompts over many pages behind earlier tokens, of unlike lengths."""
    windows = [(600, 641), (130, 130), (1, 900), (257, 300)]
    s = cu.scene(kind, 52, 2, head_dim, page, windows, visible=[c - t for t, c in windows])
    _append(kind, s, 6, dtype, head_dim, False, True)


@pytest.mark.parametrize("kind", cu.KINDS)
def test_append_of_odd_heads(kind):
    """Zeros, the smallest and the largest FP32 values, values that are not finite: each head by itself."""
    def edit(q, k, v):
        for x in (k, v):
            x[0, 0] = 0
            x[1, 0, 5] = np.inf
            x[2, 1, 9] = np.nan
            x[3, 0] = 1e-45 * np.arange(64)  # steps of the smallest numbers: the scale rounds to few bits
            x[4, 1] = 3e38 * np.cos(np.arange(64))
            x[5, 0, 1:] = 0
    s = cu.scene(kind, 53, 2, 64, 64, [(64, 64), (9, 70)], visible=[0, 61])
    D = 64

    def tiny(values, scales, x):  # of head (3, 0): within half a step of the scale, which is itself a few steps
        want = x.astype(np.float64)
        scale = np.abs(want).max() / o.TOP[kind]
        return np.abs(values * scales - want).max() <= np.abs(want).max() + 2 * scale
    cache = None
    g = gen.rng(112, 7)
    qkv = (g.standard_normal((s.n_tokens, 8, D)) * 3).astype(np.float32)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    edit(q, k, v)
    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    dev = torch.from_numpy(qkv).cuda()
    cache.append(batch, dev[:, :4], dev[:, 4:6], dev[:, 6:])
    k_out, v_out = cache.read(batch, s.n_tokens, out_dtype=torch.float32)
    torch.cuda.synchronize()
    for x, scales, load, codes, rows in ((k, cache.k_scales, o.load_keys, cache.k_pages, k_out),
                                         (v, cache.v_scales, o.load_values, cache.v_pages, v_out)):
        pg = s.table[0, 0]
        scales = scales.cpu().numpy()[pg]
        values = o.code_values(load(cu.host_codes(codes)), kind)[pg]
        rows = rows.double().cpu().numpy()
        assert scales[0, 0] == 0 and np.all(values[0, 0] == 0) and np.all(rows[0, 0] == 0)
        assert np.isnan(scales[0, 1]) and np.isnan(scales[1, 2]) and np.isnan(rows[1, 0]).all() and np.isnan(rows[2, 1]).all()
        assert np.isfinite(rows[1, 1]).all() and np.isfinite(rows[2, 0]).all()  # the heads beside them
        assert tiny(values[0, 3], scales[0, 3], x[3, 0])
        for t, h in ((4, 1), (5, 0), (6, 0), (40, 1)):
            ratio, scale = o.quantise(x[t, h], kind)
            assert abs(scales[h, t] - scale) <= scale * 2.0 ** -23
            slack = o.TOP[kind] * 2.0 ** -22
            assert np.all(np.abs(values[h, t] - ratio) <= cu.half_step(np.abs(ratio) + slack, kind) + slack)
        assert values[0, 5, 0] == np.sign(x[5, 0, 0]) * o.TOP[kind]


@pytest.mark.parametrize("kind", cu.KINDS)
def test_append_with_scales_that_are_nan_spoils_the_mean_of_its_page_alone(kind):
    def edit(q, k, v):
        k[3, 1, 9] = np.nan
    s = cu.scene(kind, 54, 2, 64, 64, [(20, 64), (70, 128)], visible=[44, 58])
    _append(kind, s, 4, torch.float32, 32, False, True, edit=edit)


@pytest.mark.parametrize("kind", cu.KINDS)
def test_append_leaves_pages_outside_the_cache_and_rows_behind(kind):
    s = cu.scene(kind, 55, 1, 64, 64, [(80, 200), (2, 10)], visible=[120, 8])
    s.table[0, 2] = s.k_codes.shape[0] + 3
    s.table[1, 0] = -1
    _append(kind, s, 2, torch.float32, 32, False, True, rows=90)


@pytest.mark.parametrize("kind", cu.KINDS)
def test_codes_do_not_depend_on_how_windows_were_cut(kind):
    """A prompt at once, in pieces, and over rejected tokens: the same pages, bit for bit."""
    s = cu.scene(kind, 56, 2, 128, 64, [(150, 150)], visible=[0])
    g = torch.Generator(device="cuda").manual_seed(3)
    y = torch.randn(150, 12, 128, device="cuda", generator=g)
    other = torch.randn(150, 12, 128, device="cuda", generator=g) * 100
    w = torch.rand(128, device="cuda", generator=g) + 0.5
    angle = torch.arange(150, device="cuda")[:, None] / 7 ** torch.arange(32, device="cuda")
    rope = torch.cat([angle.cos(), angle.sin()], 1).float()

    def pages_of(pieces):
        cache = cu.dev_cache(s)
        for x, lo, hi in pieces:
            batch = paged.Batch(torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"),
                                torch.tensor([hi], dtype=torch.int32, device="cuda"),
                                torch.from_numpy(s.table).cuda(), hi - lo, 150)
            x = x[lo:hi]
            cache.append(batch, x[:, :8], x[:, 8:10], x[:, 10:], k_norm=w, rope=rope)
        return [t.view(torch.uint8) for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales, cache.k_means)]
    whole = pages_of([(y, 0, 150)])
    pieces = pages_of([(y, 0, 3), (y, 3, 64), (y, 64, 65), (y, 65, 127), (other, 127, 150), (y, 127, 130), (y, 130, 150)])
    assert all(torch.equal(a, b) for a, b in zip(whole, pieces))


@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_read(kind, head_dim, page, kv, group, out_dtype):
    """Whole sequences and their last positions, padded tokens, pages outside the cache, rows behind the last."""
    windows = [(1, 1), (page + 3, page + 3), (40, 3 * page + 5), (0, 7), (5, 2), (1, 0), (33, 2 * page), (100, 100)]
    s = cu.scene(kind, 60, kv, head_dim, page, windows)
    s.table[7, 0] = -1
    keys, values = cu.decoded(s)
    cache, n = cu.dev_cache(s), s.n_tokens + 4
    k = torch.full((n, kv, head_dim), 5.0, device="cuda", dtype=out_dtype)
    v = torch.full_like(k, 6.0)
    assert cache.read(pu.dev_batch(s), n, k_out=k, v_out=v) == (k, v)
    torch.cuda.synchronize()
    for got, cells, rest in ((k, keys, 5.0), (v, values, 6.0)):
        want = o.read(s.batch, cells)
        rows = got.float().double().cpu().numpy()
        for m, w in want.items():
            room = np.abs(w) * (2.0 ** -24 + (2.0 ** -8 if out_dtype == torch.bfloat16 else 0))
            if kind == "bf16":
                room = 0 * room
            assert np.all(np.abs(rows[m] - w) <= room), f"row {m}"
        assert np.all(rows[s.n_tokens:] == rest)


def test_read_of_one_side():
    """The C entry takes keys or values alone."""
    s = cu.scene("int8", 61, 2, 64, 64, [(70, 70)])
    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    k, v = cache.read(batch, 70)
    one = torch.zeros_like(k)
    L = paged.lib()
    for k_at, v_at, want in ((one.data_ptr(), None, k), (None, one.data_ptr(), v)):
        one.zero_()
        assert L.hcr_cache_read(cache.handle, batch._of(70), 1, k_at, v_at,
                                torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(one, want)


# ---- attention over codes

@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_attend_short_lengths(kind, head_dim, page, kv, group, out_dtype):
    """One token over lengths around a tile's and a page's ends, an empty sequence (a row of zeros) among them."""
    lens = [1, 0, 2, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, page - 1, page, page + 1, 2 * page, 2 * page + 31, 5 * page + 7]
    s = cu.scene(kind, 70, kv, head_dim, page, [(1, c) for c in lens])
    out, want, tol = cu.attend(s, kv * group, out_dtype=out_dtype)
    assert torch.all(out[1] == 0)
    pu.check_rows(out, want, tol, "short")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
def test_attend_windows(kind, head_dim, page, kv, group):
    """Windows of 1..16 tokens, causal among themselves; a window longer than its sequence has rows that see
    nothing; a sequence without new tokens."""
    s = cu.scene(kind, 71, kv, head_dim, page, [(6, 200), (16, 16), (1, 77), (0, 50), (5, 3), (3, 3), (16, page * 3 + 1)])
    out, want, tol = cu.attend(s, kv * group)
    assert torch.all(out[23:25] == 0)  # positions -2 and -1
    pu.check_rows(out, want, tol, "windows")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T", [(256, 1, 16, 16), (128, 1, 64, 3), (64, 2, 16, 40), (128, 2, 5, 13),
                                                 (256, 1, 33, 1), (128, 1, 17, 1), (256, 2, 6, 6), (256, 1, 24, 1)])
def test_attend_many_rows(kind, head_dim, kv, group, T):
    """More rows than one work-group holds, ragged tiles of 16."""
    s = cu.scene(kind, 72, kv, head_dim, 64, [(T, 300), (max(T - 2, 1), 150)])
    out, want, tol = cu.attend(s, kv * group)
    pu.check_rows(out, want, tol, "rows")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T", [(64, 1, 16, 20), (128, 2, 10, 17), (256, 1, 24, 14)])
def test_attend_ragged_prompts(kind, head_dim, kv, group, T):
    """Far fewer tokens than the bounds allow, over many sequences: smaller row blocks, most of them empty."""
    g = gen.rng(118, head_dim)
    s = cu.scene(kind, 86, kv, head_dim, 64,
                 [(int(t), int(t) + int(c)) for t, c in zip(g.integers(0, 4, 60), g.integers(0, 200, 60))] + [(T, 400), (T, T)])
    out, want, tol = cu.attend(s, kv * group, out_dtype=torch.bfloat16)
    pu.check_rows(out, want, tol, "ragged prompts")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,group", [(64, 64), (128, 40), (256, 33)])
def test_attend_whole_sets_that_fill_the_chip(kind, head_dim, group):
    """Many sets of many rows, up to 4,096 positions: a work-group each row block and set, nothing joined."""
    g = gen.rng(119, head_dim)
    windows = [(int(t), int(t) + int(c)) for t, c in zip(g.integers(0, 9, 250), g.integers(0, 70, 250))]
    windows[100], windows[249] = (8, 4096), (8, 2049)
    s = cu.scene(kind, 87, 1, head_dim, 64, windows)
    out, want, tol = cu.attend(s, group, out_dtype=torch.bfloat16)
    pu.check_rows(out, want, tol, "whole sets")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group,T", [(128, 64, 1, 4, 1), (256, 64, 2, 6, 2), (64, 128, 1, 8, 4),
                                                      (128, 256, 1, 16, 5), (256, 64, 1, 8, 8)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_attend_split_lengths(kind, head_dim, page, kv, group, T, out_dtype):
    """Long and short sequences in one call: splits that only some sequences reach, joined."""
    s = cu.scene(kind, 73, kv, head_dim, page, [(T, 20011), (1, 5), (T, 4097), (1, 8192), (1, 0)])
    out, want, tol = cu.attend(s, kv * group, out_dtype=out_dtype)
    pu.check_rows(out, want, tol, "splits")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T", [(128, 1, 4, 1), (64, 1, 2, 3), (256, 1, 6, 4)])
def test_attend_runs_over_many_short_sequences(kind, head_dim, kv, group, T):
    """More sequences than a wave has lanes, one of them long: runs that hold several sequences, begin and end
    inside one, or skip sequences without new tokens."""
    g = gen.rng(113, head_dim)
    windows = [(int(t), int(c)) for t, c in zip(g.integers(0, T + 1, 150), g.integers(0, 150, 150))]
    windows[70] = (T, 6000)
    windows[149] = (1, 33)
    s = cu.scene(kind, 74, kv, head_dim, 64, windows)
    out, want, tol = cu.attend(s, kv * group)
    pu.check_rows(out, want, tol, "runs")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,kv,group,most", [(128, 2, 2, 500), (64, 2, 1, 2000), (256, 2, 9, 300)])
def test_attend_many_sequences(kind, head_dim, kv, group, most):
    """A work-group a sequence, more of them than the chip holds at once."""
    g = gen.rng(114, head_dim)
    s = cu.scene(kind, 75, kv, head_dim, 64, [(1, int(c)) for c in g.integers(0, most, 270)] + [(2, most)])
    out, want, tol = cu.attend(s, kv * group, out_dtype=torch.bfloat16)
    pu.check_rows(out, want, tol, "many")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group", GEOMETRIES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_attend_blocks(kind, head_dim, page, kv, group, out_dtype):
    """Listed pages in any order, -1 among them, pages past the token, one listed twice, none at all."""
    s = cu.scene(kind, 76, kv, head_dim, page, [(3, 9 * page + 5), (1, 20), (2, 4 * page), (3, 2)])
    g = gen.rng(115, head_dim, page)
    sel = g.integers(-1, 12, size=(s.n_tokens, kv, 7)).astype(np.int32)
    sel[1, 0] = [0, 9, 9, -1, 3, 2 ** 30, -7]
    sel[2, :] = -1
    out, want, tol = cu.attend(s, kv * group, out_dtype=out_dtype, sel=sel)
    assert torch.all(out[2] == 0)
    pu.check_rows(out, want, tol, "blocks")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group", [(128, 64, 1, 24), (64, 128, 2, 33), (256, 64, 1, 64), (128, 64, 1, 17),
                                                    (256, 256, 1, 48)])
def test_attend_blocks_of_many_heads(kind, head_dim, page, kv, group):
    """Groups of more than 16 heads: whole lists, lists cut over work-groups, none at all."""
    s = cu.scene(kind, 85, kv, head_dim, page, [(2, 60 * page + 5), (1, 20), (3, 2)])
    g = gen.rng(117, head_dim, group)
    for n_sel in (3, 50):
        sel = g.integers(-1, 62, size=(s.n_tokens, kv, n_sel)).astype(np.int32)
        sel[0, 0, :3] = [0, 60, 60]
        sel[4, :] = -1
        out, want, tol = cu.attend(s, kv * group, sel=sel)
        assert torch.all(out[4] == 0)
        pu.check_rows(out, want, tol, f"lists of {n_sel}")


@pytest.mark.parametrize("kind", cu.KINDS)
def test_attend_blocks_long_list(kind):
    """A list that is split over work-groups and joined."""
    s = cu.scene(kind, 77, 1, 128, 64, [(2, 12000)])
    sel = np.stack([np.sort(gen.rng(116, n).permutation(187)[:150])[None] for n in range(2)]).astype(np.int32)
    sel[1, 0, 140:] = -1
    out, want, tol = cu.attend(s, 4, sel=sel)
    pu.check_rows(out, want, tol, "long list")


@pytest.mark.parametrize("kind", cu.KINDS)
def test_attend_of_a_padded_batch_with_loose_bounds(kind):
    """A few sequences far apart among many without new tokens; bounds above what they have; rows behind them."""
    windows = [(0, 0 if i % 3 else 90) for i in range(260)]
    for i, w in ((3, (1, 1500)), (70, (2, 40)), (71, (1, 900)), (190, (2, 1300)), (259, (1, 33))):
        windows[i] = w
    s = cu.scene(kind, 78, 1, 128, 64, windows, table_extra=40)
    out, want, tol = cu.attend(s, 4, extra_rows=5, max_tokens=6, max_ctx=3000)
    pu.check_rows(out, want, tol, "padded")


@pytest.mark.parametrize("kind", cu.KINDS)
def test_attend_skips_pages_outside_the_cache(kind):
    s = cu.scene(kind, 79, 2, 64, 64, [(2, 600), (1, 64), (1, 40)])
    s.table[0, 3], s.table[0, 5] = -1, s.k_codes.shape[0]
    s.table[0, 9] = 2 ** 31 - 1
    s.table[1, :] = -5  # nothing at all: zeros
    out, want, tol = cu.attend(s, 8)
    assert torch.all(out[2] == 0)
    pu.check_rows(out, want, tol, "bad pages")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.3, 1.7, 40.0])
def test_attend_scales(kind, scale):
    """A scale of zero among them: every visible position weighs the same, and no other."""
    s = cu.scene(kind, 80, 1, 64, 64, [(3, 130), (2, 1), (2, 900)])
    out, want, tol = cu.attend(s, 4, scale=scale)
    pu.check_rows(out, want, tol, f"scale {scale}")


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,kv,group,T", [(128, 2, 4, 5), (256, 1, 6, 7), (64, 1, 8, 20), (128, 1, 12, 3),
                                                 (256, 2, 10, 3)])
def test_attend_rows_do_not_depend_on_later_tokens(kind, head_dim, kv, group, T):
    """A window's last tokens have scales that are no numbers, of a key and of a value (and an E4M3 code that is none):
    the rows before them are as ever, their own are no numbers either."""
    windows = [(T, 300), (T, 64), (T, T), (T, 5003)]
    s = cu.scene(kind, 81, kv, head_dim, 64, windows)
    heads = kv * group
    q = pu.queries(81, s.n_tokens, heads, head_dim)
    keys, values = cu.decoded(s)
    qf = oracle.bf16_bits_to_f64(q)
    want = oracle.paged.attend(s.batch, keys, values, qf, 0.1)
    tol = pu.rows_tolerance(qf, cu.reach(keys), 0.1, 5003, False)
    codes = o.load_values(s.v_codes)
    for b, (_, ctx) in enumerate(windows):
        for at in (ctx - 2, ctx - 1):
            page, slot = s.table[b, at // 64], at % 64
            if kind == "e4m3" and b % 2:
                codes[page, :, slot, 3::16] = 0xFF if at % 2 else 0x7F
            elif at == ctx - 2:
                s.v_scales[page, :, slot] = [np.nan, np.inf][b // 2]
            else:
                s.k_scales[page, :, slot] = np.nan
    s.v_codes = o.store_values(codes)
    out = cu.dev_cache(s).attend(pu.dev_batch(s), pu.dev_bits(q), scale=0.1)
    early = {n: w for n, w in want.items() if n % T < T - 2}
    pu.check_rows(out, early, tol, "early")
    nan = torch.isnan(out) | torch.isinf(out)
    late = torch.arange(s.n_tokens, device="cuda") % T >= T - 2
    assert not nan[~late].any() and nan[late][..., 3::16].all()


@pytest.mark.parametrize("kind", cu.KINDS)
def test_attend_past_2_31_codes(kind):
    """Pages behind 2^31 codes of each array."""
    KV, D, P = 8, 256, 256
    n = 2 ** 31 // (KV * D * P) + 4
    cache = paged.PagedCache.allocate(n, KV, D, P, dtype=cu.DTYPE[kind])
    s = cu.scene(kind, 82, KV, D, P, [(2, 700)], spare=0, table_extra=0)
    numbers = [n - 1, n - 2, 1]
    for j, pg in enumerate(numbers):
        cache.k_pages.view(torch.uint8)[pg] = torch.from_numpy(s.k_codes[s.table[0, j]]).cuda()
        cache.v_pages.view(torch.uint8)[pg] = torch.from_numpy(s.v_codes[s.table[0, j]]).cuda()
        cache.k_scales[pg] = torch.from_numpy(s.k_scales[s.table[0, j]]).cuda()
        cache.v_scales[pg] = torch.from_numpy(s.v_scales[s.table[0, j]]).cuda()
    q = pu.queries(82, 2, 16, D)
    qf = oracle.bf16_bits_to_f64(q)
    keys, values = cu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, qf, D ** -0.5)
    batch = pu.dev_batch(s)
    batch.block_table[0, :3] = torch.tensor(numbers, dtype=torch.int32)
    out = cache.attend(batch, pu.dev_bits(q))
    k, v = cache.read(batch, 2, out_dtype=torch.float32)
    torch.cuda.synchronize()
    pu.check_rows(out, want, pu.rows_tolerance(qf, cu.reach(keys), D ** -0.5, 700, False), "far pages")
    for got, cells in ((k, keys), (v, values)):
        rows = o.read(s.batch, cells)
        assert all(np.all(np.abs(got[m].double().cpu().numpy() - rows[m]) <= 2.0 ** -24 * np.abs(rows[m])) for m in rows)


# ---- together

@pytest.mark.parametrize("kind", cu.KINDS)
def test_a_decode_loop(kind):
    """Prompts, then windows of drafts of which some are taken back, over one cache: append, attention, selection, a
    sliding window and read-back against the reference on what the pages stand for; one graph of it all replayed as the
    sequences grow, against eager calls."""
    KV, D, P, H, T = 2, 128, 64, 8, 3
    cache = paged.PagedCache.allocate(40, KV, D, P, dtype=cu.DTYPE[kind])
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(float("nan"))
    g = torch.Generator(device="cuda").manual_seed(9)
    table = torch.randperm(40, generator=g, device="cuda").to(torch.int32).view(2, 20)
    angle = torch.arange(1280, device="cuda")[:, None] / 9 ** torch.arange(D // 2, device="cuda")
    rope = torch.cat([angle.cos(), angle.sin()], 1).float()
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    i32 = dict(dtype=torch.int32, device="cuda")
    prompt = paged.Batch(torch.tensor([0, 500, 830], **i32), torch.tensor([500, 330], **i32), table, 500, 1280)
    y = torch.randn(830, H + 2 * KV, D, generator=g, device="cuda").to(torch.bfloat16)
    cache.append(prompt, y[:, :H], y[:, H:H + KV], y[:, H + KV:], q_norm=w, k_norm=w, rope=rope)

    ctx = torch.tensor([500, 330], **i32)
    step = paged.Batch(torch.tensor([0, T, 2 * T], **i32), ctx, table, T, 1280)
    x = torch.zeros(2 * T, H + 2 * KV, D, device="cuda", dtype=torch.bfloat16)

    def calls():
        q = cache.append(step, x[:, :H], x[:, H:H + KV], x[:, H + KV:], q_norm=w, k_norm=w, rope=rope)
        sel = cache.block_topk(step, cache.block_scores(step, q), 5)
        return [q, cache.attend(step, q), sel, cache.attend_blocks(step, q, sel),
                cache.attend_window(step, q, 100, n_first=4), *cache.read(step, 2 * T, out_dtype=torch.float32)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    ctx += T
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for turn in range(6):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        q, dense, sel, listed, window, k, v = [t.clone() for t in held]
        for a, b in zip(calls(), (q, dense, sel, listed, window, k, v)):
            assert torch.equal(a, b)
        batch = (np.array([0, T, 2 * T]), ctx.cpu().numpy(), table.cpu().numpy())
        keys, values = (o.code_values(load(cu.host_codes(t)), kind) * sc.cpu().numpy()[..., None].astype(np.float64)
                        for load, t, sc in ((o.load_keys, cache.k_pages, cache.k_scales),
                                            (o.load_values, cache.v_pages, cache.v_scales)))
        qf = oracle.bf16_bits_to_f64(pu.host_bits(q))
        sc = D ** -0.5
        tol = pu.rows_tolerance(qf, cu.reach(keys), sc, 1280, False)
        pu.check_rows(dense, oracle.paged.attend(batch, keys, values, qf, sc), tol, "dense")
        pu.check_rows(listed, oracle.paged.attend(batch, keys, values, qf, sc, sel=sel.cpu().numpy()), tol, "listed")
        pu.check_rows(window, o.attend_window(batch, keys, values, qf, sc, 100, 4), tol, "window")
        for got, cells in ((k, keys), (v, values)):
            rows = o.read(batch, cells)
            assert all(np.all(np.abs(got[m].double().cpu().numpy() - rows[m]) <= 2.0 ** -24 * np.abs(rows[m])) for m in rows)
        # some of the drafts are taken back: the next window overwrites them
        ctx += torch.tensor([[1, 3], [3, 2], [2, 1]][turn % 3], **i32) * (1 if turn < 5 else 0)


@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
def test_calls_are_reproducible(kind):
    s = cu.scene(kind, 83, 2, 128, 64, [(2, 5000), (1, 77), (3, 901)])
    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    q = pu.dev_bits(pu.queries(83, s.n_tokens, 8, 128))
    first = [cache.attend(batch, q), cache.attend_window(batch, q, 700, 5), *cache.read(batch, s.n_tokens)]
    for _ in range(5):
        again = [cache.attend(batch, q), cache.attend_window(batch, q, 700, 5), *cache.read(batch, s.n_tokens)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
def test_two_streams_at_once(kind):
    """Calls on two streams, each with outputs and scratch of its own, over the same pages."""
    s = cu.scene(kind, 86, 2, 128, 64, [(5, 9000), (1, 77), (3, 4000)])
    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    qs = [pu.dev_bits(pu.queries(86 + i, s.n_tokens, 16, 128)) for i in range(2)]

    def calls(q):
        return [cache.attend(batch, q), cache.attend_window(batch, q, 3000, 5), *cache.read(batch, s.n_tokens)]
    want = [calls(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(calls(qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i], r))


@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
def test_calls_on_another_stream(kind):
    """Outputs and scratch on a stream that is not torch's current one, behind that stream's earlier work."""
    s = cu.scene(kind, 84, 2, 128, 64, [(2, 9000), (1, 77)])
    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    q = pu.dev_bits(pu.queries(84, s.n_tokens, 8, 128))
    want = [cache.attend(batch, q), cache.attend_window(batch, q, 4000, 5), *cache.read(batch, s.n_tokens)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late = torch.zeros_like(q)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
    got = [cache.attend(batch, late, stream=side.cuda_stream), cache.attend_window(batch, late, 4000, 5, stream=side.cuda_stream),
           *cache.read(batch, s.n_tokens, stream=side.cuda_stream)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
