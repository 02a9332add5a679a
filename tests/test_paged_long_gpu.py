"""The paged cache on the GPU at sizes that take its kernels' longer ways: runs over more pages than a wave holds
entries of, page scores two tiles of pages a wave, prompts of hundreds of tokens."""

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from bf16_hyper_connection_amd import paged
from tests import paged_util as pu
from tests.libhcr_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def _attend(s, heads, seed, sel=None, std=2.0):
    D = s.means.shape[2]
    q = pu.queries(seed, s.n_tokens, heads, D, std)
    qf = oracle.bf16_bits_to_f64(q)
    keys, values = pu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, qf, D ** -0.5, sel=sel)
    reach = float(np.sqrt(np.nansum(keys ** 2, axis=-1)).max())
    tol = pu.rows_tolerance(qf, reach, D ** -0.5, int(s.ctx_len.max()), False)
    cache, batch = pu.dev_cache(s), pu.dev_batch(s)
    out = cache.attend(batch, pu.dev_bits(q)) if sel is None else \
        cache.attend_blocks(batch, pu.dev_bits(q), torch.from_numpy(sel).cuda())
    pu.check_rows(out, want, tol, "long")


@pytest.mark.parametrize("name", sorted(pu.LONG_RUNS))
def test_runs_over_more_pages_than_a_wave_has_lanes(name):
    kv, heads, D, page, windows, n_sel = pu.LONG_RUNS[name]
    s = pu.scene(70, kv, D, page, windows)
    sel = None
    if n_sel:
        g = gen.rng(104, n_sel)
        sel = np.full((s.n_tokens, kv, n_sel), -1, np.int32)
        for n, b, p in oracle.paged.tokens(s.q_start, s.ctx_len):
            for h in range(kv):  # pages in any order, some twice, none here and there before and behind the 64th entry
                sel[n, h] = g.permutation(p // page + 1)[:n_sel]
                sel[n, h, g.integers(0, n_sel, n_sel // 12)] = -1
                sel[n, h, [3, 63, 64]] = [p // page, -1, sel[n, h, 0]]
    # moderate scores, so that every page counts
    _attend(s, heads, 70, sel, std=0.5)


@pytest.mark.parametrize("head_dim,group", [(64, 5), (64, 24), (128, 5), (128, 24), (256, 5), (256, 24), (128, 1)])
def test_block_scores_of_many_pages(head_dim, group):
    """Two 16-page tiles a wave (from 2^15 pages of all sequences and kv heads): windows of 1 to 5 tokens whose pages end
    anywhere in a wave's 32 and a work-group's 128, entries that are no pages in either tile."""
    kv, page, n_pages = 8, 32, 300
    g = gen.rng(105, head_dim, group)
    ends = [0, 1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 96, 97, 111, 113, 127, 128, 129, 139, 140]
    ends += [int(x) for x in g.integers(1, 141, 32 - len(ends))]
    tokens = g.integers(1, 6, 32)
    lens = np.array([max(32 * e + int(g.integers(1, 33)), t) for e, t in zip(ends, tokens)], np.int32)
    starts = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    width = -(-int(lens.max()) // page)
    table = g.integers(0, n_pages, (32, width)).astype(np.int32)
    table[g.random(table.shape) < 0.06] = -1
    table[g.random(table.shape) < 0.03] = n_pages
    pages = (int(lens.max()) - 1) // page
    assert pages * 32 * kv >= 2 * 1024 * 16
    means = pu.bf16(g.standard_normal((n_pages, kv, head_dim)) * 0.2)
    n = int(starts[-1])
    q = pu.queries(71, n, kv * group, head_dim)
    cache = paged.PagedCache.allocate(n_pages, kv, head_dim, page)
    cache.k_means.copy_(pu.dev_bits(means))
    batch = paged.Batch(*(torch.from_numpy(a).cuda() for a in (starts, lens, table)), int(tokens.max()), int(lens.max()))
    scores = torch.full((n + 1, kv, width + 2), 9.0, device="cuda")
    q_dev = torch.cat([pu.dev_bits(q), pu.dev_bits(q[:1])])  # a row behind the last sequence's
    cache.block_scores(batch, q_dev, scores=scores)
    mf, qf = oracle.bf16_bits_to_f64(means), oracle.bf16_bits_to_f64(q)
    want = oracle.paged.block_scores((starts, lens, table), mf, page, qf)
    got = scores.double().cpu().numpy()
    room = head_dim * 2.0 ** -24 * float(np.abs(qf).sum(-1).max() * np.abs(mf).max())
    for r, w in want.items():
        m = w.shape[1]
        assert np.array_equal(np.isinf(w), np.isinf(got[r, :, :m])), f"row {r}"
        fine = np.isfinite(w)
        assert np.all(np.abs(got[r, :, :m][fine] - w[fine]) <= room), f"row {r}"
        assert np.all(got[r, :, m:] == 9.0), f"row {r}: entries from the token's own page on"
    assert np.all(got[n] == 9.0)


@pytest.mark.parametrize("head_dim,kv,group,windows", [
    (128, 1, 4, [(700, 1033)]), (256, 1, 3, [(260, 260), (1, 77), (130, 900)]), (64, 2, 5, [(515, 600), (33, 33)]),
    (128, 2, 1, [(1025, 1500)]), (256, 1, 16, [(97, 300)])])
def test_attend_over_prompts(head_dim, kv, group, windows):
    """Windows of hundreds of tokens, behind earlier ones or from the first position on."""
    s = pu.scene(72, kv, head_dim, 64, windows)
    _attend(s, kv * group, 72)
