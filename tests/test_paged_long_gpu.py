"""The paged cache on the GPU at sizes that take its kernels' longer ways: runs over more pages than a wave holds
entries of."""

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
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
