"""Attention over codes, and by work-groups that share their rows, whose runs walk more pages than a wave has lanes (a wave
holds 64 entries of a table's row or of a list at a time), against the FP64 reference."""

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from tests import paged_codes_util as cu
from tests import paged_util as pu
from tests.libhcr_util import ensure_built
from tests.test_paged_pairs import sanitized  # noqa: F401

# name -> (kv heads, heads, new tokens and positions of each sequence, entries of a list, window, first positions)
LONG = {
    "a sequence cut": (32, 32, [(1, 40000)], 0, 0, 0),
    "a window cut": (32, 32, [(1, 45000)], 0, 42000, 70),
    "first positions and a window, cut": (32, 64, [(1, 45000)], 0, 36000, 6000),
    "lists whole": (8, 8, [(4, 8400)] * 8, 130, 0, 0),
    "lists of shared rows": (16, 272, [(64, 9000)], 135, 0, 0),
    "a prompt of shared rows": (8, 512, [(130, 6600)], 0, 0, 0),
    "a prompt of shared rows through a window": (8, 512, [(130, 6600)], 0, 4400, 300),
    "first positions of shared rows": (8, 512, [(130, 6600)], 0, 300, 4500),
}
D, PAGE = 64, 64


def test_index_the_runs_pass_64_pages(sanitized):  # noqa: F811
    calls = [(code, D, kv, PAGE, heads, len(w), w[0][0], w[0][1], n_sel, size, first)
             for kv, heads, w, n_sel, size, first in LONG.values() for code in (2, 3)]
    runs = [int(x) for x in sanitized(f"print(*[L.paged_more_run_pages(*c) for c in {calls}])").split()]
    assert len(runs) == len(calls) and all(r > 64 for r in runs), runs


@pytest.mark.gpu
@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("name", sorted(LONG))
def test_long_runs(kind, name):
    ensure_built()
    kv, heads, windows, n_sel, size, first = LONG[name]
    group, head = heads // kv, min(3, kv - 1)  # one kv head against the reference
    s = cu.scene(kind, 180, kv, D, PAGE, windows)
    q = pu.queries(180, s.n_tokens, heads, D)
    sel = None
    if n_sel:
        pages = -(-windows[0][1] // PAGE)
        sel = np.stack([gen.rng(181, n).permutation(pages)[:n_sel] for n in range(s.n_tokens)])
        sel = np.ascontiguousarray(np.broadcast_to(sel[:, None], (s.n_tokens, kv, n_sel)).astype(np.int32))
    cache, batch, qd = cu.dev_cache(s), pu.dev_batch(s), pu.dev_bits(q)
    if size:
        out = cache.attend_window(batch, qd, size, first)
    elif n_sel:
        out = cache.attend_blocks(batch, qd, torch.from_numpy(sel).cuda())
    else:
        out = cache.attend(batch, qd)
    torch.cuda.synchronize()
    s.k_codes, s.v_codes, s.k_scales, s.v_scales = (a[:, head:head + 1] for a in (s.k_codes, s.v_codes, s.k_scales, s.v_scales))
    keys, values = cu.decoded(s)
    mine = slice(head * group, (head + 1) * group)
    qf = oracle.bf16_bits_to_f64(np.ascontiguousarray(q[:, mine]))
    if size:
        want = oracle.paged_codes.attend_window(s.batch, keys, values, qf, D ** -0.5, size, first)
    else:
        want = oracle.paged.attend(s.batch, keys, values, qf, D ** -0.5, sel=None if sel is None else sel[:, head:head + 1])
    tol = pu.rows_tolerance(qf, cu.reach(keys), D ** -0.5, windows[0][1], False)
    pu.check_rows(out[:, mine], want, tol, name)
