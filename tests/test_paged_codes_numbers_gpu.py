"""Numbers at their ends in a cache of codes.  E4M3 codes of values that are no numbers: each reaches its own dimension of
the rows that see it and nothing else, in whatever tile and cut it lies; a scale that is none reaches all dimensions of
them.  Scales from 2^-96 up to where sums stay finite."""

import numpy as np
import pytest
import torch

import oracle
from tests import paged_codes_util as cu
from tests import paged_util as pu
from tests.libhcr_util import ensure_built

pytestmark = pytest.mark.gpu
o = oracle.paged_codes


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


# head_dim, page, kv heads, group, new tokens: a wave's rows; shared ones; several row blocks
SHAPES = [(64, 64, 2, 4, 1), (128, 64, 1, 4, 1), (256, 64, 1, 6, 1), (64, 64, 1, 4, 3), (128, 128, 2, 2, 5), (256, 64, 1, 5, 3),
          (64, 64, 1, 8, 5), (128, 64, 1, 8, 3), (256, 64, 1, 6, 6), (128, 64, 1, 8, 40)]


@pytest.mark.parametrize("head_dim,page,kv,group,T", SHAPES)
@pytest.mark.parametrize("how", ["all", "window", "listed"])
def test_a_value_that_is_no_number_stays_in_its_dimension(head_dim, page, kv, group, T, how):
    """At positions of whole tiles, of partly visible ones and of the window's own tokens; lengths in one tile and cut
    over work-groups."""
    lens = [c for c in (T, T + 2, 40, 64, 100, 700, 6001) if c >= T]
    windows = [(T, c) for c in lens]
    s = cu.scene("e4m3", 160, kv, head_dim, page, windows)
    codes = o.load_values(s.v_codes)
    size, first = (90, 5) if how == "window" else (0, 0)
    sel = None
    spoiled = {}  # row -> dimensions, of every head
    for b, (_, c) in enumerate(windows):
        for n, p in enumerate(sorted({0, 3, c // 2, c - T, c - 1, max(c - 70, 0)})):
            dim = (7 * n + 16 * b + n // 2 * 33) % head_dim
            codes[s.table[b, p // page], :, p % page, dim] = 0xFF if n % 2 else 0x7F
            for t in range(T):
                at = c - T + t
                if p <= at and (how != "window" or p > at - size or p < first):
                    spoiled.setdefault(b * T + t, set()).add(dim)
    s.v_codes = o.store_values(codes)
    if how == "listed":  # every page, backwards
        pages = max(-(-c // page) for c in lens)
        sel = np.ascontiguousarray(np.broadcast_to(np.arange(pages)[::-1].astype(np.int32), (s.n_tokens, kv, pages)))
    out, want, tol = cu.attend(s, kv * group, sel=sel, window=size or None, n_first=first)
    got = out.double().cpu().numpy()
    for m in range(s.n_tokens):
        dims = sorted(spoiled.get(m, ()))
        bad = np.zeros(head_dim, bool)
        bad[dims] = True
        assert np.array_equal(np.isnan(got[m]), np.broadcast_to(bad, got[m].shape)), f"row {m}: {dims}"
        assert np.array_equal(np.isnan(want[m]), np.broadcast_to(bad, want[m].shape)), f"the reference's row {m}"
        for hd in range(kv * group):
            off = np.linalg.norm(got[m, hd, ~bad] - want[m][hd, ~bad])
            assert off <= tol * np.linalg.norm(want[m][hd, ~bad]), f"row {m} head {hd}"


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group,T", SHAPES)
def test_scales_that_are_no_numbers_reach_the_rows_that_see_them(kind, head_dim, page, kv, group, T):
    windows = [(T, c) for c in (T + 2, 40 + T, 700, 5000)]
    for at, name in ((-1, "k_scales"), (-1, "v_scales"), (-T, "v_scales"), (0, "k_scales")):
        s = cu.scene(kind, 161, kv, head_dim, page, windows)
        for b, (_, c) in enumerate(windows):
            p = c + at if at < 0 else 0
            getattr(s, name)[s.table[b, p // page], :, p % page] = np.nan
        out, want, tol = cu.attend(s, kv * group)
        got = np.isnan(out.cpu().numpy()).all((1, 2))
        some = np.isnan(out.cpu().numpy()).any((1, 2))
        see = np.array([(c - T + t >= (c + at if at < 0 else 0)) for _, c in windows for t in range(T)])
        assert np.array_equal(got, see) and np.array_equal(some, see)
        pu.check_rows(out, {m: w for m, w in want.items() if not see[m]}, tol, name)


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,kv,group,T", SHAPES)
@pytest.mark.parametrize("exponent", [-96, -60, 60, 104])
def test_values_of_small_and_large_scales(kind, head_dim, page, kv, group, T, exponent):
    """From where a probability times its value's scale has all of its BF16 parts up to where sums stay finite."""
    s = cu.scene(kind, 162, kv, head_dim, page, [(T, T + 2), (T, 300 + T), (T, 3000)])
    s.v_scales = (s.v_scales.astype(np.float64) * 2.0 ** exponent).astype(np.float32)
    out, want, tol = cu.attend(s, kv * group)
    pu.check_rows(out, want, tol, f"2^{exponent}")
