"""Codes bit for bit: the scale is FP32's largest magnitude / top, the code the one nearest to FP32's quotient by that
scale.  Rows without norm and rotation, whose values reach the quantisation as they are, so that nothing but those two
divisions rounds and every scale and code is known exactly."""

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


def expected(x, kind):
    """(scales, values of the codes) of heads x, float32 [...][D], by FP32's divisions (numpy's, correctly rounded)."""
    top = np.abs(x).max(-1)
    scale = top / np.float32(o.TOP[kind])
    with np.errstate(invalid="ignore", divide="ignore"):
        ratio = np.where(scale[..., None] > 0, x / scale[..., None], np.float32(0))
    assert scale.dtype == ratio.dtype == np.float32
    return scale, o.nearest(ratio, kind)


def append(kind, x, dtype, page):
    """Rows x [n][heads][D] as keys and as values of one sequence; (scales, values of the codes), each of both."""
    n, heads, D = x.shape
    pages = -(-n // page)
    cache = paged.PagedCache.allocate(pages, heads, D, page, dtype=cu.DTYPE[kind])
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = paged.Batch(torch.tensor([0, n], **i32), torch.tensor([n], **i32), torch.arange(pages, **i32)[None], n, n)
    rows = torch.from_numpy(x).cuda().to(dtype)
    assert torch.equal(rows.float().cpu(), torch.from_numpy(x))
    cache.append(batch, rows, rows, rows)
    torch.cuda.synchronize()
    out = []
    for scales, codes, load in ((cache.k_scales, cache.k_pages, o.load_keys), (cache.v_scales, cache.v_pages, o.load_values)):
        got = o.code_values(load(cu.host_codes(codes)), kind)
        out.append((scales.cpu().numpy().transpose(0, 2, 1).reshape(-1, heads)[:n],
                    got.transpose(0, 2, 1, 3).reshape(-1, heads, D)[:n]))
    return out


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("head_dim,page,n", [(128, 64, 700), (64, 128, 31), (256, 64, 200)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codes_are_those_of_the_quotients(kind, head_dim, page, n, dtype):
    """Windows on both sides of 32 tokens.  BF16 rows: their quotients often lie by the middle of two codes."""
    x = (gen.rng(130, head_dim).standard_normal((n, 4, head_dim)) * 3).astype(np.float32)
    if dtype == torch.bfloat16:
        x = oracle.bf16_bits_to_f64(pu.bf16(x)).astype(np.float32)
    scale, values = expected(x, kind)
    for got_scales, got in append(kind, x, dtype, page):
        assert np.array_equal(got_scales, scale)
        assert np.array_equal(got, values), f"{(got != values).sum()} of {values.size} codes differ"


@pytest.mark.parametrize("kind", cu.KINDS)
@pytest.mark.parametrize("n", [24, 64])
def test_codes_of_small_and_large_scales(kind, n):
    """Scales of a few steps of FP32's smallest numbers, around its smallest normal one, around 2^-100 and by its largest
    number, ordinary heads in the same wave.  A scale of few bits may be well below max / top: codes stop at top."""
    g = gen.rng(131, n)
    top = o.TOP[kind]
    x = (g.uniform(-1, 1, (n, 2, 128))).astype(np.float32)
    x[..., 7] = 1  # the largest
    for i in range(0, n, 2):
        step = i // 2 % 12
        largest = np.float32([300 * 2.0 ** -149, 700 * 2.0 ** -149, 2000 * 2.0 ** -149, 50000 * 2.0 ** -149,
                              top * 2.0 ** -126 * 0.999, top * 2.0 ** -126 * 1.001, top * 2.0 ** -100 * 0.999,
                              top * 2.0 ** -100 * 1.001, 3.4028234e38, 1e38, 5e-39, top * 3 * 2.0 ** -149][step])
        x[i, i // 2 % 2] = (x[i, i // 2 % 2].astype(np.float64) * float(largest)).astype(np.float32)
    scale, values = expected(x, kind)
    assert np.all(scale > 0) and (scale < 2.0 ** -126).sum() >= n // 6
    for got_scales, got in append(kind, x, torch.float32, 64):
        assert np.array_equal(got_scales, scale)
        assert np.array_equal(got, values)
