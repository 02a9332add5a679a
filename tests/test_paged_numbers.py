"""Numbers of the paged cache's kernels at their edges: bounds close enough that a rounding at the wrong place shows,
values that are no numbers, rows that must not feel their neighbours.

The close bounds use keys and queries whose products are whole numbers below 2^24, which FP32 sums hold exactly in any
order, so that the softmax and the second product alone are off.  In half steps (2^-24 of a value), for n positions
whose exponents of two lie within E of the row's maximum:

  exponent   two fused products, each rounded once, of size E + 1 at most: 2 (E + 1) ln 2 of a probability
  power      one step: 2
  sum        a chain of at most n additions, 16 more over lanes, waves and parts
  product    three parts a probability (their sum is all of its 24 bits), each added with at most one whole step: 6 n,
             16 more over waves and parts
  quotient   reciprocal and product: 3

Exponents and powers stand in the sum and in the product, so each counts twice."""

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from tests import paged_util as pu
from tests.libhcr_util import ensure_built

HALF = 2.0 ** -24
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def room(n, E):
    return (4 * np.log(2) * (E + 1) + 4 + (n + 16) + (6 * n + 16) + 3) * HALF


def _set_keys(s, keys):
    """Visible keys (the others stay NaN) [pages][kv heads][page][D]."""
    old = oracle.paged.decode_keys(s.k_bits)
    s.k_bits = pu.store_keys(np.where(np.isnan(old), np.uint16(pu.NAN_BITS), pu.bf16(keys)))


def _large_scores(seed, D, group, windows, around):
    """Products within 24 of ``around`` (under 2^21): whole numbers."""
    g = gen.rng(110, seed)
    s = pu.scene(seed, 1, D, 32, windows)
    keys = np.full((s.k_bits.shape[0], 1, 32, D), 128, np.float32)
    keys[..., :8] = g.integers(0, 4, keys[..., :8].shape)
    keys[..., 8] = 1
    _set_keys(s, keys)
    q = np.zeros((s.n_tokens, group, D), np.float32)
    q[..., :8] = g.integers(1, 3, q[..., :8].shape)
    base = around - 24
    q[..., 8] = base % 128
    share = base // 128
    for d in range(9, D):
        q[..., d] = share // (D - d)
        share -= share // (D - d)
    assert share == 0 and q.max() <= 256
    return s, q


def _close(out, s, q, scale, E, label):
    keys, values = pu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, q, scale)
    size = oracle.paged.attend(s.batch, keys, np.abs(values), q, scale)  # probabilities times magnitudes
    got = out.double().cpu().numpy()
    for n, b, p in oracle.paged.tokens(s.q_start, s.ctx_len):
        off = np.abs(got[n] - want[n]) - room(p + 1, E) * size[n]
        assert np.all(off <= 0), f"{label}: row {n} of sequence {b}, {off.max():.2e} too much"


# the first four: scores at which v times the scale's small part crosses half a step of the maximum (or one and a half)
LARGE = [(128, 128 ** -0.5, 852189), (128, 0.1, 495313), (64, 0.3, 330209), (256, -0.2, 990626),
         (128, 128 ** -0.5, 12288), (64, 0.125, 500000), (256, 0.0625, 1000000), (128, 0.3, 300001)]


@gpu
@pytest.mark.parametrize("D,scale,around", LARGE)
def test_large_scores_keep_their_differences(lib, D, scale, around):
    """Scores of up to 10^5 that differ by a few: exponents rounded at the scores' size would be off by 2^-6."""
    s, q = _large_scores(1, D, 6, [(3, 40), (1, 290), (2, 2), (1, 9)], around)
    out = pu.dev_cache(s).attend(pu.dev_batch(s), pu.dev_bits(pu.bf16(q)), scale=scale)
    _close(out, s, q, scale, 48 * abs(scale) * np.log2(np.e) + 8, f"D {D} scale {scale}")


def _fma(a, b, c):
    """FP32, rounded once (the product of two FP32 values is exact in 64 bits; of the sum's two roundings the first is
    2^-29 of the second)."""
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(np.float32)


def _parts(scale):
    log2e = scale * 1.4426950408889634
    hi = np.float32(log2e)
    if abs(float(hi)) >= abs(log2e):
        hi = np.nextafter(hi, np.float32(0))
    return hi, np.float32(log2e - float(hi))


@pytest.mark.parametrize("D,scale,around", LARGE[:4])
def test_a_maximum_subtracted_from_the_small_part_fails_the_bound(D, scale, around):
    """The bound sees the difference between v hi - max + v lo and v lo - max + v hi."""
    s, q = _large_scores(1, D, 6, [(1, 290)], around)
    keys, values = pu.decoded(s)
    k = np.concatenate([keys[j, 0] for j in s.table[0] if j >= 0])[:290]
    v = np.concatenate([values[j, 0] for j in s.table[0] if j >= 0])[:290]
    hi, lo = _parts(scale)
    x = (q[0] @ k.T).astype(np.float32)
    w = np.exp(scale * (x.astype(np.float64) - x.max(-1, keepdims=True)))
    w /= w.sum(-1, keepdims=True)
    top = (x * hi).max(-1, keepdims=True)
    bound = room(290, 48 * abs(scale) * np.log2(np.e) + 8)
    for order, fits in ((_fma(x, lo, _fma(x, hi, -top)), True), (_fma(x, hi, _fma(x, lo, -top)), False)):
        p = np.exp2(order.astype(np.float64))
        off = np.abs((p / p.sum(-1, keepdims=True)) @ v - w @ v)
        assert np.all(off <= bound * (w @ np.abs(v))) == fits


def _pairs(seed, D, group, count):
    """``count`` sequences of two positions, the first one's value zero: each row's output is the second's value times
    its probability, one in a row's sum of two.  Products are eighths, within 16 of each other."""
    g = gen.rng(111, seed)
    s = pu.scene(seed, 1, D, 32, [(1, 2)] * count)
    keys = np.broadcast_to(g.integers(-9, 10, D), (s.k_bits.shape[0], 1, 32, D)).astype(np.float32).copy()
    keys[:, :, 1, :8] = keys[:, :, 0, :8] + 1
    _set_keys(s, keys)
    s.v_bits[:, :, 0, :, 0] = 0
    q = g.integers(-16, 17, (count, group, D)).astype(np.float32) / 8
    return s, q


def _pair_room(scale):
    # sum: one addition; product: two of three parts added to the first, one whole step each
    return (4 * np.log(2) * (16 * abs(scale) * np.log2(np.e) + 1) + 4 + 1 + 4 + 3) * HALF


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 16, 64])
def test_float_outputs_take_whole_probabilities(lib, D, group):
    """Closer than two BF16 parts of a probability come (2^-18)."""
    scale = 0.0931
    s, q = _pairs(2, D, group, 40)
    keys, values = pu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, q, scale)
    out = pu.dev_cache(s).attend(pu.dev_batch(s), pu.dev_bits(pu.bf16(q)), scale=scale).double().cpu().numpy()
    for n, w in want.items():
        assert np.all(np.abs(out[n] - w) <= _pair_room(scale) * np.abs(w)), f"row {n}"


def test_two_parts_of_a_probability_fail_the_bound():
    scale = 0.0931
    s, q = _pairs(2, 128, 64, 40)
    keys, _ = pu.decoded(s)
    hi, lo = _parts(scale)
    x = np.stack([q[b] @ keys[s.table[b, 0], 0, :2].T for b in range(40)]).astype(np.float32)  # [40][64][2]
    top = (x * hi).max(-1, keepdims=True)
    p = np.exp2(_fma(x, lo, _fma(x, hi, -top)).astype(np.float64)).astype(np.float32)
    want = 1 / (1 + np.exp(scale * (x[..., 0] - x[..., 1]).astype(np.float64)))

    def bf16(a):
        return oracle.bf16_bits_to_f64(pu.bf16(a)).astype(np.float32)
    first = bf16(p)
    second = bf16(p - first)
    third = bf16(p - first - second)
    assert np.array_equal(first.astype(np.float64) + second + third, p)
    total = p.sum(-1, dtype=np.float64)
    for parts, fits in ((first.astype(np.float64) + second + third, True), (first.astype(np.float64) + second, False)):
        off = np.abs(parts[..., 1] / total - want)
        assert np.all(off <= _pair_room(scale) * want) == fits


@gpu
@pytest.mark.parametrize("head_dim,page,kv,group", [(128, 64, 2, 4), (64, 32, 1, 24), (256, 64, 1, 6), (128, 32, 2, 1),
                                                    (64, 64, 2, 16)])
@pytest.mark.parametrize("odd", [np.nan, np.inf, -np.inf])
def test_scores_of_what_is_no_number(lib, head_dim, page, kv, group, odd):
    """One head's query, one page's mean: the scores that they enter are the definition's, NaN or infinite; no other."""
    s = pu.scene(6, kv, head_dim, page, [(4, 40 * page + 3), (2, 9 * page), (1, 2 * page + 1)])
    s.table[1, 2] = -1
    q = pu.queries(6, s.n_tokens, kv * group, head_dim)
    bits = pu.bf16([odd])[0]
    q[1, group // 2, 7] = bits
    q[5, -1, 1] = bits
    s.means[s.table[0, 11], 0, 5] = bits
    s.means[s.table[1, 4], -1, head_dim - 1] = bits
    means, qf = oracle.bf16_bits_to_f64(s.means), oracle.bf16_bits_to_f64(q)
    with np.errstate(invalid="ignore"):
        want = oracle.paged.block_scores(s.batch, means, page, qf)
    scores = torch.zeros(s.n_tokens, kv, 41, device="cuda")
    pu.dev_cache(s).block_scores(pu.dev_batch(s), pu.dev_bits(q), scores=scores)
    got = scores.double().cpu().numpy()
    fine_q, fine_m = (np.where(np.isfinite(x), x, 0) for x in (qf, means))
    room = head_dim * HALF * float(np.abs(fine_q).sum(-1).max() * np.abs(fine_m).max())
    odd_ones = 0
    for n, w in want.items():
        g = got[n, :, :w.shape[1]]
        assert np.array_equal(np.isnan(w), np.isnan(g)) and np.array_equal(np.isinf(w), np.isinf(g)), f"row {n}"
        assert np.array_equal(w[np.isinf(w)], g[np.isinf(w)])
        fine = np.isfinite(w)
        odd_ones += (~fine).sum()
        assert np.all(np.abs(g[fine] - w[fine]) <= room), f"row {n}"
    assert odd_ones > 20


SHAPES = [(128, 2, 4, 5), (256, 1, 6, 7), (64, 1, 8, 20), (128, 1, 12, 3), (256, 2, 10, 3), (256, 1, 16, 9)]


@gpu
@pytest.mark.parametrize("D,kv,group,T", SHAPES)
@pytest.mark.parametrize("odd", [np.inf, -np.inf, np.nan])
def test_a_value_that_is_no_number_reaches_its_own_dimension(lib, D, kv, group, T, odd):
    """Wherever in its tile, whichever rows see it: a product's other dimensions are as ever."""
    windows = [(T, 300), (T, 64), (T, T), (T, 5003), (T, 160 + T // 2)]
    s = pu.scene(3, kv, D, 64, windows)
    q = pu.queries(3, s.n_tokens, kv * group, D)
    qf = oracle.bf16_bits_to_f64(q)
    keys, values = pu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, qf, 0.1)
    tol = pu.rows_tolerance(qf, float(np.sqrt(np.nansum(keys ** 2, axis=-1)).max()), 0.1, 5003, False)
    bits = pu.bf16([odd])[0]
    # dimension 3 mod 16 of every sequence's last but one position, dimension 5 of its window's first
    hit = np.zeros((s.n_tokens, D), bool)
    for b, (_, c) in enumerate(windows):
        for at, dim in ((c - 2, 3), (c - T, 5)):
            s.v_bits[s.table[b, at // 64], :, at % 64 // 8, dim::16, at % 8] = bits
            hit[s.q_start[b] + at - (c - T):s.q_start[b + 1], dim::16] = True
    out = pu.dev_cache(s).attend(pu.dev_batch(s), pu.dev_bits(q), scale=0.1)
    got = out.double().cpu().numpy()
    for n, w in want.items():
        assert not np.isfinite(got[n][:, hit[n]]).any(), f"row {n}"
        off = np.linalg.norm((got[n] - w)[:, ~hit[n]], axis=1)
        assert np.all(off <= tol * np.linalg.norm(w, axis=1)), f"row {n}"


@gpu
@pytest.mark.parametrize("D,kv,group,T", SHAPES + [(128, 1, 1, 16), (64, 1, 1, 31)])
@pytest.mark.parametrize("later", ["large", np.inf, np.nan])
def test_rows_do_not_feel_later_tokens(lib, D, kv, group, T, later):
    """Bit for bit: the last token's query, key and value are others, the rows before it the same."""
    windows = [(T, 290 + T), (T, 2 * T), (T, T), (T, 3000 + T)]
    a, b = (pu.scene(4, kv, D, 64, windows) for _ in range(2))
    q = pu.queries(4, a.n_tokens, kv * group, D)
    first = pu.dev_cache(a).attend(pu.dev_batch(a), pu.dev_bits(q), scale=0.05)
    last = np.arange(a.n_tokens) % T == T - 1
    for i, (_, c) in enumerate(windows):
        page, slot = b.table[i, (c - 1) // 64], (c - 1) % 64
        if later == "large":
            b.k_bits[page, :, :, slot] ^= 0x8000
            b.v_bits[page, :, slot // 8, :, slot % 8] ^= 0x8000
        else:
            b.k_bits[page, :, 0, slot, 0] = pu.bf16([later])[0]
            b.v_bits[page, :, slot // 8, 1, slot % 8] = pu.bf16([later])[0]
    q[last] = pu.bf16(oracle.bf16_bits_to_f64(q[last]) * 16)
    again = pu.dev_cache(b).attend(pu.dev_batch(b), pu.dev_bits(q), scale=0.05)
    keep = torch.from_numpy(~last).cuda()
    assert torch.isfinite(first).all() and torch.equal(first[keep], again[keep])


@gpu
@pytest.mark.parametrize("scale", [1e-30, -3e-38, 1e-42, -1e-45, 1e-300])
def test_a_product_of_minus_infinity_weighs_nothing_at_any_scale(lib, scale):
    s = pu.scene(5, 1, 64, 32, [(2, 70), (1, 33)])
    q = pu.queries(5, s.n_tokens, 4, 64)
    q[..., 0] = pu.bf16([2.0])[0]
    for b, at in ((0, 5), (0, 66), (1, 0)):
        s.k_bits[s.table[b, at // 32], 0, 0, at % 32, 0] = pu.bf16([-np.inf if scale > 0 else np.inf])[0]
    keys, values = pu.decoded(s)
    qf = oracle.bf16_bits_to_f64(q)
    want = oracle.paged.attend(s.batch, keys, values, qf, scale)
    out = pu.dev_cache(s).attend(pu.dev_batch(s), pu.dev_bits(q), scale=scale)
    pu.check_rows(out, want, pu.rows_tolerance(qf, 20.0, scale, 70, False), "small scale")
