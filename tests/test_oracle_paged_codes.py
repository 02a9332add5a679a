"""Pins of the reference of codes and windows (oracle/paged_codes.py) against torch's own 8-bit floats, brute force and
the plain attention reference."""

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from tests import paged_util as pu

o = oracle.paged_codes


def test_e4m3_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(o.code_values(codes, "e4m3"), want, equal_nan=True)


def test_nearest_e4m3_rounds_as_torch_does():
    g = gen.rng(120, 0)
    x = np.concatenate([g.uniform(-448, 448, 4000), g.standard_normal(4000) * 0.02,
                        (o.e4m3_table()[:126] + o.e4m3_table()[1:127]) / 2])  # ties
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(o.nearest(x, "e4m3"), want)


def test_int8_ties_go_to_even():
    assert o.nearest([0.5, 1.5, -2.5, 126.5, 200.0, -200.0], "int8").tolist() == [0, 2, -2, 126, 127, -127]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_bytes_and_back(kind):
    g = gen.rng(121, 0)
    values = o.nearest(g.uniform(-o.TOP[kind], o.TOP[kind], (3, 2, 64, 64)), kind)
    codes = o.to_bytes(values, kind)
    assert np.array_equal(o.code_values(codes, kind), values)
    assert np.array_equal(o.load_keys(o.store_keys(codes)), codes)
    assert np.array_equal(o.load_values(o.store_values(codes)), codes)
    k, v = o.store_keys(codes), o.store_values(codes)
    assert k[1, 1, 2, 37, 5] == codes[1, 1, 37, 37] and v[2, 0, 3, 41, 6] == codes[2, 0, 54, 41]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_quantise(kind):
    x = gen.rng(122, 0).standard_normal((5, 64))
    x[1] = 0
    x[2, 7] = np.inf
    x[3, 9] = np.nan
    ratio, scale = o.quantise(x, kind)
    assert scale[1] == 0 and np.isnan(scale[2]) and np.isnan(scale[3])
    assert np.all(ratio[1:4] == 0) and np.abs(ratio[0]).max() == o.TOP[kind]
    assert np.allclose(ratio[0] * scale[0], x[0]) and np.allclose(ratio[4] * scale[4], x[4])


def test_a_window_of_everything_is_plain_attention():
    s = pu.scene(40, 2, 64, 32, [(3, 100), (1, 5), (4, 2), (2, 64)])
    q = oracle.bf16_bits_to_f64(pu.queries(40, s.n_tokens, 4, 64))
    keys, values = pu.decoded(s)
    want = oracle.paged.attend(s.batch, keys, values, q, 0.1)
    for window, n_first in ((100, 0), (1000, 7), (1, 100), (50, 51)):
        got = o.attend_window(s.batch, keys, values, q, 0.1, window, n_first)
        for n in want:
            assert np.allclose(got[n], want[n], rtol=1e-12, atol=0)


def test_a_window_position_by_position():
    """Against attention over a cache of which only the window's positions are left."""
    s = pu.scene(41, 1, 64, 32, [(1, 150)])
    q = oracle.bf16_bits_to_f64(pu.queries(41, 1, 2, 64))
    keys, values = pu.decoded(s)
    for window, n_first in ((1, 0), (1, 1), (40, 3), (150, 0), (60, 95)):
        cells = [j for j in range(150) if j > 149 - window or j < n_first]
        k = np.stack([keys[s.table[0, j // 32], 0, j % 32] for j in cells])
        v = np.stack([values[s.table[0, j // 32], 0, j % 32] for j in cells])
        e = np.exp(0.1 * q[0] @ k.T)
        got = o.attend_window(s.batch, keys, values, q, 0.1, window, n_first)[0]
        assert np.allclose(got, e @ v / e.sum(-1, keepdims=True), rtol=1e-12, atol=0)


def test_read():
    s = pu.scene(42, 2, 64, 32, [(3, 70), (2, 1)])
    s.table[0, 2] = -1
    keys, _ = pu.decoded(s)
    got = o.read(s.batch, keys)
    assert np.all(got[0] == 0) and np.all(got[2] == 0) and np.all(got[3] == 0)  # page -1; position -1
    assert np.array_equal(got[4], keys[s.table[1, 0], :, 0])
