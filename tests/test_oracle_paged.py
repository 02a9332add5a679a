"""The paged-cache reference against things other than itself: torch's float64 softmax and layer functions, closed
forms and permutations of its pages, and planted mistakes (CPU only)."""

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from tests import paged_util as pu

ref = oracle.paged


def _plain(s, b, length):
    """A sequence's keys and values as [length][h][D], read cell by cell from the stored arrays."""
    page, D, KV = s.page, s.means.shape[2], s.means.shape[1]
    k, v = np.zeros((length, KV, D)), np.zeros((length, KV, D))
    for p in range(length):
        pg, slot = s.table[b, p // page], p % page
        for d in range(D):
            k[p, :, d] = oracle.bf16_bits_to_f64(s.k_bits[pg, :, d // 8, slot, d % 8])
            v[p, :, d] = oracle.bf16_bits_to_f64(s.v_bits[pg, :, slot // 8, d, slot % 8])
    return k, v


def pin_attend(attend):
    s = pu.scene(1, 2, 64, 32, [(3, 70), (1, 33)])
    q = oracle.bf16_bits_to_f64(pu.queries(1, 4, 6, 64))
    keys, values = pu.decoded(s)
    got = attend(s.batch, keys, values, q, 0.125)
    for n, b, p in ((0, 0, 67), (1, 0, 68), (2, 0, 69), (3, 1, 32)):
        k, v = _plain(s, b, p + 1)
        for hd in range(6):
            w = torch.softmax(torch.from_numpy(0.125 * (k[:, hd // 3] @ q[n, hd])), 0).numpy()
            assert np.allclose(got[n][hd], w @ v[:, hd // 3], rtol=1e-12, atol=1e-14)


def pin_attend_blocks(attend):
    """A list of every page in another order gives the same; a list of one page is that page's attention."""
    s = pu.scene(2, 1, 64, 32, [(1, 100)])
    q = oracle.bf16_bits_to_f64(pu.queries(2, 1, 2, 64))
    keys, values = pu.decoded(s)
    whole = attend(s.batch, keys, values, q, 0.1)
    listed = attend(s.batch, keys, values, q, 0.1, sel=np.array([[[3, -1, 1, 0, 9, 2]]]))
    assert np.allclose(whole[0], listed[0], rtol=1e-12)
    one = attend(s.batch, keys, values, q, 0.1, sel=np.array([[[2]]]))
    w = torch.softmax(torch.from_numpy(0.1 * keys[s.table[0, 2], 0] @ q[0].T), 0).numpy()
    assert np.allclose(one[0], w.T @ values[s.table[0, 2], 0], rtol=1e-12)
    none = attend(s.batch, keys, values, q, 0.1, sel=np.array([[[-1, 4]]]))
    assert np.all(none[0] == 0)


def pin_norm_rotate(norm_rotate):
    g = gen.rng(5, 6)
    x, w = g.standard_normal(64), g.uniform(0.5, 1.5, 64)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-6).numpy()
    assert np.allclose(norm_rotate(x, w, 1e-6, None, False), want, rtol=1e-13)
    angle = g.uniform(-3, 3, 8)
    row = np.concatenate([np.cos(angle), np.sin(angle)])
    for pairs in (False, True):
        y = norm_rotate(x, None, 1e-6, row, pairs)
        a, b = (np.arange(0, 16, 2), np.arange(1, 16, 2)) if pairs else (np.arange(8), np.arange(8, 16))
        z = (x[a] + 1j * x[b]) * np.exp(1j * angle)  # a rotation of the complex plane
        assert np.allclose(y[a] + 1j * y[b], z, rtol=1e-13) and np.array_equal(y[16:], x[16:])


def pin_append_positions(append):
    starts, lens = np.array([0, 3, 4], np.int32), np.array([2, 40], np.int32)
    table = np.array([[5, -1], [7, 6]], np.int32)
    x = gen.rng(5, 7).standard_normal((4, 1, 64))
    q_out, writes = append((starts, lens, table), 32, 8, x, x, x, None, None, 0.0, None, False)
    assert np.all(q_out[0] == 0) and np.array_equal(q_out[1], x[1])
    assert set(writes) == {(5, 0), (5, 1), (6, 7)}
    assert np.array_equal(writes[6, 7][0], x[3]) and np.array_equal(writes[5, 1][1], x[2])


def pin_scores(block_scores):
    g = gen.rng(5, 8)
    means, q = g.standard_normal((4, 2, 64)), g.standard_normal((1, 6, 64))
    got = block_scores((np.array([0, 1]), np.array([100]), np.array([[2, 3, -1, 0]])), means, 32, q)[0]
    assert got.shape == (2, 3) and np.all(np.isneginf(got[:, 2]))
    want = (torch.from_numpy(q[0]).view(2, 3, 64) @ torch.from_numpy(means[[2, 3]]).permute(1, 2, 0)).amax(1)
    assert np.allclose(got[:, :2], want.numpy(), rtol=1e-13)


def pin_topk(block_topk):
    batch = (np.array([0, 1]), np.array([32 * 9 + 1]), None)
    scores = np.array([[[-9, 1, 3, 3, np.nan, 3, 2, 3, 8, 7]]], np.float32)
    assert block_topk(batch, 32, scores, 5, 1, 2)[0].tolist() == [[0, 2, 3, 8, 9]]
    assert block_topk(batch, 32, scores, 6, 0, 1)[0].tolist() == [[2, 3, 5, 7, 8, 9]]
    assert block_topk(batch, 32, scores, 12, 1, 2)[0].tolist() == [list(range(10)) + [-1, -1]]


PINS = {"attend": [pin_attend, pin_attend_blocks], "norm_rotate": [pin_norm_rotate], "append": [pin_append_positions],
        "block_scores": [pin_scores], "block_topk": [pin_topk]}


@pytest.mark.parametrize("name", sorted(PINS))
def test_reference_pins(name):
    for pin in PINS[name]:
        pin(getattr(ref, name))


def _attend_with(**change):
    """The reference's attention with a mistake in what it is given."""
    def attend(batch, keys, values, q, scale, sel=None):
        q_start, ctx_len, table = batch
        batch = (q_start, np.asarray(ctx_len) + change.get("ctx", 0), change.get("table", lambda t: t)(table))
        if sel is not None:
            sel = change.get("sel", lambda x: x)(sel)
        q = change.get("q", lambda x: x)(q)
        return ref.attend(batch, change.get("keys", lambda x: x)(keys), change.get("values", lambda x: x)(values), q,
                          scale * change.get("scale", 1.0), sel=sel)
    return attend


MUTANTS = [
    ("attend", _attend_with(ctx=-1)),                                  # a position short
    ("attend", _attend_with(scale=1.01)),
    ("attend", _attend_with(keys=lambda k: k[:, ::-1])),               # another kv head
    ("attend", _attend_with(values=lambda v: np.roll(v, 1, axis=2))),  # another slot
    ("attend", _attend_with(table=lambda t: t[:, ::-1])),              # pages in another order
    ("attend", _attend_with(sel=lambda x: x[..., 1:])),
    ("norm_rotate", lambda x, w, eps, row, pairs: ref.norm_rotate(x, w, eps, row, not pairs)),
    ("norm_rotate", lambda x, w, eps, row, pairs: ref.norm_rotate(x, None, eps, row, pairs)),
    ("norm_rotate", lambda x, w, eps, row, pairs: ref.norm_rotate(x, w, eps, None if row is None else -row, pairs)),
    ("block_scores", lambda b, m, p, q: {n: -s for n, s in ref.block_scores(b, m, p, -q).items()}),  # the least head
    ("block_topk", lambda b, p, s, k, f, l: ref.block_topk(b, p, -s, k, f, l)),
    ("block_topk", lambda b, p, s, k, f, l: ref.block_topk(b, p, s, k, 0, l)),
]


@pytest.mark.parametrize("i", range(len(MUTANTS)))
def test_a_planted_mistake_fails_a_pin(i):
    name, wrong = MUTANTS[i]
    failed = 0
    for pin in PINS[name]:
        try:
            pin(wrong)
        except (AssertionError, IndexError, ValueError):  # noqa: PERF203
            failed += 1
    assert failed, f"mutant {i} of {name} passed every pin"


def test_stored_orders():
    """decode_keys and decode_values undo the stored orders."""
    x = gen.rng(5, 9).integers(0, 0x7F00, size=(2, 3, 32, 64)).astype(np.uint16)
    assert np.array_equal(ref.decode_keys(pu.store_keys(x)), oracle.bf16_bits_to_f64(x))
    assert np.array_equal(ref.decode_values(pu.store_values(x)), oracle.bf16_bits_to_f64(x))
