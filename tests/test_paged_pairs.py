"""Batches of prompts and single tokens together: attention counts the pairs of a sequence and a row block that there are, so
that no work-group has much more to do than its share.  The index arithmetic on the host, under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/asan/paged_pairs_stubs.cpp); outputs on the GPU against the FP64 reference."""

import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from bf16_hyper_connection_amd import inputs as gen
from bf16_hyper_connection_amd import paged
from tests import paged_codes_util as cu
from tests import paged_util as pu
from tests.libhcr_util import ROOT, ensure_built

CSRC = os.path.join(ROOT, "bf16_hyper_connection_amd", "csrc")


@pytest.fixture(scope="module")
def sanitized(tmp_path_factory):
    cxx = next((c for c in ("g++", "c++") if shutil.which(c)), None)
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("paged_pairs") / "libpaged_pairs_asan.so")
    asan = [os.path.join(ROOT, "tests", "asan", f) for f in ("paged_stubs.cpp", "paged_q8_stubs.cpp", "paged_pairs_stubs.cpp")]
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-shared", "-fPIC", "-Wall", "-Werror", "-D__host__=", "-D__device__=",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "hcr_paged_api.cpp"),
           os.path.join(CSRC, "hcr_paged_q8_api.cpp"), *asan, "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    libasan = subprocess.run([cxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()

    def run(code):
        env = dict(os.environ, LD_PRELOAD=libasan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
                   UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        head = f"import ctypes\nL = ctypes.CDLL({out!r})\nL.paged_pairs_checks.restype = ctypes.c_char_p\n" \
               "L.paged_pairs_longest.restype = ctypes.c_longlong\n"
        r = subprocess.run([sys.executable, "-c", head + code], env=env, capture_output=True, text=True, timeout=900)
        assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
        assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr
        return r.stdout.strip()
    return run


def test_index_runs_of_pairs_cover_every_tile_once(sanitized):
    assert sanitized("print(L.paged_pairs_checks().decode())") == "ok"


@pytest.mark.parametrize("code", [1, 2, 3])
@pytest.mark.parametrize("size", [0, 5000])
@pytest.mark.parametrize("head_dim,heads", [(64, 64), (128, 32), (256, 48)])
@pytest.mark.parametrize("ctx", [8192, 60000])
def test_index_a_prompt_among_single_tokens_leaves_no_work_group_with_many(sanitized, code, size, head_dim, heads, ctx):
    """63 single tokens beside a prompt of 2,048: no run is longer than two shares of what 256 CUs have to do together (a
    work-group used to walk all of the 63 sequences)."""
    longest, total = map(int, sanitized(
        "t = ctypes.c_longlong()\n"
        f"print(L.paged_pairs_longest({code}, {head_dim}, 8, {heads}, {size}, 2048, 63, {ctx}, ctypes.byref(t)), t.value)").split())
    assert 0 < longest <= 2 * total * 8 / 256


@pytest.mark.parametrize("code", [1, 2, 3])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_index_no_set_of_more_than_4096_positions_is_one_work_groups(sanitized, code, head_dim):
    """Whatever a tile has: a long sequence among short ones would hold a single CU for the whole call."""
    lines = sanitized(f"for size in (0, 4096, 4500, 10000):\n  for sets in (1, 4, 16, 31, 32, 63, 64, 128, 1000):\n"
                      f"    for ctx in (1000, 1500, 2040, 4096, 4160, 5000, 8192, 10000, 20000):\n"
                      f"      print(size, sets, ctx, L.paged_plan_whole({code}, {head_dim}, 8, 32, size, sets, ctx))").splitlines()
    assert len(lines) == 4 * 9 * 9
    for line in lines:
        size, sets, ctx, whole = map(int, line.split())
        if code != 1 or size:
            # fewer sets than CUs: those that end as soon as runs and their join
            most = {64: 1024, 128: 768, 256: 384}[head_dim] * (4096 + max(8 * sets - 64, 0) ** 2) / 4096
            if whole and sets < 32 and code != 1:
                assert min(ctx, size or ctx) <= most, line
            if whole:
                assert min(ctx, size or ctx) <= 4096 + (256 if size else 0), line  # the ends of a window's tiles
            elif sets >= 64:
                assert min(ctx, size or ctx) > 4096, line


BATCHES = {  # windows (new tokens, positions), bounds above what there is
    "a prompt among single tokens": ([(1, 3 + 37 * i) for i in range(20)] + [(230, 230)] + [(1, 900 - 41 * i) for i in range(20)], {}),
    "prompts behind long contexts": ([(97, 5000), (1, 9001), (33, 33), (150, 700), (0, 300), (1, 0)], {}),
    "past 64 sequences": ([(0, 50)] * 30 + [(1, 7000)] + [(1, 40)] * 40 + [(140, 300)] + [(1, 11)] * 30 + [(35, 4500)], {}),
    "loose bounds": ([(1, 600), (70, 800), (1, 2300), (2, 1)], dict(max_tokens=400, max_ctx=9000)),
    "tokens before the first position": ([(130, 100), (1, 6000), (40, 20)], {}),
    "whole sequences": ([(1, 20 + 3 * i) for i in range(60)] + [(300, 300)], {}),
    "alike prompts": ([(64, 4500), (60, 3100), (57, 60)], {}),
}
SHAPES = [(128, 64, 8, 16), (64, 64, 16, 16), (256, 64, 8, 12)]  # head_dim, page, kv heads, group


def bounds_of(windows, bounds):
    return bounds.get("max_tokens", max(t for t, _ in windows)), bounds.get("max_ctx", max(c for _, c in windows))


def test_index_the_scenes_pairs_are_counted(sanitized):
    calls = [(code, D, kv, page, kv * group, size, len(w), sum(t for t, _ in w), *bounds_of(w, b))
             for w, b in BATCHES.values() for D, page, kv, group in SHAPES for code in (1, 2, 3) for size in (0, 90, 6000)]
    counted = sanitized(f"print(*[L.paged_plan_paired(*c) for c in {calls}])").split()
    assert len(counted) == len(calls)
    for name, (w, b) in BATCHES.items():
        for size in (0, 6000):
            for code in (1, 2, 3):
                of = [int(x) for c, x in zip(calls, counted) if c[0] == code and c[5] == size and c[6] == len(w)]
                assert sum(of) >= 2, (name, size, code, of)


def check_one_head(s, kind, kv, group, head, out, q, window=None, n_first=0):
    """One kv head's rows against the reference."""
    keys, values = (x[:, head:head + 1] for x in cu.decoded(s))
    mine = slice(head * group, (head + 1) * group)
    qf = oracle.bf16_bits_to_f64(np.ascontiguousarray(q[:, mine]))
    sc = q.shape[2] ** -0.5
    if window is None:
        want = oracle.paged.attend(s.batch, keys, values, qf, sc)
    else:
        want = oracle.paged_codes.attend_window(s.batch, keys, values, qf, sc, window, n_first)
    tol = pu.rows_tolerance(qf, cu.reach(keys), sc, int(max(s.ctx_len.max(), 1)), out.dtype == torch.bfloat16)
    pu.check_rows(out[:, mine], want, tol, f"{kind} head {head}")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
@pytest.mark.parametrize("head_dim,page,kv,group", SHAPES)
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_attend(kind, head_dim, page, kv, group, name):
    ensure_built()
    windows, bounds = BATCHES[name]
    s = cu.scene(kind, 140, kv, head_dim, page, windows, table_extra=150)
    q = pu.queries(140, s.n_tokens + 3, kv * group, head_dim)
    out = torch.full((s.n_tokens + 3, kv * group, head_dim), 5.0, device="cuda")
    cu.dev_cache(s).attend(pu.dev_batch(s, **bounds), pu.dev_bits(q), out=out)
    torch.cuda.synchronize()
    assert torch.all(out[s.n_tokens:] == 5.0)
    check_one_head(s, kind, kv, group, 1, out, q)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,head_dim,page,kv,group", [("int8", 128, 64, 8, 16), ("bf16", 128, 64, 8, 16), ("bf16", 64, 32, 16, 16),
                                                         ("e4m3", 64, 64, 16, 16), ("int8", 256, 64, 8, 12)])
@pytest.mark.parametrize("window,n_first", [(90, 0), (6000, 70)])
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_attend_window(kind, head_dim, page, kv, group, window, n_first, name):
    ensure_built()
    windows, bounds = BATCHES[name]
    s = cu.scene(kind, 141, kv, head_dim, page, windows, table_extra=300)
    q = pu.queries(141, s.n_tokens, kv * group, head_dim)
    out = cu.dev_cache(s).attend_window(pu.dev_batch(s, **bounds), pu.dev_bits(q), window, n_first, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    check_one_head(s, kind, kv, group, kv - 1, out, q, window, n_first)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
def test_a_graph_of_mixed_batches_reads_the_lengths_of_its_replay(kind):
    """Which sequence is the prompt, and how long they all are, changes between replays."""
    ensure_built()
    windows = [(200, 200), (1, 6000), (1, 33), (40, 3000)]
    s = cu.scene(kind, 142, 16, 64, 64, [(1, 6000)] * 4)
    cache = cu.dev_cache(s)
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, lens = torch.zeros(5, **i32), torch.ones(4, **i32)
    batch = paged.Batch(starts, lens, torch.from_numpy(s.table).cuda(), 200, 6000)
    bits = pu.queries(142, 242, 128, 64)
    q = pu.dev_bits(bits)
    tol = pu.rows_tolerance(oracle.bf16_bits_to_f64(bits), cu.reach(cu.decoded(s)[0]), 64 ** -0.5, 6000, False)

    def calls():
        return [cache.attend(batch, q), cache.attend_window(batch, q, 1000, 5)]
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for turn in range(5):
        now = windows[turn % 4:] + windows[:turn % 4]
        starts.copy_(torch.from_numpy(np.cumsum([0] + [t for t, _ in now])))
        lens.copy_(torch.tensor([c for _, c in now]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, calls()))
        # each sequence by itself: the same sums in another cut
        for b, (t, c) in enumerate(now):
            one = paged.Batch(torch.tensor([0, t], **i32), lens[b:b + 1].contiguous(), batch.block_table[b:b + 1].contiguous(), t, c)
            rows = slice(int(starts[b]), int(starts[b]) + t)
            for all_, alone in zip(got, (cache.attend(one, q[rows].contiguous()),
                                         cache.attend_window(one, q[rows].contiguous(), 1000, 5))):
                off, norm = ((x.double().norm(dim=2) for x in (all_[rows] - alone, alone)))
                assert torch.all(off <= 2 * tol * norm)


def test_index_batches_whose_pairs_no_launch_holds_are_not_refused(sanitized):
    """A million sequences, most of them padding, with a bound of 4 tokens of 256 heads over 8: 8 million pairs may be there."""
    from bf16_hyper_connection_amd import hcr
    for code, ctx in ((1, 20000), (2, 20000)):
        make = "hcr_cache_create_q8(V(K), V(2 * K), V(3 * K), V(4 * K), None, 2, 1000, 8, 64, 64, P(h))" if code == 2 else \
            "hcr_cache_create(V(K), V(2 * K), None, 1000, 8, 64, 64, P(h))"
        rc = int(sanitized(
            "import sys; sys.path.insert(0, '.')\nfrom bf16_hyper_connection_amd import paged\n"
            "K = 1 << 46\nh, V, P = ctypes.c_void_p(), ctypes.c_void_p, ctypes.byref\n"
            f"assert L.{make} == 0\n"
            f"b = paged.hcr_batch(1000000, 16, 4, {ctx}, 1 << 10, 16, 1 << 30, 1 << 40)\n"
            "L.hcr_attn.argtypes = [V, V, ctypes.c_int, ctypes.c_double, V, ctypes.c_int, V, V, ctypes.c_size_t, V]\n"
            "print(L.hcr_attn(h, P(b), 256, 0.1, 5 * K, 1, 6 * K, 7 * K, 1 << 40, None))"))
        assert rc == hcr.HCR_EHIP, (code, ctx)  # every check passed: the stand-in's answer


@pytest.mark.gpu
@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
@pytest.mark.parametrize("alike", [True, False])
def test_many_sequences_of_several_row_blocks(kind, alike):
    """More sequences than a wave has lanes over the same pages, of as many row blocks each and not: each as by itself."""
    ensure_built()
    kv, group, T, n = 32, 64, 34 if kind != "bf16" else 80, 70
    s = cu.scene(kind, 143, kv, 64, 64, [(T, 4500)])
    cache = cu.dev_cache(s)
    g = gen.rng(144)
    tokens = [T if alike or i % 3 == 0 else int(g.integers(0, 4)) for i in range(n)]
    ctx = [int(c) for c in g.integers(T, 4501, n)]
    i32 = dict(dtype=torch.int32, device="cuda")
    starts = np.cumsum([0] + tokens)
    batch = paged.Batch(torch.tensor(starts, **i32), torch.tensor(ctx, **i32),
                        torch.from_numpy(np.repeat(s.table, n, 0)).cuda(), T, 4500)
    q = torch.randn(int(starts[-1]), kv * group, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(5)) * 2
    q = q.to(torch.bfloat16)
    for call in (lambda b, x: cache.attend(b, x), lambda b, x: cache.attend_window(b, x, 4300, 3)):
        out = call(batch, q)
        for i in (0, 1, 2, 33, 63, 64, 69):
            if not tokens[i]:
                continue
            one = paged.Batch(torch.tensor([0, tokens[i]], **i32), torch.tensor([ctx[i]], **i32), batch.block_table[:1], tokens[i], 4500)
            rows = slice(int(starts[i]), int(starts[i + 1]))
            alone = call(one, q[rows].contiguous())
            tol = pu.rows_tolerance(q[rows].double().cpu().numpy(), cu.reach(cu.decoded(s)[0]), 64 ** -0.5, 4500, False)
            off, norm = (x.double().norm(dim=2) for x in (out[rows] - alone, alone))
            assert torch.all(off <= 2 * tol * norm), i
