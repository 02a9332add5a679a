"""The paged cache's C ABI on the host: the library exports what include/hcr_paged.h declares and rejects bad
arguments before any HIP call; its index arithmetic stays inside the buffers.  No GPU is used: the device
addresses are made up, and every call here is one that the checks reject or an empty one.

The same calls run against a build of the host code under AddressSanitizer and UndefinedBehaviorSanitizer
(PAGED_ABI_LIB), where the launchers are stand-ins."""

import ctypes
import os
import re
import shutil
import subprocess
import sys
import types

import pytest
import torch

from bf16_hyper_connection_amd import hcr, paged
from tests.libhcr_util import ROOT, ensure_built

CSRC = os.path.join(ROOT, "bf16_hyper_connection_amd", "csrc")
SANITIZED = os.environ.get("PAGED_ABI_LIB")

GB = 1 << 30
K, V, M, Q, O, SC, SEL, S, R = (i * 4 * GB for i in range(16, 25))
STARTS, LENS, TABLE = 30 * 4 * GB, 31 * 4 * GB, 32 * 4 * GB
WN = 33 * 4 * GB


@pytest.fixture(scope="module")
def lib():
    if SANITIZED:
        L = ctypes.CDLL(SANITIZED)
        real = paged.lib() if os.path.exists(hcr.LIB_PATH) else None
        for n in declared():
            f = getattr(L, n)
            if real is not None:
                f.restype, f.argtypes = getattr(real, n).restype, getattr(real, n).argtypes
        return L
    ensure_built()
    return paged.lib()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hcr_paged.h")).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(hcr_[a-z_]+)\s*\(", text)))


def test_exports_every_declared_symbol(lib):
    names = declared()
    assert {"hcr_cache_create", "hcr_cache_append", "hcr_attn", "hcr_attn_blocks", "hcr_block_scores",
            "hcr_block_topk"} <= set(names)
    for n in names:
        assert hasattr(lib, n), n


def create(lib, **kw):
    a = dict(k=K, v=V, m=M, n=1000, kv=8, d=128, page=64)
    a.update(kw)
    h = ctypes.c_void_p()
    rc = lib.hcr_cache_create(a["k"], a["v"], a["m"], a["n"], a["kv"], a["d"], a["page"], ctypes.byref(h))
    return rc, h.value


@pytest.fixture()
def cache(lib):
    rc, h = create(lib)
    assert rc == hcr.HCR_OK
    yield h
    lib.hcr_cache_destroy(h)


@pytest.mark.parametrize("kw,rc", [
    (dict(k=None), hcr.HCR_EINVAL), (dict(v=None), hcr.HCR_EINVAL), (dict(n=0), hcr.HCR_EINVAL),
    (dict(kv=0), hcr.HCR_EINVAL), (dict(kv=-8), hcr.HCR_EINVAL), (dict(d=96), hcr.HCR_EINVAL),
    (dict(d=512), hcr.HCR_EINVAL), (dict(page=16), hcr.HCR_EINVAL), (dict(page=48), hcr.HCR_EINVAL),
    (dict(page=512), hcr.HCR_EINVAL), (dict(k=K + 8), hcr.HCR_EALIGN), (dict(m=M + 2), hcr.HCR_EALIGN),
    (dict(v=K + 4096), hcr.HCR_EALIAS), (dict(m=K), hcr.HCR_EALIAS), (dict(m=V + 16), hcr.HCR_EALIAS),
])
def test_create_rejects(lib, kw, rc):
    assert create(lib, **kw) == (rc, None)


def test_create_and_sizes(lib):
    assert lib.hcr_cache_create(K, V, M, 10, 1, 64, 32, None) == hcr.HCR_EINVAL
    rc, h = create(lib, m=None)
    assert rc == hcr.HCR_OK
    lib.hcr_cache_destroy(h)
    lib.hcr_cache_destroy(None)
    assert lib.hcr_cache_pages_bytes(10, 8, 128, 64) == 10 * 8 * 128 * 64 * 2
    assert lib.hcr_cache_pages_bytes(10, 8, 100, 64) == 0
    assert lib.hcr_cache_pages_bytes(1 << 20, 16, 256, 256) == (1 << 20) * 16 * 256 * 256 * 2


def batch(**kw):
    a = dict(n_seqs=4, n_tokens=8, max_tokens=3, max_ctx=5000, table_stride=100, q_start=STARTS, ctx_len=LENS,
             block_table=TABLE)
    a.update(kw)
    return paged.hcr_batch(*(a[n] for n, _ in paged.hcr_batch._fields_))


BAD_BATCHES = [
    (dict(n_seqs=-1), hcr.HCR_EINVAL), (dict(n_tokens=-1), hcr.HCR_EINVAL), (dict(max_tokens=-2), hcr.HCR_EINVAL),
    (dict(max_ctx=-1), hcr.HCR_EINVAL), (dict(table_stride=-1), hcr.HCR_EINVAL),
    (dict(max_ctx=6401), hcr.HCR_EINVAL),           # more positions than the table's 100 pages of 64
    (dict(q_start=None), hcr.HCR_EINVAL), (dict(ctx_len=None), hcr.HCR_EINVAL),
    (dict(block_table=None), hcr.HCR_EINVAL),
    (dict(q_start=STARTS + 2), hcr.HCR_EALIGN), (dict(ctx_len=LENS + 1), hcr.HCR_EALIGN),
    (dict(block_table=TABLE + 3), hcr.HCR_EALIGN),
    (dict(n_tokens=1 << 30), hcr.HCR_EINVAL),       # more rows than 32 bits hold
    (dict(n_seqs=1 << 30), hcr.HCR_EINVAL),
]


def attn(lib, h, b, heads=32, scale=0.1, q=Q, out_type=0, out=O, scratch=SC, bytes_=GB, sel=None, n_sel=0):
    if sel is None and n_sel == 0:
        return lib.hcr_attn(h, b and ctypes.byref(b), heads, scale, q, out_type, out, scratch, bytes_, None)
    return lib.hcr_attn_blocks(h, b and ctypes.byref(b), heads, scale, q, sel, n_sel, out_type, out, scratch, bytes_,
                               None)


BAD_ATTN = [
    (dict(heads=0), hcr.HCR_EINVAL), (dict(heads=12), hcr.HCR_EINVAL), (dict(heads=8 * 65), hcr.HCR_EINVAL),
    (dict(scale=float("nan")), hcr.HCR_EINVAL), (dict(scale=float("inf")), hcr.HCR_EINVAL),
    (dict(scale=-1e31), hcr.HCR_EINVAL), (dict(q=None), hcr.HCR_EINVAL), (dict(out=None), hcr.HCR_EINVAL),
    (dict(out_type=2), hcr.HCR_EINVAL), (dict(q=Q + 8), hcr.HCR_EALIGN), (dict(out=O + 4), hcr.HCR_EALIGN),
    (dict(scratch=SC + 128), hcr.HCR_EALIGN), (dict(scratch=None), hcr.HCR_ESCRATCH),
    (dict(bytes_=1024), hcr.HCR_ESCRATCH), (dict(out=Q), hcr.HCR_EALIAS), (dict(out=K + 4096), hcr.HCR_EALIAS),
    (dict(out=V), hcr.HCR_EALIAS), (dict(out=TABLE), hcr.HCR_EALIAS), (dict(out=SC), hcr.HCR_EALIAS),
    (dict(scratch=Q), hcr.HCR_EALIAS), (dict(scratch=M), hcr.HCR_EALIAS), (dict(scratch=LENS), hcr.HCR_EALIAS),
]


@pytest.mark.parametrize("kw,rc", BAD_ATTN)
def test_attn_rejects(lib, cache, kw, rc):
    assert attn(lib, cache, batch(), **kw) == rc
    assert attn(lib, cache, batch(), sel=SEL, n_sel=40, **kw) == rc


@pytest.mark.parametrize("kw,rc", BAD_BATCHES)
def test_batches_rejected(lib, cache, kw, rc):
    b = batch(**kw)
    assert attn(lib, cache, b) == rc
    assert attn(lib, cache, b, sel=SEL, n_sel=4) == rc
    assert append(lib, cache, b) == rc
    assert scores(lib, cache, b) == rc
    if "n_tokens" not in kw:  # its rows are kv heads: fewer
        assert topk(lib, cache, b) == rc


def test_attn_blocks_rejects(lib, cache):
    assert attn(lib, cache, batch(), sel=None, n_sel=3) == hcr.HCR_EINVAL
    assert attn(lib, cache, batch(), sel=SEL, n_sel=0) == hcr.HCR_EINVAL
    assert attn(lib, cache, batch(), sel=SEL, n_sel=-4) == hcr.HCR_EINVAL
    assert attn(lib, cache, batch(), sel=SEL, n_sel=1 << 26) == hcr.HCR_EINVAL
    assert attn(lib, cache, batch(), sel=SEL + 2, n_sel=3) == hcr.HCR_EALIGN
    assert attn(lib, cache, batch(), sel=O + 256, n_sel=3) == hcr.HCR_EALIAS
    assert attn(lib, cache, None) == hcr.HCR_EINVAL
    assert attn(lib, None, batch()) == hcr.HCR_EINVAL


def append(lib, h, b, heads=32, type_=0, q=(Q, 6144, 128), k=(Q + 16384, 6144, 128), v=(Q + 20480, 6144, 128),
           q_norm=WN, k_norm=WN, eps=1e-6, rope=R, rows=5000, dim=64, style=0, out=O):
    rows_of = [None if x is None else ctypes.byref(paged.hcr_rows(*x)) for x in (q, k, v)]
    return lib.hcr_cache_append(h, b and ctypes.byref(b), heads, type_, *rows_of, q_norm, k_norm, eps, rope, rows,
                                dim, style, out, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(heads=4), hcr.HCR_EINVAL), (dict(type_=3), hcr.HCR_EINVAL), (dict(q=None), hcr.HCR_EINVAL),
    (dict(k=(None, 6144, 128)), hcr.HCR_EINVAL), (dict(v=(Q, -6144, 128)), hcr.HCR_EINVAL),
    (dict(q=(Q, 1 << 47, 128)), hcr.HCR_EINVAL), (dict(k=(Q, 6144, 1 << 50)), hcr.HCR_EINVAL),
    (dict(v=(Q, (1 << 63) - 16, 128)), hcr.HCR_EINVAL), (dict(q=(Q, 6144, 1 << 46)), hcr.HCR_EINVAL),
    (dict(eps=-1.0), hcr.HCR_EINVAL), (dict(eps=float("nan")), hcr.HCR_EINVAL), (dict(eps=float("inf")), hcr.HCR_EINVAL),
    (dict(rope=None), hcr.HCR_EINVAL), (dict(dim=136), hcr.HCR_EINVAL), (dict(dim=24), hcr.HCR_EINVAL),
    (dict(dim=-8), hcr.HCR_EINVAL), (dict(rows=4999), hcr.HCR_EINVAL), (dict(style=2), hcr.HCR_EINVAL),
    (dict(out=None), hcr.HCR_EINVAL), (dict(out=O + 8), hcr.HCR_EALIGN), (dict(q_norm=WN + 4), hcr.HCR_EALIGN),
    (dict(q=(Q + 8, 6144, 128)), hcr.HCR_EALIGN), (dict(k=(Q, 6146, 128)), hcr.HCR_EALIGN),
    (dict(type_=1, v=(Q, 6144, 132)), hcr.HCR_EALIGN), (dict(rope=R + 4), hcr.HCR_EALIGN),
    (dict(out=Q + 256), hcr.HCR_EALIAS), (dict(out=K), hcr.HCR_EALIAS), (dict(out=M + 16), hcr.HCR_EALIAS),
    (dict(k=(V, 6144, 128)), hcr.HCR_EALIAS), (dict(rope=K), hcr.HCR_EALIAS), (dict(k_norm=V), hcr.HCR_EALIAS),
    (dict(out=STARTS), hcr.HCR_EALIAS), (dict(out=R), hcr.HCR_EALIAS), (dict(out=WN), hcr.HCR_EALIAS),
])
def test_append_rejects(lib, cache, kw, rc):
    assert append(lib, cache, batch(), **kw) == rc
    assert append(lib, None, batch()) == hcr.HCR_EINVAL
    assert append(lib, cache, None) == hcr.HCR_EINVAL


def test_append_rejects_a_table_inside_the_cache(lib, cache):
    assert append(lib, cache, batch(block_table=K)) == hcr.HCR_EALIAS
    assert append(lib, cache, batch(ctx_len=M + 64)) == hcr.HCR_EALIAS


def scores(lib, h, b, heads=32, q=Q, out=S, stride=100):
    return lib.hcr_block_scores(h, b and ctypes.byref(b), heads, q, out, stride, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(heads=7), hcr.HCR_EINVAL), (dict(q=None), hcr.HCR_EINVAL), (dict(out=None), hcr.HCR_EINVAL),
    (dict(stride=77), hcr.HCR_EINVAL), (dict(stride=-1), hcr.HCR_EINVAL), (dict(q=Q + 2), hcr.HCR_EALIGN),
    (dict(out=S + 4), hcr.HCR_EALIGN), (dict(out=Q), hcr.HCR_EALIAS), (dict(out=M), hcr.HCR_EALIAS),
    (dict(out=TABLE), hcr.HCR_EALIAS),
])
def test_scores_rejects(lib, cache, kw, rc):
    assert scores(lib, cache, batch(), **kw) == rc


def test_scores_rejects_a_cache_without_means(lib):
    rc, h = create(lib, m=None)
    assert rc == hcr.HCR_OK and scores(lib, h, batch()) == hcr.HCR_EINVAL
    lib.hcr_cache_destroy(h)


def topk(lib, h, b, s=S, stride=100, n_sel=8, n_first=1, n_last=2, sel=SEL):
    return lib.hcr_block_topk(h, b and ctypes.byref(b), s, stride, n_sel, n_first, n_last, sel, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n_sel=0), hcr.HCR_EINVAL), (dict(n_first=-1), hcr.HCR_EINVAL), (dict(n_last=0), hcr.HCR_EINVAL),
    (dict(n_sel=2), hcr.HCR_EINVAL), (dict(n_first=2 ** 31 - 1, n_last=2 ** 31 - 1), hcr.HCR_EINVAL),
    (dict(stride=77), hcr.HCR_EINVAL), (dict(s=None), hcr.HCR_EINVAL), (dict(sel=None), hcr.HCR_EINVAL),
    (dict(s=S + 8), hcr.HCR_EALIGN), (dict(sel=SEL + 1), hcr.HCR_EALIGN), (dict(sel=S + 64), hcr.HCR_EALIAS),
    (dict(sel=LENS), hcr.HCR_EALIAS),
])
def test_topk_rejects(lib, cache, kw, rc):
    assert topk(lib, cache, batch(), **kw) == rc


@pytest.mark.parametrize("sel", [K, V + 4096, M + 64, K - 4, M + 1000 * 8 * 128 * 2 - 4])
def test_topk_rejects_a_list_inside_the_cache(lib, cache, sel):
    assert topk(lib, cache, batch(), sel=sel) == hcr.HCR_EALIAS


@pytest.mark.parametrize("n_sel", [(1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1])
def test_topk_rejects_lists_past_its_counters(lib, n_sel):
    """A lane steps through a list in 32 bits, 1,024 entries at a time."""
    rc, h = create(lib, kv=1)
    b = batch(n_seqs=1, n_tokens=1, max_tokens=1)
    assert rc == hcr.HCR_OK
    assert topk(lib, h, b, n_sel=n_sel, sel=200 * GB) == hcr.HCR_EINVAL
    lib.hcr_cache_destroy(h)


def test_empty_calls_do_nothing(lib, cache):
    for kw in (dict(n_seqs=0), dict(n_tokens=0), dict(max_tokens=0)):
        b = batch(q_start=None, ctx_len=None, block_table=None, **kw)
        assert attn(lib, cache, b, q=None, out=None, scratch=None, bytes_=0) == hcr.HCR_OK
        assert append(lib, cache, b, q=None, k=None, v=None, out=None) == hcr.HCR_OK
        assert scores(lib, cache, b, q=None, out=None) == hcr.HCR_OK
        assert topk(lib, cache, b, s=None, sel=None) == hcr.HCR_OK
    # no complete page to score before the only one
    assert scores(lib, cache, batch(max_ctx=64), q=None, out=None, stride=0) == hcr.HCR_OK


def test_scratch_sizes(lib, cache):
    b = batch(n_seqs=1, n_tokens=2, max_tokens=2, max_ctx=6400)
    n = lib.hcr_attn_scratch_bytes(cache, ctypes.byref(b), 32, 0)
    assert n > 0 and n % 256 == 0
    assert lib.hcr_attn_scratch_bytes(cache, ctypes.byref(b), 31, 0) == 0
    assert lib.hcr_attn_scratch_bytes(None, ctypes.byref(b), 32, 0) == 0
    small = batch(n_seqs=1, max_ctx=64)
    assert lib.hcr_attn_scratch_bytes(cache, ctypes.byref(small), 32, 0) == 0
    assert attn(lib, cache, b, bytes_=n - 1) == hcr.HCR_ESCRATCH


def test_binding_rejects_what_it_can_see():
    """Shapes, types and devices are refused in Python before any pointer is taken."""
    x = torch.zeros(2, 8, 8, 32, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        paged.PagedCache(x, x)  # not on a device
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        paged.Batch(i, i, i, 1, 1)
    with pytest.raises(ValueError):
        paged.Batch(i.long(), i, i, 1, 1)


def _binding_tensor(at, *shape, dtype=torch.bfloat16):
    """What the binding asks of a device tensor; the address is made up."""
    return types.SimpleNamespace(dtype=dtype, shape=torch.Size(shape), is_cuda=True, device=torch.device("cuda:0"),
                                 is_contiguous=lambda: True, dim=lambda: len(shape), data_ptr=lambda: at)


def test_a_binding_cache_keeps_its_pages():
    """The handle holds the pages' addresses: another tensor in their place would leave it with memory let go."""
    ensure_built()
    k = _binding_tensor(K, 10, 2, 8, 32, 8)
    cache = paged.PagedCache(k, _binding_tensor(V, 10, 2, 4, 64, 8), _binding_tensor(M, 10, 2, 64))
    handle = cache.handle
    for name in ("k_pages", "v_pages", "k_means", "handle", "page", "device", "kv_heads", "head_dim", "n_pages"):
        with pytest.raises(AttributeError):
            setattr(cache, name, None)
    cache.layer = 3  # an attribute of the caller's own
    del cache.layer
    for name in ("k_pages", "v_pages", "k_means", "handle"):
        with pytest.raises(AttributeError):
            delattr(cache, name)
    assert cache.k_pages is k and cache.handle == handle


def _binding_batch(**bounds):
    i32 = torch.int32
    return paged.Batch(_binding_tensor(STARTS, 5, dtype=i32), _binding_tensor(LENS, 4, dtype=i32),
                       _binding_tensor(TABLE, 4, 100, dtype=i32), **{"max_tokens": 3, "max_ctx": 5000, **bounds})


def test_a_binding_batch_keeps_its_tensors():
    """Calls keep the addresses: a tensor deleted from the batch would be let go under them."""
    b = _binding_batch()
    b._of(8)
    for name in ("q_start", "ctx_len", "block_table", "max_ctx", "_by_rows"):
        with pytest.raises(AttributeError):
            delattr(b, name)
    with pytest.raises(AttributeError):
        b.max_ctx = 7


@pytest.mark.parametrize("bounds", [dict(max_ctx=2 ** 31), dict(max_ctx=2 ** 32 + 5000), dict(max_tokens=2 ** 32 + 3),
                                    dict(max_tokens=2 ** 63), dict(max_ctx=-1)])
def test_a_binding_batch_refuses_bounds_past_32_bits(bounds):
    """ctypes would cut them: 2^32 + 5,000 positions to 5,000."""
    with pytest.raises(ValueError):
        _binding_batch(**bounds)
    assert _binding_batch(max_ctx=2 ** 31 - 1).max_ctx == 2 ** 31 - 1


@pytest.mark.parametrize("counts", [dict(n_first=2 ** 32 + 1), dict(n_last=2 ** 32 + 2), dict(n_first=-2 ** 32),
                                    dict(n_last=2 ** 31)])
def test_binding_topk_refuses_counts_past_32_bits(counts):
    ensure_built()
    cache = paged.PagedCache(_binding_tensor(K, 10, 2, 8, 32, 8), _binding_tensor(V, 10, 2, 4, 64, 8))
    scores = _binding_tensor(S, 8, 2, 200, dtype=torch.float32)
    sel = _binding_tensor(SEL, 8, 2, 9, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.block_topk(_binding_batch(), scores, 9, **counts, sel=sel)


def test_a_binding_copy_has_a_handle_of_its_own():
    """Two caches that destroy one handle would free it twice; a batch's copy holds its own tensors' addresses."""
    ensure_built()
    code = ("import copy, sys\nimport torch\nsys.path.insert(0, '.')\nfrom bf16_hyper_connection_amd import paged\n"
            "from tests.test_paged_abi import K, M, V, _binding_batch, _binding_tensor\n"
            "c = paged.PagedCache(_binding_tensor(K, 10, 2, 8, 32, 8), _binding_tensor(V, 10, 2, 4, 64, 8),\n"
            "                     _binding_tensor(M, 10, 2, 64))\n"
            "d = copy.copy(c)\n"
            "assert d.handle != c.handle and d.k_pages is c.k_pages and d.k_means is c.k_means and d.page == 32\n"
            "del c, d\n"
            "b = _binding_batch()\nb._of(8)\nx = copy.copy(b)\n"
            "assert x.q_start is b.q_start and x.max_ctx == b.max_ctx and not x._by_rows\n"
            "print('fine', flush=True)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_a_binding_cache_may_be_derived_from():
    ensure_built()

    class Layer(paged.PagedCache):
        def __init__(self, number, *pages):
            super().__init__(*pages)
            self.number = number
    layer = Layer(7, _binding_tensor(K, 10, 2, 8, 32, 8), _binding_tensor(V, 10, 2, 4, 64, 8))
    assert layer.number == 7 and layer.k_means is None


@pytest.fixture(scope="module")
def sanitized(tmp_path_factory):
    cxx = next((c for c in ("g++", "c++") if shutil.which(c)), None)
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("paged") / "libpaged_asan.so")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-shared", "-fPIC", "-Wall", "-Werror", "-D__host__=", "-D__device__=",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "hcr_paged_api.cpp"),
           os.path.join(ROOT, "tests", "asan", "paged_stubs.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return out, subprocess.run([cxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()


def _under_asan(sanitized, args):
    lib_path, libasan = sanitized
    env = dict(os.environ, PAGED_ABI_LIB=lib_path, LD_PRELOAD=libasan,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, *args], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr
    return r.stdout


@pytest.mark.skipif(bool(SANITIZED), reason="the child itself")
def test_checks_clean_under_asan_and_ubsan(sanitized):
    ensure_built()
    out = _under_asan(sanitized, ["-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                                  "tests/test_paged_abi.py", "-k", "not asan and not binding and not index"])
    assert " passed" in out


@pytest.mark.skipif(bool(SANITIZED), reason="the parent's")
def test_index_arithmetic_stays_in_bounds(sanitized):
    """seq_of, page_or_none, the page orders and the attention plan over odd values (tests/asan/paged_stubs.cpp)."""
    out = _under_asan(sanitized, ["-c", "import ctypes, os; L = ctypes.CDLL(os.environ['PAGED_ABI_LIB'])\n"
                                        "L.paged_index_checks.restype = ctypes.c_char_p\n"
                                        "print(L.paged_index_checks().decode())"])
    assert out.strip().endswith("ok"), out


@pytest.mark.skipif(bool(SANITIZED), reason="the parent's")
def test_index_long_runs_pass_a_waves_lanes(sanitized):
    """The GPU tests' scenes of long runs do what they are for under the present plan."""
    from tests import paged_util as pu
    calls = []
    for name, (kv, heads, D, page, windows, n_sel) in sorted(pu.LONG_RUNS.items()):
        tiles = [max(-(-c // 32), 1) for _, c in windows]
        calls.append((D, kv, page, heads, len(windows), sum(t for t, _ in windows), max(t for t, _ in windows),
                      max(c for _, c in windows), n_sel, sum(tiles), max(tiles)))
    out = _under_asan(sanitized, ["-c", "import ctypes, os; L = ctypes.CDLL(os.environ['PAGED_ABI_LIB'])\n"
                                        f"print([L.paged_run_pages(*c) for c in {calls}])"])
    runs = [int(x) for x in out.strip().strip("[]").split(",")]
    assert len(runs) == len(calls) and all(r > 64 for r in runs), runs
