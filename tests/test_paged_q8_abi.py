"""The C ABI of codes, read-back and windows (include/hcr_paged_q8.h) on the host: exports, refusals before any HIP call,
index arithmetic.  No GPU is used: the device addresses are made up, and every call here is one that the checks reject
or an empty one.

The same calls run against a build of the host code under AddressSanitizer and UndefinedBehaviorSanitizer
(PAGED_Q8_ABI_LIB), where the launchers are stand-ins."""

import copy
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
SANITIZED = os.environ.get("PAGED_Q8_ABI_LIB")

GB = 1 << 30
K, V, KS, VS, M, Q, O, O2, SC, SEL = (i * 4 * GB for i in range(16, 26))
STARTS, LENS, TABLE, R = (i * 4 * GB for i in range(30, 34))


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hcr_paged_q8.h")).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(hcr_[a-z_0-9]+)\s*\(", text)))


@pytest.fixture(scope="module")
def lib():
    if SANITIZED:
        L = ctypes.CDLL(SANITIZED)
        real = paged.lib() if os.path.exists(hcr.LIB_PATH) else None
        for n in declared() + ["hcr_cache_create", "hcr_cache_destroy", "hcr_cache_append", "hcr_attn", "hcr_attn_blocks",
                               "hcr_attn_scratch_bytes", "hcr_block_scores", "hcr_block_topk"]:
            f = getattr(L, n)
            if real is not None:
                f.restype, f.argtypes = getattr(real, n).restype, getattr(real, n).argtypes
        return L
    ensure_built()
    return paged.lib()


def test_exports_every_declared_symbol(lib):
    names = declared()
    assert names == ["hcr_attn_window", "hcr_attn_window_scratch_bytes", "hcr_cache_create_q8",
                     "hcr_cache_pages_bytes_q8", "hcr_cache_read"]
    for n in names:
        assert hasattr(lib, n), n


def create(lib, **kw):
    a = dict(k=K, v=V, ks=KS, vs=VS, m=M, code=2, n=1000, kv=8, d=128, page=64)
    a.update(kw)
    h = ctypes.c_void_p()
    rc = lib.hcr_cache_create_q8(a["k"], a["v"], a["ks"], a["vs"], a["m"], a["code"], a["n"], a["kv"], a["d"], a["page"],
                                 ctypes.byref(h))
    return rc, h.value


@pytest.fixture(params=[2, 3])
def cache(lib, request):
    rc, h = create(lib, code=request.param)
    assert rc == hcr.HCR_OK
    yield h
    lib.hcr_cache_destroy(h)


@pytest.fixture()
def plain(lib):
    h = ctypes.c_void_p()
    assert lib.hcr_cache_create(K, V, M, 1000, 8, 128, 64, ctypes.byref(h)) == hcr.HCR_OK
    yield h.value
    lib.hcr_cache_destroy(h.value)


@pytest.mark.parametrize("kw,rc", [
    (dict(k=None), hcr.HCR_EINVAL), (dict(v=None), hcr.HCR_EINVAL), (dict(ks=None), hcr.HCR_EINVAL),
    (dict(vs=None), hcr.HCR_EINVAL), (dict(code=0), hcr.HCR_EINVAL), (dict(code=1), hcr.HCR_EINVAL),
    (dict(code=4), hcr.HCR_EINVAL), (dict(code=-2), hcr.HCR_EINVAL), (dict(n=0), hcr.HCR_EINVAL),
    (dict(kv=0), hcr.HCR_EINVAL), (dict(kv=5000), hcr.HCR_EINVAL), (dict(d=96), hcr.HCR_EINVAL),
    (dict(page=32), hcr.HCR_EINVAL), (dict(page=512), hcr.HCR_EINVAL), (dict(k=K + 8), hcr.HCR_EALIGN),
    (dict(ks=KS + 4), hcr.HCR_EALIGN), (dict(vs=VS + 8), hcr.HCR_EALIGN), (dict(m=M + 2), hcr.HCR_EALIGN),
    (dict(v=K + 4096), hcr.HCR_EALIAS), (dict(ks=K), hcr.HCR_EALIAS), (dict(vs=KS + 16), hcr.HCR_EALIAS),
    (dict(m=VS), hcr.HCR_EALIAS), (dict(vs=V + 1000 * 8 * 128 * 64 - 16), hcr.HCR_EALIAS),
    (dict(m=KS + 1000 * 8 * 64 * 4 - 16), hcr.HCR_EALIAS),
])
def test_create_rejects(lib, kw, rc):
    assert create(lib, **kw) == (rc, None)


def test_create_and_sizes(lib):
    assert lib.hcr_cache_create_q8(K, V, KS, VS, M, 2, 10, 1, 64, 64, None) == hcr.HCR_EINVAL
    # the arrays end where a byte a value says
    rc, h = create(lib, m=None, v=K + 1000 * 8 * 128 * 64, ks=V, vs=V + 1000 * 8 * 64 * 4)
    assert rc == hcr.HCR_OK
    lib.hcr_cache_destroy(h)
    assert lib.hcr_cache_pages_bytes_q8(10, 8, 128, 64) == 10 * 8 * 128 * 64
    assert lib.hcr_cache_pages_bytes_q8(10, 8, 128, 32) == 0
    assert lib.hcr_cache_pages_bytes_q8(10, 8, 100, 64) == 0
    assert lib.hcr_cache_pages_bytes_q8(1 << 20, 16, 256, 256) == (1 << 20) * 16 * 256 * 256


def batch(**kw):
    a = dict(n_seqs=4, n_tokens=8, max_tokens=3, max_ctx=5000, table_stride=100, q_start=STARTS, ctx_len=LENS,
             block_table=TABLE)
    a.update(kw)
    return paged.hcr_batch(*(a[n] for n, _ in paged.hcr_batch._fields_))


def attn(lib, h, b, heads=32, scale=0.1, q=Q, window=4500, n_first=4, out_type=0, out=O, scratch=SC, bytes_=GB):
    return lib.hcr_attn_window(h, b and ctypes.byref(b), heads, scale, q, window, n_first, out_type, out, scratch, bytes_,
                               None)


def read(lib, h, b, out_type=1, k=O, v=O2):
    return lib.hcr_cache_read(h, b and ctypes.byref(b), out_type, k, v, None)


BAD_BATCHES = [
    (dict(n_seqs=-1), hcr.HCR_EINVAL), (dict(n_tokens=-1), hcr.HCR_EINVAL), (dict(max_tokens=-2), hcr.HCR_EINVAL),
    (dict(max_ctx=-1), hcr.HCR_EINVAL), (dict(table_stride=-1), hcr.HCR_EINVAL), (dict(max_ctx=6401), hcr.HCR_EINVAL),
    (dict(q_start=None), hcr.HCR_EINVAL), (dict(ctx_len=None), hcr.HCR_EINVAL), (dict(block_table=None), hcr.HCR_EINVAL),
    (dict(q_start=STARTS + 2), hcr.HCR_EALIGN), (dict(ctx_len=LENS + 1), hcr.HCR_EALIGN),
    (dict(block_table=TABLE + 3), hcr.HCR_EALIGN), (dict(n_tokens=1 << 30), hcr.HCR_EINVAL),
    (dict(n_seqs=1 << 30), hcr.HCR_EINVAL),
]


@pytest.mark.parametrize("kw,rc", BAD_BATCHES)
def test_batches_rejected(lib, cache, plain, kw, rc):
    for h in (cache, plain):
        assert attn(lib, h, batch(**kw)) == rc
        assert read(lib, h, batch(**kw)) == rc
    assert lib.hcr_attn(cache, ctypes.byref(batch(**kw)), 32, 0.1, Q, 0, O, SC, GB, None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(window=0), hcr.HCR_EINVAL), (dict(window=-5), hcr.HCR_EINVAL), (dict(n_first=-1), hcr.HCR_EINVAL),
    (dict(heads=0), hcr.HCR_EINVAL), (dict(heads=12), hcr.HCR_EINVAL), (dict(heads=8 * 65), hcr.HCR_EINVAL),
    (dict(scale=float("nan")), hcr.HCR_EINVAL), (dict(scale=1e31), hcr.HCR_EINVAL), (dict(q=None), hcr.HCR_EINVAL),
    (dict(out=None), hcr.HCR_EINVAL), (dict(out_type=2), hcr.HCR_EINVAL), (dict(out_type=3), hcr.HCR_EINVAL),
    (dict(q=Q + 8), hcr.HCR_EALIGN), (dict(out=O + 4), hcr.HCR_EALIGN), (dict(scratch=SC + 128), hcr.HCR_EALIGN),
    (dict(scratch=None), hcr.HCR_ESCRATCH), (dict(bytes_=1024), hcr.HCR_ESCRATCH), (dict(out=Q), hcr.HCR_EALIAS),
    (dict(out=K + 4096), hcr.HCR_EALIAS), (dict(out=V), hcr.HCR_EALIAS), (dict(out=TABLE), hcr.HCR_EALIAS),
    (dict(out=SC), hcr.HCR_EALIAS), (dict(scratch=M), hcr.HCR_EALIAS), (dict(scratch=LENS), hcr.HCR_EALIAS),
])
def test_window_rejects(lib, cache, plain, kw, rc):
    assert attn(lib, cache, batch(), **kw) == rc
    assert attn(lib, plain, batch(), **kw) == rc
    assert attn(lib, None, batch()) == hcr.HCR_EINVAL and attn(lib, cache, None) == hcr.HCR_EINVAL


@pytest.mark.parametrize("at", [KS, KS + 1000 * 8 * 64 * 4 - 16, VS])
def test_outputs_inside_the_scales_are_rejected(lib, cache, plain, at):
    assert attn(lib, cache, batch(), out=at) == hcr.HCR_EALIAS
    assert read(lib, cache, batch(), v=at) == hcr.HCR_EALIAS
    b = batch()
    assert lib.hcr_attn(cache, ctypes.byref(b), 32, 0.1, Q, 0, at, SC, GB, None) == hcr.HCR_EALIAS
    assert lib.hcr_attn_blocks(cache, ctypes.byref(b), 32, 0.1, Q, SEL, 9, 0, at, SC, GB, None) == hcr.HCR_EALIAS
    assert lib.hcr_block_scores(cache, ctypes.byref(b), 32, Q, at, 100, None) == hcr.HCR_EALIAS
    assert lib.hcr_block_topk(cache, ctypes.byref(b), R, 100, 8, 1, 2, at, None) == hcr.HCR_EALIAS
    rows = [ctypes.byref(paged.hcr_rows(x, 6144, 128)) for x in (Q, Q + 16384, Q + 20480)]

    def append(q_out=O, norm=None, table=TABLE):
        return lib.hcr_cache_append(cache, ctypes.byref(batch(block_table=table)), 32, 0, *rows, norm, None, 1e-6, None, 0, 0,
                                    0, q_out, None)
    assert append(q_out=at) == append(norm=at) == append(table=at) == hcr.HCR_EALIAS


@pytest.mark.parametrize("kw,rc", [
    (dict(out_type=2), hcr.HCR_EINVAL), (dict(out_type=-1), hcr.HCR_EINVAL), (dict(k=None, v=None), hcr.HCR_EINVAL),
    (dict(k=O + 8), hcr.HCR_EALIGN), (dict(v=O2 + 4), hcr.HCR_EALIGN), (dict(v=O), hcr.HCR_EALIAS),
    (dict(v=O + 8 * 8 * 128 * 2 - 16), hcr.HCR_EALIAS), (dict(k=K), hcr.HCR_EALIAS), (dict(v=M), hcr.HCR_EALIAS),
    (dict(k=STARTS), hcr.HCR_EALIAS), (dict(v=TABLE + 16), hcr.HCR_EALIAS),
])
def test_read_rejects(lib, cache, plain, kw, rc):
    assert read(lib, cache, batch(), **kw) == rc
    assert read(lib, plain, batch(), **kw) == rc
    assert read(lib, None, batch()) == hcr.HCR_EINVAL and read(lib, cache, None) == hcr.HCR_EINVAL


def test_empty_calls_do_nothing(lib, cache):
    for kw in (dict(n_seqs=0), dict(n_tokens=0), dict(max_tokens=0)):
        b = batch(q_start=None, ctx_len=None, block_table=None, **kw)
        assert attn(lib, cache, b, q=None, out=None, scratch=None, bytes_=0) == hcr.HCR_OK
        assert read(lib, cache, b, k=None, v=None) == hcr.HCR_OK


def test_scratch_sizes(lib, cache, plain):
    b = batch(n_seqs=1, n_tokens=2, max_tokens=2, max_ctx=6400)
    for h in (cache, plain):
        n = lib.hcr_attn_window_scratch_bytes(h, ctypes.byref(b), 32, 5000, 4)
        assert n > 0 and n % 256 == 0 and attn(lib, h, b, window=5000, bytes_=n - 1) == hcr.HCR_ESCRATCH
        # a window longer than any sequence needs what the longest does
        assert lib.hcr_attn_window_scratch_bytes(h, ctypes.byref(b), 32, 2 ** 31 - 1, 2 ** 31 - 1) == \
            lib.hcr_attn_window_scratch_bytes(h, ctypes.byref(b), 32, 6400, 6400)
        for bad in ((31, 5000, 4), (32, 0, 4), (32, 5000, -1)):
            assert lib.hcr_attn_window_scratch_bytes(h, ctypes.byref(b), *bad) == 0
    assert lib.hcr_attn_window_scratch_bytes(None, ctypes.byref(b), 32, 5000, 4) == 0
    assert lib.hcr_attn_scratch_bytes(cache, ctypes.byref(b), 32, 0) > 0


def _tensor(at, *shape, dtype=torch.int8):
    """What the binding asks of a device tensor; the address is made up."""
    return types.SimpleNamespace(dtype=dtype, shape=torch.Size(shape), is_cuda=True, device=torch.device("cuda:0"),
                                 is_contiguous=lambda: True, dim=lambda: len(shape), data_ptr=lambda: at)


def _cache(dtype=torch.int8, **kw):
    a = dict(k_pages=_tensor(K, 10, 2, 4, 64, 16, dtype=dtype), v_pages=_tensor(V, 10, 2, 4, 64, 16, dtype=dtype),
             k_means=_tensor(M, 10, 2, 64, dtype=torch.bfloat16), k_scales=_tensor(KS, 10, 2, 64, dtype=torch.float32),
             v_scales=_tensor(VS, 10, 2, 64, dtype=torch.float32))
    a.update(kw)
    return paged.PagedCache(**a)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_binding_makes_a_cache_of_codes(dtype):
    ensure_built()
    c = _cache(dtype)
    assert (c.n_pages, c.kv_heads, c.head_dim, c.page) == (10, 2, 64, 64)
    other = copy.copy(c)
    assert other.handle != c.handle and other.k_scales is c.k_scales and other.v_scales is c.v_scales
    for name in ("k_scales", "v_scales", "k_pages"):
        with pytest.raises(AttributeError):
            setattr(c, name, None)
    assert _cache(dtype, k_means=None).k_means is None


@pytest.mark.parametrize("kw", [
    dict(k_scales=None), dict(v_scales=None), dict(v_pages=_tensor(V, 10, 2, 4, 64, 16, dtype=torch.uint8)),
    dict(k_pages=_tensor(K, 10, 2, 8, 64, 8)), dict(v_pages=_tensor(V, 10, 2, 8, 64, 8)),
    dict(k_scales=_tensor(KS, 10, 2, 32, dtype=torch.float32)), dict(v_scales=_tensor(VS, 10, 2, 64, dtype=torch.bfloat16)),
    dict(k_pages=_tensor(K, 10, 2, 8, 64, 8, dtype=torch.bfloat16)), dict(k_means=_tensor(M, 10, 2, 32, dtype=torch.bfloat16)),
    dict(k_pages=_tensor(K, 10, 2, 4, 64, 16, dtype=torch.float8_e5m2), v_pages=_tensor(V, 10, 2, 4, 64, 16, dtype=torch.float8_e5m2)),
])
def test_binding_refuses_what_is_no_cache(kw):
    ensure_built()
    with pytest.raises(ValueError):
        _cache(**kw)


def test_binding_refuses_windows_and_rows_past_32_bits():
    """ctypes would cut them: a window of 2^32 + 7 to 7."""
    ensure_built()
    c, i32 = _cache(), torch.int32
    b = paged.Batch(_tensor(STARTS, 5, dtype=i32), _tensor(LENS, 4, dtype=i32), _tensor(TABLE, 4, 100, dtype=i32), 3, 5000)
    q = _tensor(Q, 4, 8, 64, dtype=torch.bfloat16)
    for window, n_first in ((2 ** 32 + 7, 0), (7, 2 ** 32), (2 ** 31, 0), (-2 ** 32, 0)):
        with pytest.raises(ValueError):
            c.attend_window(b, q, window, n_first)
    for n in (-1, 2 ** 32 + 4, 2 ** 31):
        with pytest.raises(ValueError):
            c.read(b, n)
    with pytest.raises(ValueError):
        c.read(b, 4, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        paged.PagedCache.allocate(4, 2, 64, dtype=torch.float16)


@pytest.fixture(scope="module")
def sanitized(tmp_path_factory):
    cxx = next((c for c in ("g++", "c++") if shutil.which(c)), None)
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("paged_q8") / "libpaged_q8_asan.so")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-shared", "-fPIC", "-Wall", "-Werror", "-D__host__=", "-D__device__=",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "hcr_paged_api.cpp"),
           os.path.join(CSRC, "hcr_paged_q8_api.cpp"), os.path.join(ROOT, "tests", "asan", "paged_stubs.cpp"),
           os.path.join(ROOT, "tests", "asan", "paged_q8_stubs.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return out, subprocess.run([cxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()


def _under_asan(sanitized, args):
    lib_path, libasan = sanitized
    env = dict(os.environ, PAGED_Q8_ABI_LIB=lib_path, LD_PRELOAD=libasan,
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
                                  "tests/test_paged_q8_abi.py", "-k", "not asan and not binding and not index"])
    assert " passed" in out


@pytest.mark.skipif(bool(SANITIZED), reason="the child itself")
def test_index_arithmetic(sanitized):
    """The orders of codes, a tile's operands, the tiles of a window, plans and parts of a read
    (tests/asan/paged_q8_stubs.cpp)."""
    code = ("import ctypes, sys; L = ctypes.CDLL(sys.argv[1]); L.paged_q8_index_checks.restype = ctypes.c_char_p; "
            "r = L.paged_q8_index_checks().decode(); print(r); sys.exit(r != 'ok')")
    assert _under_asan(sanitized, ["-c", code, sanitized[0]]).strip() == "ok"
