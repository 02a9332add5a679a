"""hcr_cache_read's bound on its launch: work-groups of 256 threads, one for 64 positions of a sequence and kv head, keys and
values together, as many as 32 bits of threads hold.  On the
host the launcher is a stand-in that returns HCR_EHIP."""

import pytest
import torch

from bf16_hyper_connection_amd import hcr, paged
from tests import paged_codes_util as cu
from tests import paged_util as pu
from tests.libhcr_util import ensure_built
from tests.test_paged_pairs import sanitized  # noqa: F401  (the host code with stand-ins for the launchers)


def read(sanitized, n_seqs, max_tokens, kv):
    return int(sanitized(
        "import sys; sys.path.insert(0, '.')\n"
        "from bf16_hyper_connection_amd import paged\n"
        "GB = 1 << 30\n"
        "h = ctypes.c_void_p()\n"
        "V, I, P = ctypes.c_void_p, ctypes.c_int, ctypes.byref\n"
        f"assert L.hcr_cache_create(V(1024 * GB), V(2048 * GB), None, 1000, {kv}, 64, 64, P(h)) == 0\n"
        f"b = paged.hcr_batch({n_seqs}, {max_tokens}, {max_tokens}, 1 << 20, 1 << 15, 8 * GB, 16 * GB, 3200 * GB)\n"
        "print(L.hcr_cache_read(h, P(b), 1, V(4096 * GB), V(6144 * GB), None))\n"))


def test_the_launch_takes_what_32_bits_hold(sanitized):  # noqa: F811
    # 1,000 sequences of up to 100,000 tokens: 1,564 parts of 64, 8 heads: 12.5 of 16.8 million work-groups
    assert read(sanitized, 1000, 100000, 8) == hcr.HCR_EHIP
    # the last number of sequences that fits, and the next
    tokens = 1024 * 64 - 62
    assert -(-(tokens - 1) // 64) + 1 == 1025
    assert read(sanitized, 16777215 // (1025 * 8), tokens, 8) == hcr.HCR_EHIP
    assert read(sanitized, 16777215 // (1025 * 8) + 1, tokens, 8) == hcr.HCR_EINVAL


@pytest.mark.gpu
def test_loose_bounds_past_half_of_that():
    """12.5 million work-groups, of which 1,000 sequences of a few tokens need some thousand."""
    ensure_built()
    windows = [(i % 5, 3 * (i % 60)) for i in range(1000)]
    s = cu.scene("int8", 150, 8, 64, 64, windows, table_extra=1600)
    cache = cu.dev_cache(s)
    want = cache.read(pu.dev_batch(s), s.n_tokens)
    loose = pu.dev_batch(s, max_tokens=100000, max_ctx=100000)
    out = torch.full((100000, 8, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    k, v = cache.read(loose, 100000, k_out=out, v_out=torch.full_like(out, 6.0))
    torch.cuda.synchronize()
    assert torch.equal(k[:s.n_tokens], want[0]) and torch.equal(v[:s.n_tokens], want[1])
    assert torch.all(k[s.n_tokens:] == 5.0) and torch.all(v[s.n_tokens:] == 6.0)
