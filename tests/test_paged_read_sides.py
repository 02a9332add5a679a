"""The binding's read-back of keys or values alone."""

import pytest
import torch

from bf16_hyper_connection_amd import paged
from tests import paged_codes_util as cu
from tests import paged_util as pu
from tests.libhcr_util import ensure_built
from tests.test_paged_q8_abi import LENS, O, STARTS, TABLE, _cache, _tensor


def test_refuses_no_side_and_outputs_of_a_side_that_is_not_read():
    ensure_built()
    c, i32 = _cache(), torch.int32
    b = paged.Batch(_tensor(STARTS, 5, dtype=i32), _tensor(LENS, 4, dtype=i32), _tensor(TABLE, 4, 100, dtype=i32), 3, 5000)
    out = _tensor(O, 4, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(keys=False, values=False), dict(keys=False, k_out=out), dict(values=False, v_out=out),
               dict(keys=False, values=False, k_out=out)):
        with pytest.raises(ValueError):
            c.read(b, 4, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", cu.KINDS + ["bf16"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_one_side(kind, out_dtype):
    ensure_built()
    s = cu.scene(kind, 170, 2, 128, 64, [(70, 70), (3, 200)])
    cache, batch = cu.dev_cache(s), pu.dev_batch(s)
    k, v = cache.read(batch, 73, out_dtype)
    only, none = cache.read(batch, 73, out_dtype, values=False)
    assert none is None and torch.equal(only, k)
    none, only = cache.read(batch, 73, out_dtype, keys=False)
    assert none is None and torch.equal(only, v)
    given = torch.zeros_like(v)
    assert cache.read(batch, 73, v_out=given, keys=False) == (None, given) and torch.equal(given, v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    only, none = cache.read(batch, 73, out_dtype, stream=side.cuda_stream, values=False)
    side.synchronize()
    assert none is None and torch.equal(only, k)
