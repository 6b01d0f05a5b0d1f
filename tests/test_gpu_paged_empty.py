"""Requests without keys whose queries hold anything, as idle rows of a padded or captured batch do: output 0 and
log-sum-exp -inf, and their neighbours' results keep their bits."""
import math

import pytest
import torch

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DS = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 16, BF16, 16), (DS, 64, BF16, 64), (DS, 128, BF16, 64), (DS, 130, BF16, 8),
                                                   (DS, 16, BF16, 5), (DS, 16, F32, 16), (TINY, 4, F32, 7)])
def test_empty_requests_with_any_queries(dims, heads, dtype, page, junk):
    d = mla.dims(heads, **dims)
    g = ref.generator(heads + page)
    lens = [0, 3 * page + 1, 0, 1, 2 * page, 0]
    c, k, table = ref.cache(g, d, dtype, lens, page)
    table[4, :2] = -1                                # a request whose pages are all bad
    q, r, w = ref.queries(g, d, dtype, len(lens))
    dev = [x.cuda() for x in (q, r, c, k, table, torch.tensor(lens, dtype=torch.int32), w)]
    want = mla.paged_decode(d, *dev)
    idle = [0, 2, 4, 5]
    q2, r2 = dev[0].clone(), dev[1].clone()
    q2[idle], r2[idle] = junk, junk
    q2[2, :, 1:], r2[2, :, ::2] = 0.5, 0.5           # some of the elements only
    out, lse = mla.paged_decode(d, q2, r2, *dev[2:])
    assert bool((out[idle] == 0).all()) and bool((lse[idle] == -math.inf).all())
    for b in (1, 3):
        assert torch.equal(out[b], want[0][b]) and torch.equal(lse[b], want[1][b])
    assert bool(torch.isfinite(out).all()) and mla.mla_check_device_error() == 0
