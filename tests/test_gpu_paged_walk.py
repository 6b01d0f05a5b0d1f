"""The paged decode's walk over parts of one to three key tiles: several of each to a cluster, whose queries and
keys take turns in the same shared memory."""
import pytest
import torch

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

ONE, TWO, THREE = (1, 64), (65, 128), (129, 192)   # keys of a request of that many tiles


@pytest.mark.parametrize("heads,batch,page,kinds", [
    (128, 330, 64, [ONE]), (128, 300, 8, [ONE, ONE, TWO]), (128, 260, 16, [ONE, TWO, ONE, THREE]), (130, 150, 64, [ONE]),
    (65, 250, 32, [THREE, ONE]), (16, 330, 16, [ONE]), (64, 260, 64, [ONE, ONE, ONE, TWO]), (40, 200, 24, [ONE, THREE, ONE]),
])
def test_many_short_requests(heads, batch, page, kinds):
    d = mla.dims(heads, 512, 128, 64, 128)
    g = ref.generator(batch + heads)
    lens = []
    for b in range(batch):
        lo, hi = kinds[b % len(kinds)]
        lens.append(int(torch.randint(lo, hi + 1, (1,), generator=g)))
    c, k, table = ref.cache(g, d, BF16, lens, page)
    q, r, w = ref.queries(g, d, BF16, batch)
    t = (q, r, c, k, table, torch.tensor(lens, dtype=torch.int32), w)
    dev = [x.cuda() for x in t]
    ws = mla.paged_decode_workspace(d, dev[2], dev[4])
    out, lse = mla.paged_decode(d, *dev, workspace=ws)
    assert mla.last_path() == mla.PATH_TC and mla.mla_check_device_error() == 0
    ref.check_decode(BF16, out, lse, ref.decode(d, *t))
    for _ in range(40):
        o, l = mla.paged_decode(d, *dev, workspace=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert mla.mla_check_device_error() == 0
