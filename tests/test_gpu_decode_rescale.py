"""Split-KV decode whose running maximum grows tile after tile, so that the accumulator is rescaled late
in a split, with its earlier products long complete."""
import pytest
import torch

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("heads,length,n_splits", [(128, 900, 1), (128, 4000, 3), (256, 1500, 1)])
def test_growing_maximum(heads, length, n_splits):
    d = mla.dims(heads, 512, 128, 64, 128)
    g = ref.generator(heads + length)
    q, r, w = ref.queries(g, d, BF16, 2)
    # (900 keys: 9 tiles at which some row's maximum grows by more than the 2^8 that O waits for)
    rise = 0.25 + 6.0 * torch.arange(length)[None, :, None] / length
    c = (torch.randn(2, length, 512, generator=g) * rise).to(BF16)
    k = torch.randn(2, length, 64, generator=g).to(BF16)
    out, lse = mla.decode_splitkv(d, *(x.cuda() for x in (q, r, c, k, w)), n_splits=n_splits)
    torch.cuda.synchronize()
    assert mla.last_path() == mla.PATH_TC
    table = torch.arange(2, dtype=torch.int32)[:, None]
    lens = torch.full((2,), length, dtype=torch.int32)
    ro, rl, mass, sq = ref.decode(d, q, r, c, k, table, lens, w)
    bound, rel = ref.decode_bounds(BF16, rl, mass, sq)
    # Besides what those bounds count, this path holds the absorbed and the rotated query in fp16: each q_d is
    # off by at most 2^-11 of itself, uniformly, so a score by a deviation of 2^-11 sqrt(sq / 3).  The
    # log-sum-exp averages such errors of one sign at most: four deviations with the factor for the tail.
    # A weight's relative error is its score's, and the output's one deviation of that.
    dev = 2.0 ** -11 * torch.sqrt(sq / 3)
    err = (lse.double().cpu() - rl).abs()
    assert bool((err <= bound + 4 * dev).all()), float((err / (bound + 4 * dev)).max())
    off = float((out.double().cpu() - ro).norm() / ro.norm())
    assert off <= rel + float(dev.max()), (off, rel)
