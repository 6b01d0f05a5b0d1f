"""NaN and infinity in the queries of the explicit form: the token that holds them gives NaN, as in the absorbed form and on
the CUDA cores; a log-sum-exp of -inf says that a token sees no key, and nothing else."""
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
BF = torch.bfloat16


@pytest.mark.parametrize("heads,lens", [(16, [(300, 200)]), (3, [(64, 130), (100, 64)]), (128, [(40, 257)])])
@pytest.mark.parametrize("which", ["q_nope", "q_pe"])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_a_row_of_nan_is_not_one_without_keys(heads, lens, which, junk):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads), d, BF, lens, 16)
    n = s["positions"].numel()
    s["positions"][3] = -1                                    # sees no key, whatever its queries hold
    at = [1, 2, 3, n - 1]
    head = heads - 1
    for t in at:
        s[which][t, head] = junk if t == 1 or junk != junk else 0.0
        s[which][t, head, 5] = junk                           # one dim or all
    a = sref.on_gpu(s)
    explicit = mla.paged_prefill(d, *a)
    absorbed = mla.paged_prefill(d, *a, key_rows=0)
    mla.set_path_override(1)
    try:
        simt = mla.paged_prefill(d, *a)
    finally:
        mla.set_path_override(0)
    assert mla.mla_check_device_error(None) == 0
    for out, lse in (explicit, absorbed, simt):
        assert bool((lse[3] == -math.inf).all()) and bool((out[3] == 0).all())
        bad = torch.zeros(n, heads, dtype=torch.bool)
        bad[[1, 2, n - 1], head] = True   # (infinite queries: scores of both signs among forty keys and more, so NaN)
        assert bool(lse.cpu()[bad].isnan().all()) and bool(out.cpu()[bad].isnan().all())
        good = ~bad
        good[3] = False
        assert bool(torch.isfinite(lse.cpu()[good]).all()) and bool(torch.isfinite(out.cpu()[good]).all())
