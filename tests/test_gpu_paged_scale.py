"""A model's own softmax_scale and rope_base in every form of paged prefill and of the page weights."""
import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from test_gpu_paged_chunks import check_rows, spread
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("scale,base", [(0.02, 10000.0), (0.11, 300.0), (0.0, 5e6)])
@pytest.mark.parametrize("heads,dims,dtype,lens", [
    (4, TINY, F32, [(90, 3), (40, 1)]), (4, V3, F32, [(50, 2), (5, 1)]), (16, V3, BF, [(900, 3), (40, 1)]),
    (128, V3, BF, [(300, 2), (70, 9)]), (32, V3, BF, [(50, 30)] * 5), (16, V3, BF, [(300, 200), (40, 1)]),
])
def test_scale_and_base(heads, dims, dtype, lens, scale, base):
    d = mla.dims(heads, rope_base=base, softmax_scale=scale, **dims)
    s = sref.step(ref.generator(heads + len(lens)), d, dtype, lens, 16)
    a = sref.on_gpu(s)
    out, lse = mla.paged_prefill(d, *a)
    if max(n for _, n in lens) > 100:
        cu = s["cu_tokens"].tolist()
        for b in range(len(lens)):
            check_rows(d, s, out, lse, spread(cu, b, 9))
    else:
        sref.check_prefill(dtype, out, lse, sref.prefill(d, s))
    got = mla.paged_weights(d, *a[:2], lse, *a[2:]).cpu()
    want, bound = sref.weights(d, s, lse.cpu())
    assert bool(((got.double() - want).abs() <= bound).all())
    # the default scale and base would not pass for these
    other = mla.paged_prefill(mla.dims(heads, **dims), *a)[1]
    assert float((other - lse).abs().max()) > 2.0 ** -6
