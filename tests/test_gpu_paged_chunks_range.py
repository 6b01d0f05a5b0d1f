"""The size of the values does not matter to the explicit form: it holds V in fp16 times a power of two of each head and
request, so W_V or the cache times a power of two give outputs times that power, to the bit, as in the absorbed form."""
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from test_gpu_paged_chunks import check_rows, spread
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
BF = torch.bfloat16
LENS = [(600, 200), (3, 2), (0, 300)]


def parts(d, w):
    """W_K and W_V of w_kv_b, as views."""
    x = w.view(d.n_heads, d.d_nope + d.d_v, d.d_kv)
    return x[:, :d.d_nope], x[:, d.d_nope:]


@pytest.mark.parametrize("heads", [3, 16])
@pytest.mark.parametrize("key_rows", [None, 0])
@pytest.mark.parametrize("power", [-80, -40, -24, -12, 12, 17, 40, 80])
def test_weights_times_a_power_of_two(heads, key_rows, power):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads), d, BF, LENS, 16)
    want = mla.paged_prefill(d, *sref.on_gpu(s), key_rows=key_rows)
    parts(d, s["w_kv_b"])[1].mul_(2.0 ** power)
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s), key_rows=key_rows)
    assert torch.equal(lse, want[1]) and torch.equal(out.double(), want[0].double() * 2.0 ** power)


@pytest.mark.parametrize("heads", [3, 16])
@pytest.mark.parametrize("power", [-60, -20, 20, 60])
def test_cache_times_a_power_of_two(heads, power):
    """W_K the other way, so that the scores stay."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads), d, BF, LENS, 16)
    want = mla.paged_prefill(d, *sref.on_gpu(s))
    s["c_cache"].mul_(2.0 ** power)
    parts(d, s["w_kv_b"])[0].mul_(2.0 ** -power)
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s))
    assert torch.equal(lse, want[1]) and torch.equal(out.double(), want[0].double() * 2.0 ** power)


@pytest.mark.parametrize("heads,shard", [(16, 0), (16, 5), (128, 64)])
def test_heads_of_their_own_sizes(heads, shard):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads), d, BF, LENS, 16)
    want = mla.paged_prefill(d, *sref.on_gpu(s), head_shard=shard)
    power = (torch.arange(heads) * 37 % 121 - 60).double()
    v = parts(d, s["w_kv_b"])[1]
    v.copy_((v.double() * torch.exp2(power)[:, None, None]).to(BF))
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s), head_shard=shard)
    assert torch.equal(lse, want[1]) and torch.equal(out.double(), want[0].double() * torch.exp2(power).cuda()[:, None])


@pytest.mark.parametrize("key_rows", [None, 0])
def test_requests_of_their_own_sizes(key_rows):
    """Caches of other sizes side by side, to 64 bits; a request's do not touch its neighbour's bits."""
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(5), d, BF, [(600, 200), (0, 300), (700, 250)], 16)
    first = mla.paged_prefill(d, *sref.on_gpu(s), key_rows=key_rows)
    cu = s["cu_tokens"].tolist()
    for b, size in ((0, 1e-9), (2, 3e-6)):
        ids = s["block_table"][b]
        s["c_cache"][ids[ids >= 0].long()] *= size
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s), key_rows=key_rows)
    if key_rows is None:   # (the absorbed form's parts are cut alike too, but that is not promised)
        t = slice(cu[1], cu[2])
        assert torch.equal(out[t], first[0][t]) and torch.equal(lse[t], first[1][t])
    for b in range(3):
        check_rows(d, s, out, lse, spread(cu, b, 5))


def test_infinities_in_a_request_or_head_stay_there():
    """NaN and infinity in one request's cache, and in one head's W_V, leave the bits of the others."""
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(6), d, BF, [(600, 200), (0, 300)], 16)
    cu = s["cu_tokens"].tolist()
    want = mla.paged_prefill(d, *sref.on_gpu(s))
    for junk in (math.nan, math.inf):
        b = dict(s, c_cache=s["c_cache"].clone(), w_kv_b=s["w_kv_b"].clone())
        b["c_cache"][b["block_table"][0, 3].long(), 5, 7] = junk
        parts(d, b["w_kv_b"])[1][4, 9, 11] = junk
        out, lse = mla.paged_prefill(d, *sref.on_gpu(b))
        t, rest = slice(cu[1], cu[2]), [h for h in range(16) if h != 4]
        assert torch.equal(out[t][:, rest], want[0][t][:, rest]) and torch.equal(lse[t], want[1][t])
        keep = [v for v in range(128) if v != 9]
        assert torch.equal(out[t][:, 4, keep], want[0][t][:, 4, keep]) and bool((~torch.isfinite(out[t][:, 4, 9])).all())


@pytest.mark.parametrize("heads", [3, 16])
@pytest.mark.parametrize("power", [-10, -8, 8, 10])
def test_score_operands_of_other_sizes(heads, power):
    """K_nope times a power of two and q_nope the other way, inside fp16's range: K_nope's typical 2^-10 is held to
    2^-12 of itself, its small values to 2^-25, which is 2^-15 of it, and q_nope's likewise: the bounds of unit scale."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads), d, BF, LENS, 16)
    parts(d, s["w_kv_b"])[0].mul_(2.0 ** power)
    s["q_nope"].mul_(2.0 ** -power)
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s))
    cu = s["cu_tokens"].tolist()
    for b in range(3):
        check_rows(d, s, out, lse, spread(cu, b, 6))


def test_nothing_but_zeros():
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(7), d, BF, LENS, 16)
    want = mla.paged_prefill(d, *sref.on_gpu(s))
    parts(d, s["w_kv_b"])[1].zero_()
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s))
    assert bool((out == 0).all()) and torch.equal(lse, want[1])
