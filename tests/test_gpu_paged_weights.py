"""mla_paged_weights on a GPU against 64 bits."""
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
SMALL = dict(d_kv=20, d_nope=8, d_rope=6, d_v=10)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)
BF, F32 = torch.bfloat16, torch.float32


def call(d, s, lse, prior=None, **kw):
    a = sref.on_gpu(s)
    w = mla.paged_weights(d, *a[:2], lse.cuda(), *a[2:], prior=None if prior is None else prior.cuda(), **kw)
    torch.cuda.synchronize()
    assert mla.mla_check_device_error(None) == 0
    return w.cpu()


def check(d, s, lse, got, prior=None):
    want, bound = sref.weights(d, s, lse, prior)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (float(err.max()), float((err / bound.clamp(min=1e-300)).max()))


def lse_of(d, s):
    return sref.prefill(d, s)[1].nan_to_num(3.0, neginf=-math.inf).float()


CASES = [   # heads, dims, dtype, page, (past, new) of each request
    (3, SMALL, F32, 5, [(0, 1), (4, 3), (0, 0), (13, 7)]),
    (18, TINY, F32, 16, [(40, 3), (0, 20)]),
    (5, SMALL, BF, 4, [(3, 9), (0, 2)]),
    (16, V3, F32, 32, [(70, 3), (0, 5)]),
    (128, V3, BF, 64, [(0, 1)]),
    (128, V3, BF, 64, [(62, 5), (0, 3), (0, 0), (700, 1)]),
    (128, V3, BF, 8, [(250, 6), (7, 9)]),
    (16, V3, BF, 16, [(0, 1), (1000, 4), (0, 0), (62, 17), (5, 61)]),
    (8, V3, BF, 64, [(100, 17), (0, 70)]),
    (1, V3, BF, 16, [(0, 130), (77, 1), (3, 64)]),
    (20, V3, BF, 48, [(45, 10), (290, 3)]),
    (64, V3, BF, 128, [(120, 4), (0, 9)]),
    (80, V3, BF, 32, [(33, 3), (600, 2)]),
    (160, V3, BF, 64, [(70, 2), (0, 3)]),
    (3, V3, BF, 24, [(5, 3), (511, 1), (512, 1), (255, 2)]),
    (16, V3, BF, 7, [(20, 5), (0, 3)]),
]


@pytest.mark.parametrize("heads,dims,dtype,page,lens", CASES)
def test_against_64_bits(heads, dims, dtype, page, lens):
    d = mla.dims(heads, **dims)
    s = sref.step(ref.generator(heads + page), d, dtype, lens, page, extra_rows=2, lead=1)
    lse = lse_of(d, s)
    prior = torch.rand(s["block_table"].shape, generator=ref.generator(1))
    for p in (None, prior):
        check(d, s, lse, call(d, s, lse, p), p)


@pytest.mark.parametrize("heads,dtype", [(4, F32), (16, BF), (128, BF)])
def test_masks_and_odd_log_sum_exps(heads, dtype):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(6), d, dtype, [(60, 6), (3, 4), (300, 5)], 16)
    s["positions"][[0, 7]] = -1                     # no keys
    s["positions"][2] = 1000000
    s["positions"][4] = 2147483647
    s["positions"][[10, 11]] = torch.tensor([133, 2], dtype=torch.int32)
    s["block_table"][2, 1] = -1
    s["block_table"][2, 3:5] = 1 << 20
    s["block_table"][0, 4] = -7
    lse = lse_of(d, s)
    lse[1] = -math.inf       # as a token that saw nothing
    lse[12, 0] = math.nan    # counts as nothing
    lse[13, 0] = math.inf
    got = call(d, s, lse)
    check(d, s, lse.nan_to_num(math.inf, posinf=math.inf, neginf=-math.inf), got)


@pytest.mark.parametrize("heads,dtype", [(4, F32), (128, BF)])
def test_each_weight_is_cut(heads, dtype):
    """A log-sum-exp that does not belong to the scores: every weight is 2."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(7), d, dtype, [(300, 3)], 64)
    got = call(d, s, torch.full((3, heads), -200.0))
    want = torch.zeros_like(got)
    for t in range(3):
        for c in range(5):
            want[0, c] += 2.0 * heads * min(64, 301 + t - 64 * c)
    assert torch.equal(got, want)


@pytest.mark.parametrize("heads,dims,dtype", [(2, TINY, F32), (16, V3, BF)])
def test_more_tokens_than_a_round(heads, dims, dtype):
    """4200 tokens: every token's weights sum to 1 a head."""
    d = mla.dims(heads, **dims)
    s = sref.step(ref.generator(9), d, dtype, [(5, 1), (0, 2100), (30, 60), (100, 2039)], 64, extra_rows=2)
    a = sref.on_gpu(s)
    _, lse = mla.paged_prefill(d, *a)
    got = call(d, s, lse.cpu())
    total = got.double().sum(1)
    # lse and the scores here: 2^-16 (1 + mass) each, the mass of these scores below 16 (12 deviations of a sum of products)
    for b, n in enumerate((1, 2100, 60, 2039)):
        assert abs(float(total[b]) - n * heads) <= n * heads * 2.0 ** -15 * 17


def test_no_tokens_no_requests():
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(2), d, BF, [(20, 0), (5, 0)], 8)
    prior = torch.rand(s["block_table"].shape, generator=ref.generator(1))
    empty = torch.zeros(0, 16)
    assert torch.equal(call(d, s, empty, prior), prior)
    assert torch.equal(call(d, s, empty), torch.zeros_like(prior))


def test_in_place_same_bits_and_in_a_graph():
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(10), d, BF, [(900, 5), (0, 40), (300, 1)], 16)
    a = sref.on_gpu(s)
    lse = lse_of(d, s).cuda()
    ws = mla.paged_weights_workspace(d, s["positions"].numel(), a[2], a[4])
    first = mla.paged_weights(d, *a[:2], lse, *a[2:], workspace=ws)
    assert torch.equal(first, mla.paged_weights(d, *a[:2], lse, *a[2:], workspace=ws))
    acc = torch.zeros_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.paged_weights(d, *a[:2], lse, *a[2:], prior=acc, out=acc, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mla.paged_weights(d, *a[:2], lse, *a[2:], prior=acc, out=acc, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    # three calls added up: each rounds the running sum, half a step of at most three times the weight
    assert bool(((acc.double() - 3 * first.double()).abs() <= 3 * 3 * 2.0 ** -24 * first.double()).all())
