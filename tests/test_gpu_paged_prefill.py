"""mla_paged_prefill on a GPU against 64 bits: types, heads, lengths from one token, odd sizes, pages that end
inside a tile, empty and padded rows, evicted pages."""
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


def call(d, s, **kw):
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s), **kw)
    torch.cuda.synchronize()
    assert mla.mla_check_device_error(None) == 0
    return out, lse


CASES = [   # heads, dims, dtype, page, (past, new) of each request
    (3, SMALL, F32, 5, [(0, 1), (4, 3), (0, 0), (13, 7)]),
    (4, TINY, F32, 7, [(0, 33), (200, 5), (1, 1)]),
    (18, TINY, F32, 16, [(40, 3), (0, 20)]),
    (5, SMALL, BF, 4, [(3, 9), (0, 2)]),
    (16, V3, F32, 32, [(70, 3), (0, 5)]),
    (128, V3, BF, 64, [(0, 1)]),
    (128, V3, BF, 64, [(62, 5), (0, 3), (0, 0), (300, 1)]),
    (128, V3, BF, 8, [(129, 2), (7, 9)]),
    (16, V3, BF, 16, [(0, 1), (1000, 4), (0, 0), (62, 7), (5, 61)]),
    (8, V3, BF, 64, [(100, 17), (0, 70)]),
    (1, V3, BF, 16, [(0, 130), (77, 1), (3, 64)]),
    (20, V3, BF, 48, [(45, 10), (190, 3)]),
    (64, V3, BF, 128, [(120, 4), (0, 9)]),
    (80, V3, BF, 32, [(33, 3), (200, 2)]),
    (160, V3, BF, 64, [(70, 2), (0, 3)]),
    (16, V3, BF, 7, [(20, 5), (0, 3)]),
]


@pytest.mark.parametrize("heads,dims,dtype,page,lens", CASES)
def test_against_64_bits(heads, dims, dtype, page, lens):
    d = mla.dims(heads, **dims)
    s = sref.step(ref.generator(heads + page), d, dtype, lens, page)
    out, lse = call(d, s)
    sref.check_prefill(dtype, out, lse, sref.prefill(d, s))


@pytest.mark.parametrize("heads,dtype,page", [(4, F32, 16), (16, BF, 16), (128, BF, 64)])
def test_rows_of_no_request_are_left_alone(heads, dtype, page):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(3), d, dtype, [(9, 3), (0, 0), (50, 2)], page, extra_rows=5, lead=3)
    n = s["positions"].numel()
    out = torch.randn(n, heads, 128, generator=ref.generator(4)).to(dtype).cuda()
    lse = torch.randn(n, heads, generator=ref.generator(5)).cuda()
    before = out.clone(), lse.clone()
    call(d, s, out=out, lse=lse)
    sref.check_prefill(dtype, out, lse, sref.prefill(d, s), before)


@pytest.mark.parametrize("heads,dtype", [(4, F32), (16, BF), (128, BF)])
def test_tokens_that_see_nothing_or_less_than_the_request(heads, dtype):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(6), d, dtype, [(60, 6), (3, 4), (130, 5)], 16)
    s["positions"][[0, 7]] = -1                     # no keys
    s["positions"][2] = 1000000                     # all of the request's
    s["positions"][4] = 2147483647
    s["positions"][[10, 11]] = torch.tensor([133, 2], dtype=torch.int32)   # out of order
    s["kv_lens"][1] = 0
    s["block_table"][2, 1] = -1
    s["block_table"][2, 3:5] = 1 << 20
    s["block_table"][0, 4] = -7
    out, lse = call(d, s)
    sref.check_prefill(dtype, out, lse, sref.prefill(d, s))


@pytest.mark.parametrize("heads,dtype", [(4, F32), (16, BF), (128, BF)])
def test_all_pages_evicted(heads, dtype):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(7), d, dtype, [(20, 3), (7, 2)], 8)
    s["block_table"][0] = -1
    out, lse = call(d, s)
    assert bool((lse[:3] == -math.inf).all()) and bool((out[:3] == 0).all())
    sref.check_prefill(dtype, out, lse, sref.prefill(d, s))


@pytest.mark.parametrize("heads,dtype,page", [(16, BF, 64), (128, BF, 64), (8, F32, 16)])
def test_one_token_a_request_is_decode(heads, dtype, page):
    """The same rows as mla_paged_decode's, which is held to 64 bits by its own tests."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(8), d, dtype, [(500, 1), (0, 1), (63, 1), (64, 1), (1200, 1)], page)
    out, lse = call(d, s)
    sref.check_prefill(dtype, out, lse, sref.prefill(d, s))
    q, r, c, k, table, lens, _, _, w = sref.on_gpu(s)
    o2, l2 = mla.paged_decode(d, q, r, c, k, table, lens, w)
    assert float((lse - l2).abs().max()) <= 1e-5 and float((out.float() - o2.float()).abs().max()) <= 0.05


@pytest.mark.parametrize("heads,dims,dtype,key_rows", [(2, TINY, F32, None), (16, V3, BF, None), (16, V3, BF, 0),
                                                       (128, V3, BF, None), (128, V3, BF, 0)])
def test_more_tokens_than_a_round(heads, dims, dtype, key_rows):
    """4300 tokens: two rounds of the absorbed form; sampled rows against 64 bits, all rows finite."""
    d = mla.dims(heads, **dims)
    lens = [(5, 1), (0, 2100), (30, 60), (100, 2139)]
    s = sref.step(ref.generator(9), d, dtype, lens, 64, extra_rows=2)
    n = s["positions"].numel()
    out, lse = call(d, s, key_rows=key_rows)
    assert bool(torch.isfinite(lse[:-2]).all()) and bool((lse[-2:] == 0).all()) and bool((out[-2:] == 0).all())
    rows = [0, 1, 2, 700, 2047, 2048, 2049, 2100, 2101, 2130, 2160, 2161, 2162, 4095, 4096, 4097, n - 3]
    want = sref.prefill(d, dict(s, **sample(s, rows)))
    ref.check_decode(dtype, out[rows], lse[rows], want)


def sample(s, rows):
    """The step of those rows alone: one row a request."""
    own = sref.owners(s)
    i32 = dict(dtype=torch.int32)
    b = [own[t] for t in rows]
    return dict(q_nope=s["q_nope"][rows], q_pe=s["q_pe"][rows], positions=s["positions"][rows],
                block_table=s["block_table"][b], kv_lens=s["kv_lens"][b], cu_tokens=torch.arange(len(rows) + 1, **i32))


def test_the_same_bits_twice_and_in_a_graph():
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(10), d, BF, [(900, 5), (0, 40), (300, 1)], 16)
    a = sref.on_gpu(s)
    ws = mla.paged_prefill_workspace(d, s["positions"].numel(), a[2], a[4])
    first = mla.paged_prefill(d, *a, workspace=ws)
    again = mla.paged_prefill(d, *a, workspace=ws)
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.paged_prefill(d, *a, out=out, lse=lse, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mla.paged_prefill(d, *a, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    out.zero_()
    lse.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x in (again, (out, lse)):
        assert torch.equal(x[0], first[0]) and torch.equal(x[1], first[1])
    # the replayed step follows the lengths on the device
    a[7][:5] -= 1
    s["positions"][:5] -= 1
    graph.replay()
    torch.cuda.synchronize()
    sref.check_prefill(BF, out, lse, sref.prefill(d, s))
