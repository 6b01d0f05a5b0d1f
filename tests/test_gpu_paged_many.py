"""Steps of many tokens in the absorbed form, whose absorb and join take tiles of 128 tokens, against 64 bits: heads below
and above 64 and a row tile, ends of tiles, tokens of few keys and of many parts, lists of tokens, padded rows."""
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
BF = torch.bfloat16


def call(d, s, **kw):
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s), **kw)
    torch.cuda.synchronize()
    assert mla.mla_check_device_error(None) == 0
    return out, lse


CASES = [   # heads, page, (past, new) of each request
    (128, 64, [(0, 40), (300, 60), (0, 1), (1500, 33), (62, 10)]),             # third parts, one and two blocks of q_lo
    (128, 16, [(5000, 2)] + [(3, 63)] * 2 + [(90, 1)]),                        # 129 tokens
    (128, 64, [(9000, 1), (0, 0)] + [(10, 33)] * 4),                           # one token in parts of a few key tiles each
    (64, 64, [(9000, 1), (0, 0)] + [(10, 63)] * 3),
    (96, 32, [(40, 60)] * 4 + [(0, 16)]),                                      # 256 tokens
    (64, 8, [(1, 63), (200, 50), (0, 62), (61, 6)]),
    (20, 64, [(3, 63)] * 8 + [(700, 9)]),                                      # several tokens an item
    (200, 64, [(0, 60), (80, 50), (900, 25)]),                                 # two items a token
]


@pytest.mark.parametrize("heads,page,lens", CASES)
def test_against_64_bits(heads, page, lens):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads + page), d, BF, lens, page)
    out, lse = call(d, s, key_rows=0)
    sref.check_prefill(BF, out, lse, sref.prefill(d, s))


@pytest.mark.parametrize("heads", [20, 128])
def test_next_to_requests_in_the_explicit_form(heads):
    """A list of the absorbed requests' tokens, fewer than the step's."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(2), d, BF, [(100, 40), (0, 70), (500, 3), (0, 400), (30, 60), (0, 1)], 16, extra_rows=3, lead=2)
    n = s["positions"].numel()
    out = torch.randn(n, heads, 128, generator=ref.generator(4)).to(BF).cuda()
    lse = torch.randn(n, heads, generator=ref.generator(5)).cuda()
    before = out.clone(), lse.clone()
    call(d, s, out=out, lse=lse)
    sref.check_prefill(BF, out, lse, sref.prefill(d, s), before)


@pytest.mark.parametrize("heads", [64, 128])
def test_rows_of_no_request_and_tokens_that_see_nothing(heads):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(3), d, BF, [(9, 60), (0, 0), (50, 62), (130, 30), (20, 8)], 16, extra_rows=90, lead=3)
    s["positions"][[3, 40, 70]] = -1
    s["q_nope"][[3, 40]] = math.nan                      # queries of no keys
    s["q_nope"][[0, 1, 2]] = math.nan                    # and of no request
    s["positions"][80] = 2147483647
    s["kv_lens"][3] = 0
    s["block_table"][4] = -1
    s["block_table"][2, 3] = 1 << 20
    n = s["positions"].numel()
    out = torch.randn(n, heads, 128, generator=ref.generator(4)).to(BF).cuda()
    lse = torch.randn(n, heads, generator=ref.generator(5)).cuda()
    before = out.clone(), lse.clone()
    call(d, s, out=out, lse=lse, key_rows=0)
    sref.check_prefill(BF, out, lse, sref.prefill(d, s), before)


@pytest.mark.parametrize("heads,lens", [(128, [(70, 63), (0, 60), (600, 20)]), (20, [(64, 63)] * 8 + [(0, 30)])])
def test_weights(heads, lens):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(8), d, BF, lens, 16, extra_rows=2)
    lse = sref.prefill(d, s)[1].nan_to_num(3.0, neginf=-math.inf).float()
    a = sref.on_gpu(s)
    got = mla.paged_weights(d, *a[:2], lse.cuda(), *a[2:])
    torch.cuda.synchronize()
    assert mla.mla_check_device_error(None) == 0
    want, bound = sref.weights(d, s, lse)
    assert bool(((got.cpu().double() - want).abs() <= bound).all())


def test_the_same_bits_twice_in_a_graph_and_two_at_once():
    d = mla.dims(128, **V3)
    a = sref.on_gpu(sref.step(ref.generator(10), d, BF, [(900, 60), (0, 40), (300, 63)], 16))
    first = mla.paged_prefill(d, *a)
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    ws = mla.paged_prefill_workspace(d, a[0].shape[0], a[2], a[4])
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
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    others = [mla.paged_prefill(d, *a) for _ in range(3)]   # next to the graph
    torch.cuda.synchronize()
    assert mla.mla_check_device_error(None) == 0
    for x in others + [(out, lse)]:
        assert torch.equal(x[0], first[0]) and torch.equal(x[1], first[1])


@pytest.mark.parametrize("heads,lens", [(16, [(0, 40), (0, 33), (5, 47), (0, 32), (100, 48), (0, 31), (0, 63), (330, 60)]),
                                        (64, [(0, 32), (0, 0), (90, 47), (200, 63)]), (20, [(1, 34), (64, 50), (127, 33)]),
                                        (128, [(0, 45), (83, 45), (150, 63)])])
def test_short_requests_that_go_explicit(heads, lens):
    """32 tokens and more over few keys: tiles of 128 rows that are mostly empty, rests of fewer key tiles than there are."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads), d, BF, lens, 16, extra_rows=2, lead=1)
    n = s["positions"].numel()
    out = torch.randn(n, heads, 128, generator=ref.generator(4)).to(BF).cuda()
    lse = torch.randn(n, heads, generator=ref.generator(5)).cuda()
    before = out.clone(), lse.clone()
    call(d, s, out=out, lse=lse)
    sref.check_prefill(BF, out, lse, sref.prefill(d, s), before)
