"""Long chunks of mla_paged_prefill on a GPU, in both of their forms: sampled rows against 64 bits, the forms
against one another, missing pages, requests that do not fit the key buffers."""
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
BF = torch.bfloat16


def kernels(fn):
    """fn()'s result and the names of the kernels that it launched."""
    mla.profile_enable(True)
    mla.profile_reset()
    got = fn()
    torch.cuda.synchronize()
    names = set(mla.profile_all())
    mla.profile_enable(False)
    assert mla.mla_check_device_error(None) == 0
    return got, names


def sample(s, rows):
    """The step of those rows alone: one row a request."""
    own = sref.owners(s)
    b = [own[t] for t in rows]
    return dict(s, q_nope=s["q_nope"][rows], q_pe=s["q_pe"][rows], positions=s["positions"][rows],
                block_table=s["block_table"][b], kv_lens=s["kv_lens"][b],
                cu_tokens=torch.arange(len(rows) + 1, dtype=torch.int32))


def check_rows(d, s, out, lse, rows):
    """Rows of the explicit form: its score operands are fp16 (half a step 2^-12 where bf16's is 2^-8, which the
    bounds of ref.decode_bounds are about: K_nope is rounded where those round the absorbed query), and the weights
    of a row are of fp16 too, so the log-sum-exp adds half a step of those, over as many as carry the sum."""
    want = sref.prefill(d, sample(s, rows))
    ref.check_decode(BF, out[rows].cpu(), lse[rows].cpu(), want)


def spread(cu, b, n):
    """Rows of request b: its first, last, and those at tiles' borders."""
    t0, t1 = cu[b], cu[b + 1]
    return sorted({t for t in (t0, t0 + 1, t0 + 127, t0 + 128, t0 + (t1 - t0) // 2, t1 - 129, t1 - 128, t1 - 2, t1 - 1) if t0 <= t < t1})[:n]


CASES = [   # heads, page, (past, new) of each request, requests that go explicit
    (16, 16, [(0, 700)], [0]),
    (16, 64, [(900, 161), (3, 2), (0, 1300), (0, 0), (8000, 65)], [0, 2]),
    (128, 64, [(600, 200), (50, 1), (1024, 128)], [0]),
    (20, 48, [(511, 333), (512, 333)], [0, 1]),
    (1, 8, [(1000, 300), (0, 673)], [0, 1]),
    (3, 128, [(0, 5), (5, 800)], [1]),
    (16, 16, [(0, 64), (0, 63), (100, 65)], [0, 2]),
    (16, 64, [(2048, 300)] * 3 + [(130, 70), (40000, 200)], [0, 1, 2, 3, 4]),
]


@pytest.mark.parametrize("heads,page,lens,explicit", CASES)
@pytest.mark.parametrize("head_shard", [0, 3])
def test_against_64_bits(heads, page, lens, explicit, head_shard):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads + page), d, BF, lens, page, extra_rows=3, lead=2)
    a = sref.on_gpu(s)
    n = s["positions"].numel()
    out = torch.full((n, heads, 128), 5.0, dtype=BF).cuda()
    lse = torch.full((n, heads), 6.0).cuda()
    _, names = kernels(lambda: mla.paged_prefill(d, *a, out=out, lse=lse, head_shard=head_shard))
    assert {"paged_chunk", "tc_gemm", "tc_step_attn"} <= names
    for t in (0, 1, n - 3, n - 2, n - 1):
        assert bool((out[t] == 5).all()) and bool((lse[t] == 6).all())
    cu = s["cu_tokens"].tolist()
    for b, (_, new) in enumerate(lens):
        if new:
            check_rows(d, s, out, lse, spread(cu, b, 9 if heads < 128 else 4))
    # the same step absorbed: another kernel's rounding, so within both bounds of the values; here a coarse one on all
    # rows, bf16 outputs of which each is off by at most a few half steps of the row's largest value
    o2, l2 = mla.paged_prefill(d, *a, key_rows=0)
    mine = slice(2, n - 3)
    # a score's error: 192 products of fp16 operands, each off by 2^-12 relative, at unit scale below 2^-11
    assert float((lse[mine] - l2[mine]).abs().max()) <= 2.0 ** -9
    diff = (out[mine].float() - o2[mine].float()).norm(dim=-1) / o2[mine].float().norm(dim=-1).clamp(min=1e-9)
    assert float(diff.max()) <= 2.0 ** -5


@pytest.mark.parametrize("heads", [16, 128])
def test_missing_pages_and_odd_positions(heads):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(5), d, BF, [(700, 300), (900, 170), (0, 2)], 32)
    t = s["block_table"]
    t[0, 1] = t[0, 4:9] = t[0, 30] = -1
    t[1, 2] = 1 << 20
    t[1, 0] = -9
    pos = s["positions"]
    pos[5] = -1
    pos[6] = 3
    pos[7] = 1 << 30
    pos[[20, 299]] = pos[[299, 20]]
    s["kv_lens"][1] = 1000
    a = sref.on_gpu(s)
    (out, lse), names = kernels(lambda: mla.paged_prefill(d, *a))
    assert "tc_step_attn" in names
    check_rows(d, s, out, lse, [0, 4, 5, 6, 7, 20, 128, 299, 300, 399, 400, 469, 470, 471])


def test_all_pages_gone():
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(6), d, BF, [(600, 200)], 16)
    s["block_table"][0] = -1
    out, lse = mla.paged_prefill(d, *sref.on_gpu(s))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_what_lies_behind_the_length_does_not_matter():
    """The cache's other slots hold NaN in every test here; infinities and large values give the same bits."""
    d = mla.dims(16, **V3)
    got = []
    for junk in (math.nan, math.inf, 1e30):
        s = sref.step(ref.generator(7), d, BF, [(600, 301), (5, 3)], 16, junk=junk)
        got.append(mla.paged_prefill(d, *sref.on_gpu(s)))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_requests_that_do_not_fit_go_absorbed():
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(8), d, BF, [(600, 200), (700, 300), (900, 200)], 16)
    a = sref.on_gpu(s)
    full = mla.paged_prefill(d, *a)
    for rows in (0, 255, 768, 1023, 1024, 2047, 2304, 1 << 14):
        out, lse = mla.paged_prefill(d, *a, key_rows=rows)
        assert float((lse - full[1]).abs().max()) <= 2.0 ** -9 and float((out.float() - full[0].float()).abs().max()) <= 2.0 ** -5
    check_rows(d, s, out, lse, [0, 199, 200, 499, 500, 699])


def test_the_same_bits_whatever_the_shard_and_in_a_graph():
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(9), d, BF, [(600, 200), (0, 900), (77, 1)], 64)
    a = sref.on_gpu(s)
    first = mla.paged_prefill(d, *a)
    for shard in (0, 1, 5, 99):
        o, l = mla.paged_prefill(d, *a, head_shard=shard)
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    ws = mla.paged_prefill_workspace(d, s["positions"].numel(), a[2], a[4])
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.paged_prefill(d, *a, out=out, lse=lse, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mla.paged_prefill(d, *a, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    # the replayed step follows the lengths on the device: another division of the same rows
    s["cu_tokens"] = torch.tensor([0, 150, 1100, 1101], dtype=torch.int32)
    s["positions"][150:200] = torch.arange(50, dtype=torch.int32)
    s["positions"][200:1100] = torch.arange(0, 900, dtype=torch.int32)
    a[6].copy_(s["cu_tokens"])
    a[7].copy_(s["positions"])
    graph.replay()
    torch.cuda.synchronize()
    check_rows(d, s, out, lse, [0, 149, 150, 199, 200, 800, 1099, 1100])
