"""How mla_paged_prefill, mla_paged_weights and mla_paged_evict are called: on streams of the caller's, two at once, captured
on a forked stream, with workspaces that do not do; far pages, many requests, one token's NaN, decode's log-sum-exps."""
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla
from test_gpu_launch_stream import Allocations, flat

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)
BF, F32 = torch.bfloat16, torch.float32
I32 = dict(dtype=torch.int32)


def prefill(heads, dims, dtype, lens, seed=1, page=16):
    d = mla.dims(heads, **dims)
    a = sref.on_gpu(sref.step(ref.generator(seed), d, dtype, lens, page, extra_rows=1))
    return lambda **kw: mla.paged_prefill(d, *a, **kw)


def weights(heads, dims, dtype, lens, seed=1):
    d = mla.dims(heads, **dims)
    a = sref.on_gpu(sref.step(ref.generator(seed), d, dtype, lens, 16))
    _, lse = mla.paged_prefill(d, *a)
    torch.cuda.synchronize()
    return lambda **kw: mla.paged_weights(d, *a[:2], lse, *a[2:], **kw)


def evict():
    g = ref.generator(3)
    table = torch.randperm(3 * 40, generator=g).to(torch.int32).view(3, 40).cuda()
    w = torch.rand(3, 40, generator=g).cuda()
    lens = torch.tensor([300, 0, 317], **I32).cuda()

    def call(**kw):
        e = mla.paged_evict(lens, table, w, page_size=8, keep_pages=9, table_out=torch.empty_like(table),
                            weights_out=torch.empty_like(w), **kw)
        return e.freed[:60], e.counts   # 38 and 40 pages, of which nine stay each
    return call


CALLS = {
    "prefill_absorbed": lambda: prefill(16, V3, BF, [(900, 3), (40, 1)]),
    "prefill_both_forms": lambda: prefill(16, V3, BF, [(900, 300), (40, 1)]),
    "prefill_simt": lambda: prefill(4, TINY, F32, [(90, 3), (40, 1)]),
    "weights_tc": lambda: weights(16, V3, BF, [(900, 3), (40, 1)]),
    "weights_simt": lambda: weights(4, TINY, F32, [(90, 3), (40, 1)]),
}


@pytest.mark.parametrize("kind", ["stream", "handle", "external"])
@pytest.mark.parametrize("name", list(CALLS))
def test_allocates_for_the_launch_stream(name, kind):
    call = CALLS[name]()
    want = [x.clone() for x in flat(call())]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given = s if kind == "stream" else s.cuda_stream if kind == "handle" else torch.cuda.ExternalStream(s.cuda_stream)
    with Allocations() as seen:
        got = flat(call(stream=given))
    assert seen.streams == {s.cuda_stream}
    s.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("off", [16, 32, 48])
@pytest.mark.parametrize("name", list(CALLS))
def test_workspace_at_any_16_bytes(name, off):
    call = CALLS[name]()
    want = [x.clone() for x in flat(call())]
    room = torch.empty((512 << 20) + off, dtype=torch.uint8, device="cuda")
    assert room.data_ptr() % 32 == 0
    got = flat(call(workspace=room[off:]))
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_evict_on_a_stream():
    call = evict()
    want = [x.clone() for x in call()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    s.synchronize()
    assert want[1].tolist() == [60, 60] and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("names", [("prefill_both_forms", "prefill_absorbed"), ("prefill_both_forms", "prefill_both_forms"),
                                   ("weights_tc", "prefill_both_forms"), ("weights_tc", "weights_tc")])
def test_two_calls_at_once(names):
    calls = [CALLS[n]() for n in names]
    want = [[x.clone() for x in flat(c())] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [flat(c(stream=s)) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    assert mla.mla_check_device_error(None) == 0
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("name", list(CALLS))
def test_captured_on_a_forked_stream(name):
    call = CALLS[name]()
    want = [x.clone() for x in flat(call())]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = flat(call(stream=side))
        here.wait_stream(side)
    for _ in range(3):
        for x in got:
            x.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["prefill_both_forms", "weights_tc", "weights_simt"])
def test_workspace_refusals(name):
    call = CALLS[name]()
    room = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    for bad in (room[::2], room[:1].expand(1 << 24), room.view(1 << 13, 1 << 13).t()):
        with pytest.raises(ValueError, match="contiguous"):
            call(workspace=bad)
    for bad in (room.cpu(), 4096):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=bad)
    with pytest.raises(mla.MlaError, match="WORKSPACE"):
        call(workspace=room[:16])
    assert not bool(room.any())


def test_argument_refusals():
    d = mla.dims(16, **V3)
    a = sref.on_gpu(sref.step(ref.generator(1), d, BF, [(20, 3), (4, 1)], 8))
    lse = torch.zeros(4, 16).cuda()
    bad = {0: a[0][:, :8], 1: a[1].float(), 2: a[2][0], 3: a[3][:, :, :32], 4: a[4].long(), 5: a[5][:1], 6: a[6][:-1], 7: a[7][::2],
           8: a[8][:-1]}
    for i, t in bad.items():
        b = list(a)
        b[i] = t
        with pytest.raises((ValueError, TypeError)):
            mla.paged_prefill(d, *b)
        with pytest.raises((ValueError, TypeError)):
            mla.paged_weights(d, *b[:2], lse, *b[2:])
    with pytest.raises((ValueError, TypeError)):
        mla.paged_weights(d, *a[:2], lse.half(), *a[2:])
    for kw in (dict(prior=torch.zeros(2, 3).cuda()), dict(out=torch.zeros(3, 4).cuda()), dict(prior=torch.zeros(2, 4))):
        with pytest.raises(ValueError):
            mla.paged_weights(d, *a[:2], lse, *a[2:], **kw)
    with pytest.raises(mla.MlaError, match="SHAPE"):
        mla.paged_prefill(d, *a, key_rows=-1)
    w = torch.zeros_like(a[4], dtype=F32)
    for kw in (dict(table_out=a[4][:1]), dict(weights_out=w.half()), dict(freed=torch.zeros(4).cuda()), dict(counts=torch.zeros(3, **I32).cuda())):
        with pytest.raises((ValueError, TypeError)):
            mla.paged_evict(a[5], a[4], w, page_size=8, keep_pages=1, **kw)
    for kw in (dict(keep_pages=-1), dict(keep_pages=1, first_pages=-1), dict(keep_pages=1, last_pages=0)):
        with pytest.raises(mla.MlaError, match="SHAPE"):
            mla.paged_evict(a[5], a[4], w, page_size=8, **kw)


@pytest.mark.parametrize("heads,dtype,lens", [(4, F32, [(20, 4)]), (16, BF, [(20, 4)]), (128, BF, [(100, 3)]), (16, BF, [(300, 200)])])
def test_one_tokens_nan_stays_with_it(heads, dtype, lens):
    """A query of NaN or infinity leaves the other tokens' bits, in their group too, and gives pages no weight."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(8), d, dtype, lens, 16)
    a = sref.on_gpu(s)
    out, lse = mla.paged_prefill(d, *a)
    w = mla.paged_weights(d, *a[:2], lse, *a[2:])
    for junk in (math.nan, math.inf):
        for i in (0, 1):
            b = list(a)
            b[i] = a[i].clone()
            b[i][1] = junk
            o2, l2 = mla.paged_prefill(d, *b)
            rest = [t for t in range(out.shape[0]) if t != 1]
            assert torch.equal(o2[rest], out[rest]) and torch.equal(l2[rest], lse[rest])
            gone = lse.clone()
            gone[1] = -math.inf
            assert torch.equal(mla.paged_weights(d, *b[:2], gone, *b[2:]), mla.paged_weights(d, *a[:2], gone, *a[2:]))
            w2 = mla.paged_weights(d, *b[:2], lse, *b[2:])
            assert bool(torch.isfinite(w2).all())
            if junk != junk:   # (an infinity may also stand for a weight of 2)
                assert torch.equal(w2, mla.paged_weights(d, *a[:2], gone, *a[2:]))
    assert bool(torch.isfinite(w).all())


@pytest.mark.parametrize("heads", [16, 128])
def test_pages_past_four_gigabytes(heads):
    """The request's pages at the end of a cache of 4.7 GB, explicit and absorbed tokens, weights."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(9), d, BF, [(600, 200), (130, 2)], 64)
    used = s["c_cache"].shape[0]
    pages = 72000
    c = torch.zeros(pages, 64, 512, dtype=BF, device="cuda")
    k = torch.zeros(pages, 64, 64, dtype=BF, device="cuda")
    c[-used:], k[-used:] = s["c_cache"].cuda(), s["kpe_cache"].cuda()
    a = sref.on_gpu(s)
    near = mla.paged_prefill(d, *a)
    near_w = mla.paged_weights(d, *a[:2], near[1], *a[2:])
    a[2], a[3] = c, k
    a[4] = torch.where(a[4] >= 0, a[4] + (pages - used), a[4])
    out, lse = mla.paged_prefill(d, *a)
    assert torch.equal(out, near[0]) and torch.equal(lse, near[1])
    assert torch.equal(mla.paged_weights(d, *a[:2], lse, *a[2:]), near_w)


@pytest.mark.parametrize("heads,dims,dtype", [(4, TINY, F32), (16, V3, BF)])
def test_many_requests(heads, dims, dtype):
    """6000 requests, most of them without tokens: more than the plan keeps at hand."""
    d = mla.dims(heads, **dims)
    lens = [(3, 2) if b % 97 == 5 else (2, 1) if b in (0, 5999) else (1 if b % 7 == 0 else 0, 0) for b in range(6000)]
    lens[77] = (0, 150)
    s = sref.step(ref.generator(11), d, dtype, lens, 8, extra_rows=2, lead=1)
    a = sref.on_gpu(s)
    out, lse = mla.paged_prefill(d, *a)
    want = sref.prefill(d, s)
    sref.check_prefill(dtype, out, lse, want)
    want_w, bound = sref.weights(d, s, want[1].nan_to_num(0.0, neginf=-math.inf).float())
    got = mla.paged_weights(d, *a[:2], want[1].nan_to_num(0.0, neginf=-math.inf).float().cuda(), *a[2:]).cpu()
    assert bool(((got.double() - want_w).abs() <= bound).all())


@pytest.mark.parametrize("heads,dtype,page", [(16, BF, 64), (128, BF, 8), (4, F32, 16)])
def test_weights_of_a_decode(heads, dtype, page):
    """Decode's log-sum-exps as they are: the weights of a token sum to its heads."""
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(12), d, dtype, [(500, 1), (0, 1), (63, 1), (1200, 1)], page)
    a = sref.on_gpu(s)
    q, r, c, k, table, lens, _, _, w = a
    _, lse = mla.paged_decode(d, q, r, c, k, table, lens, w)
    got = mla.paged_weights(d, q, r, lse, c, k, table, lens, torch.arange(5, **I32).cuda(), lens - 1, w).cpu()
    want, bound = sref.weights(d, s, lse.cpu())
    assert bool(((got.double() - want).abs() <= bound).all())
    # each lse is within ref.decode_bounds' 2^-17 (1 + mass) + .. of the scores'; masses of these scores stay below 16
    assert bool(((got.double().sum(1) - heads).abs() <= heads * 2.0 ** -10).all())


def test_sixty_four_tokens_and_the_other_kernels():
    """The smallest step that the explicit form may serve, against the CUDA cores."""
    d = mla.dims(16, **V3)
    s = sref.step(ref.generator(13), d, BF, [(0, 64)], 16)
    a = sref.on_gpu(s)
    want = sref.prefill(d, s)
    for rows in (None, 0, 256):
        sref.check_prefill(BF, *mla.paged_prefill(d, *a, key_rows=rows), want)
    mla.set_path_override(1)
    try:
        got = mla.paged_prefill(d, *a)
        assert mla.last_path() == mla.PATH_SIMT
        w = mla.paged_weights(d, *a[:2], got[1], *a[2:])
    finally:
        mla.set_path_override(0)
    sref.check_prefill(BF, *got, want)
    ref_w, bound = sref.weights(d, s, got[1].cpu())
    assert bool(((w.cpu().double() - ref_w).abs() <= bound).all())
