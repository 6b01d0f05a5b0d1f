"""Calls on a stream of the caller's: everything that a call allocates belongs to that stream, so that no other
work gets a workspace which the call's kernels still use; results are those of a call on the current stream."""
import pytest
import torch
from torch.overrides import TorchFunctionMode

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import configs, inputs, mla

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


class Allocations(TorchFunctionMode):
    """The streams that were current when tensors were made, and the tensors' addresses."""
    def __init__(self):
        super().__init__()
        self.streams, self.made = set(), []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func in (torch.empty, torch.zeros, torch.empty_like, torch.zeros_like, torch.full):
            self.streams.add(torch.cuda.current_stream().cuda_stream)
            self.made.append((out.data_ptr(), out.numel() * out.element_size()))
        return out


def flat(result):
    if isinstance(result, dict):
        return [result[k] for k in sorted(result)]
    return list(result) if isinstance(result, tuple) else [result]


def prefill():
    cfg = configs.TINY
    t = {k: v.cuda() for k, v in inputs.prefill_inputs(cfg).items()}
    return mla.dims_of(cfg), [t[k] for k in ("q_nope", "q_pe", "c_kv", "k_pe", "w_kv_b", "rms_w")]


def backward():
    d, t = prefill()
    out, lse = mla.latent_attn_fwd(d, *t)
    dout = torch.ones_like(out)
    torch.cuda.synchronize()
    return lambda **kw: mla.latent_attn_bwd(d, *t, out, lse, dout, **kw)


def paged(dims, heads, dtype):
    d = mla.dims(heads, **dims)
    g = ref.generator(4)
    c, k, table = ref.cache(g, d, dtype, [900, 40], 16)
    q, r, w = ref.queries(g, d, dtype, 2)
    t = [x.cuda() for x in (q, r, c, k, table, torch.tensor([900, 40], dtype=torch.int32), w)]
    return lambda **kw: mla.paged_decode(d, *t, **kw)


def dense(fn, heads, **more):
    d = mla.dims(heads, 512, 128, 64, 128)
    g = ref.generator(5)
    q, r, w = (x.cuda() for x in ref.queries(g, d, BF16, 2))
    c, k = torch.randn(2, 300, 512, generator=g).to(BF16).cuda(), torch.randn(2, 300, 64, generator=g).to(BF16).cuda()
    return lambda **kw: fn(d, q, r, c, k, w, n_splits=2, **more, **kw)


def tables():
    i = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    free = torch.arange(20, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    return lambda **kw: mla.paged_tables(i, i, free, table, page_size=4, n_tokens=9, **kw)


def rows(bwd):
    g = ref.generator(6)
    x, w, dy = torch.randn(77, 96, generator=g).cuda(), torch.randn(96, generator=g).cuda(), torch.randn(77, 96, generator=g).cuda()
    return (lambda **kw: mla.rmsnorm_bwd(x, w, dy, **kw)) if bwd else (lambda **kw: mla.rmsnorm(x, w, **kw))


def combine():
    g = ref.generator(7)
    po, pl = torch.randn(3, 50, 16, generator=g).cuda(), torch.randn(3, 50, generator=g).cuda()
    return lambda **kw: mla.lse_combine(po, pl, **kw)


DS = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)
CALLS = {
    "latent_attn_fwd": lambda: (lambda d, t: lambda **kw: mla.latent_attn_fwd(d, *t, **kw))(*prefill()),
    "absorbed_attn_fwd": lambda: (lambda d, t: lambda **kw: mla.absorbed_attn_fwd(d, *t, **kw))(*prefill()),
    "latent_attn_bwd": backward,
    "decode_splitkv": lambda: dense(mla.decode_splitkv, 128),
    "tpla_decode": lambda: dense(mla.tpla_decode, 128, n_shards=2),
    "rmsnorm": lambda: rows(False), "rmsnorm_bwd": lambda: rows(True), "lse_combine": combine, "paged_tables": tables,
    "paged_decode_tc": lambda: paged(DS, 16, BF16), "paged_decode_simt": lambda: paged(TINY, 4, F32),
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
        # the current stream asks for memory of the same sizes at once
        again = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda") for _, n in list(seen.made)]
    here = torch.cuda.current_stream().cuda_stream
    assert seen.made[:len(again)] and s.cuda_stream in seen.streams and seen.streams <= {s.cuda_stream, here}
    for x in again:
        lo, hi = x.data_ptr(), x.data_ptr() + x.numel()
        assert all(hi <= p or p + n <= lo for p, n in seen.made[:len(again)])
    assert torch.cuda.current_stream().cuda_stream == here
    s.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_append_on_a_stream():
    d = mla.dims(1, **TINY)
    x, w = torch.randn(5, 80, device="cuda"), torch.ones(64, device="cuda")
    i = torch.arange(5, dtype=torch.int32, device="cuda")
    a = [torch.zeros(2, 4, n, device="cuda") for n in (64, 16, 64, 16)]
    mla.paged_append(d, x[:, :64], x[:, 64:], w, i, i, a[0], a[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mla.paged_append(d, x[:, :64], x[:, 64:], w, i, i, a[2], a[3], stream=s)
    s.synchronize()
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])


def test_the_default_stream_by_its_handles():
    call = CALLS["paged_decode_tc"]()
    want = call()
    for handle in (0, 1):   # the legacy default stream
        got = call(stream=handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_on_a_forked_stream():
    """A call on a side stream inside a capture: its workspace is the graph's, and replays have the call's bits."""
    call = CALLS["paged_decode_tc"]()
    want = [x.clone() for x in call()]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = call(stream=side)
        here.wait_stream(side)
    for _ in range(3):
        for x in got:
            x.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
