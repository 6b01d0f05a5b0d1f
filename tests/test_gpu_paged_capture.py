"""A serving step captured once with the upkeep of its free list and lengths on the device, replayed without a host
read in between."""
import pytest
import torch

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dims,heads,dtype,page", [
    (dict(d_kv=512, d_nope=128, d_rope=64, d_v=128), 16, BF16, 8), (dict(d_kv=512, d_nope=128, d_rope=64, d_v=128), 128, BF16, 16),
    (dict(d_kv=64, d_nope=32, d_rope=16, d_v=32), 4, F32, 5)])
def test_replays_without_the_host(dims, heads, dtype, page):
    d = mla.dims(heads, **dims)
    g = ref.generator(page + heads)
    B, cols, pages, steps, width = 4, 9, 40, 2 * page + 3, d.d_kv + d.d_rope
    i32 = dict(dtype=torch.int32, device="cuda")
    start = [0, 3, page, 2 * page - 1]
    held = [-(-n // page) for n in start]
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table_host = torch.full((B, cols), -1, dtype=torch.int32)
    used = 0
    for b, n in enumerate(held):
        table_host[b, :n] = order[used:used + n]
        used += n
    n_free = pages - used
    free = order[used:].cuda()
    table, past = table_host.cuda(), torch.tensor(start, **i32)
    rows = torch.randn(steps, B, width, generator=g).to(dtype)
    first = torch.randn(B, max(start), width, generator=g).to(dtype)
    w_norm = (1 + 0.1 * torch.randn(d.d_kv, generator=g)).to(dtype).cuda()
    c = torch.zeros(pages, page, d.d_kv, dtype=dtype, device="cuda")
    k = torch.zeros(pages, page, d.d_rope, dtype=dtype, device="cuda")
    for b, n in enumerate(start):
        if n:
            slots = torch.tensor([int(table_host[b, p // page]) * page + p % page for p in range(n)], **i32)
            x = first[b, :n].cuda()
            mla.paged_append(d, x[:, :d.d_kv], x[:, d.d_kv:], w_norm, slots, torch.arange(n, **i32), c, k)
    all_rows, at = rows.cuda(), torch.zeros(1, dtype=torch.long, device="cuda")
    new, ids = torch.ones(B, **i32), torch.arange(n_free, device="cuda")
    q, r, w = (x.cuda() for x in ref.queries(g, d, dtype, B))
    outs = torch.zeros(steps, B, heads, d.d_v, dtype=dtype, device="cuda")
    lses, lens = torch.zeros(steps, B, heads, device="cuda"), torch.zeros(steps, B, **i32)

    def step():
        t = mla.paged_tables(past, new, free, table, page_size=page, n_tokens=B)
        x = all_rows.index_select(0, at)[0]
        mla.paged_append(d, x[:, :d.d_kv], x[:, d.d_kv:], w_norm, t.slots, t.positions, c, k)
        o, l = mla.paged_decode(d, q, r, c, k, table, t.kv_lens, w)
        outs.index_copy_(0, at, o[None])
        lses.index_copy_(0, at, l[None])
        lens.index_copy_(0, at, t.kv_lens[None])
        free.copy_(free[(ids + t.counts[0]).clamp(max=n_free - 1)])   # the list moved up by the pages taken
        past.copy_(t.kv_lens)
        at.add_(1)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    assert mla.mla_check_device_error() == 0
    assert lens.tolist() == [[n + i + 1 for n in start] for i in range(steps)]
    for i in (0, page - 1, steps - 1):   # the reference from everything written up to step i
        hist = [torch.cat([first[b, :n], rows[:i + 1, b]]) for b, n in enumerate(start)]
        most = max(h.shape[0] for h in hist)
        dc, dk = torch.zeros(B, most, d.d_kv, dtype=dtype), torch.zeros(B, most, d.d_rope, dtype=dtype)
        for b, h in enumerate(hist):
            dc[b, :h.shape[0]] = ref.rmsnorm(h[:, :d.d_kv], w_norm.cpu(), d.rms_eps).to(dtype)
            dk[b, :h.shape[0]] = ref.rope(h[:, d.d_kv:], torch.arange(h.shape[0]), d.rope_base).to(dtype)
        want = ref.decode(d, q.cpu(), r.cpu(), dc, dk, torch.arange(B)[:, None], [h.shape[0] for h in hist], w.cpu())
        ref.check_decode(dtype, outs[i], lses[i], want)
