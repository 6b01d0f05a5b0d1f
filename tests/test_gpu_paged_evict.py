"""mla_paged_evict on a GPU against a plain eviction, and a run of tables, append, prefill, weights and eviction together."""
import math
import random

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32)


def case(seed, B, cols, page, lens, kinds):
    g = ref.generator(seed)
    table = torch.randperm(B * cols, generator=g).to(torch.int32).view(B, cols)
    table = torch.where(torch.rand(B, cols, generator=g) < 0.1, torch.tensor(-1, **I32), table)
    w = torch.exp(2 * torch.randn(B, cols, generator=g))
    if "ties" in kinds:
        w = (w * 2).round() / 2
    if "odd" in kinds:
        odd = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, -1.5, 1e-40, -1e-40])
        pick = torch.randint(0, 8, (B, cols), generator=g)
        w = torch.where(torch.rand(B, cols, generator=g) < 0.4, odd[pick], w)
    return torch.tensor(lens, **I32), table, w


def same(a, b):
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("kinds", ["plain", "ties", "odd ties"])
@pytest.mark.parametrize("B,cols,page,keep,first,last", [
    (1, 1, 16, 0, 0, 1), (1, 40, 8, 10, 0, 1), (7, 33, 64, 12, 2, 3), (5, 130, 7, 0, 0, 1), (3, 700, 16, 333, 1, 40),
    (2, 5000, 16, 1000, 4, 64), (300, 20, 32, 7, 1, 2), (3, 8192, 1, 4000, 0, 1),
    (2, 8200, 4, 4001, 3, 9), (2, 30001, 2, 7000, 100, 17), (1, 66000, 3, 20000, 5, 64), (2, 70001, 1, 70000, 0, 1), (1, 140000, 1, 500, 0, 1), (4, 20, 32, 100, 0, 1), (4, 20, 32, 3, 30, 1), (4, 20, 32, 3, 0, 30),
])
def test_against_a_plain_eviction(kinds, B, cols, page, keep, first, last):
    rng = random.Random(B * cols + keep)
    lens = [rng.choice([0, 1, cols * page, rng.randint(0, cols * page), cols * page + 99, -3]) for _ in range(B)]
    lens[0] = cols * page - rng.randint(0, page - 1)
    kv, table, w = case(B + cols, B, cols, page, lens, kinds)
    for room in (B * cols, 5, 0):
        want = sref.evict(kv, table, w, page, keep, first, last, room)
        freed = torch.full((room,), -9, **I32).cuda()
        t, x = table.cuda(), w.cuda()
        to, wo = torch.empty_like(t), torch.empty_like(x)
        e = mla.paged_evict(kv.cuda(), t, x, page_size=page, keep_pages=keep, first_pages=first, last_pages=last,
                            table_out=to, weights_out=wo, freed=freed)
        assert e.counts.tolist() == want[3]
        assert torch.equal(to.cpu(), want[0]) and same(wo.cpu(), want[1])
        assert freed.tolist() == want[2] + [-9] * (room - len(want[2]))
        assert torch.equal(t.cpu(), table) and same(x.cpu(), w)
        e = mla.paged_evict(kv.cuda(), t, x, page_size=page, keep_pages=keep, first_pages=first, last_pages=last, freed=freed)
        assert torch.equal(t.cpu(), want[0]) and same(x.cpu(), want[1])   # in place


def test_no_requests():
    e = mla.paged_evict(torch.zeros(0, **I32).cuda(), torch.zeros(0, 4, **I32).cuda(), torch.zeros(0, 4).cuda(), page_size=8,
                        keep_pages=1)
    assert e.counts.tolist() == [0, 0] and e.freed.numel() == 0


@pytest.mark.parametrize("heads,dtype,page", [(16, torch.bfloat16, 16), (128, torch.bfloat16, 32), (4, torch.float32, 5)])
def test_a_server_with_a_budget(heads, dtype, page):
    """Prompts in chunks, then tokens, over a cache that is held to a budget: tables, append, prefill, weights and
    eviction in turn.  What each prefill gives is held to 64 bits over the pages that are left, the weights too, the
    pages that go are those of a plain eviction, and no page is lost or held twice."""
    d = mla.dims(heads, 512, 128, 64, 128)
    g = ref.generator(heads)
    B, pages, cols, keep = 3, 60, 24, 5
    c = torch.zeros(pages, page, 512, dtype=dtype).cuda()
    k = torch.zeros(pages, page, 64, dtype=dtype).cuda()
    table = torch.full((B, cols), -1, **I32).cuda()
    free = torch.randperm(pages, generator=g).to(torch.int32).tolist()
    kv = torch.zeros(B, **I32).cuda()
    held_weights = torch.zeros(B, cols).cuda()
    w = (torch.randn(heads * 256, 512, generator=g) / math.sqrt(512)).to(dtype)
    rms = torch.ones(512, dtype=dtype).cuda()
    evicted = 0
    for new in ([page * 3 + 1, 0, 2], [page * 4, page + 3, 1], [1, page * 5, 1], [1, 1, 1], [2, 4, 1], [1, 1, page]):
        n = sum(new)
        t = mla.paged_tables(kv, torch.tensor(new, **I32).cuda(), torch.tensor(free, **I32).cuda(), table, page_size=page, n_tokens=n)
        free = free[int(t.counts[0]):]
        kv = t.kv_lens
        latent = torch.randn(n, 512, generator=g).to(dtype).cuda()
        band = torch.randn(n, 64, generator=g).to(dtype).cuda()
        mla.paged_append(d, latent, band, rms, t.slots, t.positions, c, k)
        q, r = (torch.randn(n, heads, x, generator=g).to(dtype) for x in (128, 64))
        a = [q.cuda(), r.cuda(), c, k, table, kv, t.cu_tokens, t.positions, w.cuda()]
        out, lse = mla.paged_prefill(d, *a)
        s = dict(zip(sref.NAMES, [x.cpu() for x in a]))
        want = sref.prefill(d, s)
        sref.check_prefill(dtype, out, lse, want)
        before = held_weights.cpu()
        held_weights = mla.paged_weights(d, *a[:2], lse, *a[2:], prior=held_weights)
        ref_w, bound = sref.weights(d, s, lse.cpu(), before)
        assert bool(((held_weights.cpu().double() - ref_w).abs() <= bound).all())
        plan = sref.evict(kv.cpu(), table.cpu(), held_weights.cpu(), page, keep, 1, 1, B * cols)
        e = mla.paged_evict(kv, table, held_weights, page_size=page, keep_pages=keep, first_pages=1)
        gone = e.freed[:int(e.counts[0])].tolist()
        assert gone == plan[2] and torch.equal(table.cpu(), plan[0])
        evicted += len(gone)
        free += gone
        live = [i for row in table.tolist() for i in row if i >= 0]
        assert sorted(free + live) == list(range(pages))
        for b in range(B):
            assert sum(i >= 0 for i in table[b].tolist()) <= max(keep, 1)
    assert evicted >= 5   # the first request grows to 8 pages, the second to 7, of which 5 stay each
