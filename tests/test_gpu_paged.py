"""The paged latent cache on the GPU: tables, cache write and decode against the 64-bit reference,
at the sizes, pages, strides and lengths where they can go wrong, and the three in a row."""
import math

import pytest
import torch

import paged_ref as ref
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

DS = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)
ODD = dict(d_kv=45, d_nope=9, d_rope=6, d_v=11)
F32, BF16 = torch.float32, torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------- tables ----
def run_tables(past, new, free, table, page, n_tokens):
    t = i32(table)
    got = mla.paged_tables(i32(past), i32(new), i32(free), t, page_size=page, n_tokens=n_tokens)
    want = ref.tables(past, new, free, table, page, n_tokens)
    assert t.tolist() == want[0]
    for a, b in zip(got, want[1:]):
        assert a.tolist() == b
    return got


def table_of(past, page, cols, first=1000):
    rows = []
    for b, p in enumerate(past):
        held = -(-min(max(p, 0), cols * page) // page)
        rows.append([first + 100 * b + j for j in range(held)] + [-7] * (cols - held))
    return rows


@pytest.mark.parametrize("past,new,page,pad", [
    ([0], [1], 16, 0),
    ([15, 16, 17, 0], [1, 1, 1, 1], 16, 0),             # ends of pages
    ([5, 0, 31], [0, 0, 0], 16, 4),                      # nothing new, only padding
    ([0, 3, 0, 40, 0], [0, 50, 0, 7, 0], 8, 5),          # empty requests between
    ([100, 7, 9], [33, 1, 64], 7, 0),
    ([0, 0], [1, 1], 1, 1),
])
def test_tables(past, new, page, pad):
    cols = max(-(-(p + n) // page) for p, n in zip(past, new)) + 2
    run_tables(past, new, list(range(500, 0, -1)), table_of(past, page, cols), page, sum(new) + pad)


@pytest.mark.parametrize("n_free", [0, 1, 3, 6])
def test_tables_out_of_pages(n_free):
    past, new, page = [14, 0, 30, 5], [10, 9, 40, 1], 8
    run_tables(past, new, list(range(n_free)), table_of(past, page, 12), page, sum(new))


def test_tables_clamps():
    # a table row too short, too few token rows, negative lengths, a past above the row
    run_tables([10, 60, -3, 400], [30, 20, 4, 5], list(range(90)), table_of([10, 60, -3, 400], 8, 8), 8, 59)
    run_tables([10, 3], [9, 9], list(range(90)), table_of([10, 3], 8, 8), 8, 5)
    run_tables([4, 4], [-5, 3], list(range(9)), table_of([4, 4], 8, 3), 8, 6)
    run_tables([12], [3], list(range(9)), [[5, -1, 0]], 8, 3)   # a held page without an id


def test_tables_empty():
    got = mla.paged_tables(i32([]), i32([]), i32([3, 4]), torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                           page_size=8, n_tokens=3)
    assert got.cu_tokens.tolist() == [0] and got.counts.tolist() == [0, 0] and got.slots.tolist() == [-1] * 3
    got = mla.paged_tables(i32([8]), i32([0]), i32([]), i32([[1, 2]]), page_size=8, n_tokens=0)
    assert got.kv_lens.tolist() == [8] and got.slots.numel() == 0


def test_arrays_at_any_word():
    """Index arrays that are slices: 4-byte aligned only."""
    past, new, free = i32([9, 3, 30]), i32([9, 2, 3]), i32(list(range(70, 90)))
    out = [torch.zeros(n + 1, dtype=torch.int32, device="cuda")[1:] for n in (2, 3, 5, 5, 2)]
    table = torch.full((13,), -1, dtype=torch.int32, device="cuda")[1:].view(2, 6)
    table[0, 0] = 5
    table[1, :4] = i32([1, 2, 3, 4])
    want = ref.tables([3, 30], [2, 3], list(range(73, 90)), table.tolist(), 8, 5)
    mla.paged_tables(past[1:], new[1:], free[3:], table, page_size=8, kv_lens=out[0], cu_tokens=out[1], slots=out[2],
                     positions=out[3], counts=out[4])
    assert [table.tolist()] + [o.tolist() for o in out] == list(want)
    d, t = decode_case(DS, 16, BF16, [40, 90], 16)
    dev = [x.cuda() for x in t]
    a = mla.paged_decode(d, *dev)
    odd = torch.zeros(dev[4].numel() + 1, dtype=torch.int32, device="cuda")[1:].view_as(dev[4]).copy_(dev[4])
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")[1:].copy_(dev[5])
    b = mla.paged_decode(d, *dev[:4], odd, lens, dev[6])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tables_many_requests():
    g = ref.generator(11)
    B, page = 2500, 16
    past = torch.randint(0, 70, (B,), generator=g).tolist()
    new = torch.randint(0, 9, (B,), generator=g).tolist()
    table = [[(b * 8 + j) if j < -(-p // page) else -1 for j in range(8)] for b, p in enumerate(past)]
    run_tables(past, new, list(range(30000, 33000)), table, page, sum(new) + 17)


def test_tables_most_requests():
    B, page = 16384, 4
    past, new = [b % 5 for b in range(B)], [1] * B
    table = [[b if j < -(-p // page) else -1 for j in range(2)] for b, p in enumerate(past)]
    run_tables(past, new, list(range(100000, 100000 + B)), table, page, B)


def test_tables_long_prompt():
    run_tables([0, 5], [20000, 3000], list(range(4000)), table_of([0, 5], 7, 3000), 7, 23000)


# ----------------------------------------------------------------------- append ----
def check_append(dims, dtype, n, page, pages, positions, slots=None, wide=None, seed=0, base=10000.0):
    d = mla.dims(2, **dims, rope_base=base)
    g = ref.generator(seed)
    width = wide or (d.d_kv + d.d_rope)
    kv = torch.randn(n, width, generator=g).to(dtype).cuda()
    c, k = kv[:, :d.d_kv], kv[:, width - d.d_rope:]
    w = (1 + 0.2 * torch.randn(d.d_kv, generator=g)).to(dtype).cuda()
    if slots is None:
        slots = torch.randperm(pages * page, generator=g)[:n].tolist()
    c0 = torch.full((pages, page, d.d_kv), 7.0, dtype=dtype, device="cuda")
    k0 = torch.full((pages, page, d.d_rope), 7.0, dtype=dtype, device="cuda")
    mla.paged_append(d, c, k, w, i32(slots), i32(positions), c0, k0)
    rc = torch.full((pages * page, d.d_kv), 7.0, dtype=torch.float64)
    rk = torch.full((pages * page, d.d_rope), 7.0, dtype=torch.float64)
    bc, bk = torch.zeros_like(rc), torch.zeros_like(rk)
    h = ref.half_step(dtype)
    keep = [t for t in range(n) if 0 <= slots[t] < pages * page]
    at = [slots[t] for t in keep]
    y = ref.rmsnorm(c.cpu(), w.cpu(), d.rms_eps)[keep]
    z = ref.rope(k.cpu(), torch.tensor(positions), base)[keep]
    rc[at], rk[at] = y, z
    # norm: the mean of d_kv squares is off by a few half steps of fp32 (lane sums of at most 32
    # terms, five halvings), the products by three more: 2^-18 relative is 64 of them
    bc[at] = (h + 2.0 ** -18) * y.abs()
    # rotation: the angle is off by half a step of at most pi and sincospi by two steps, so cos
    # and sin by 2^-22, and the products add three half steps: 2^-21 of |x| + |y|
    half = d.d_rope // 2
    a = k.cpu().double().abs()[keep]
    # On top, the angle pos * f in 64 bits: the reference rounds the frequency f and the product
    # (two half steps of 2^-53), the kernel f and f / 2 pi (two more), each pos * f * 2^-53 radians:
    # nothing at 2^20, 2^31 * 2 * 2^-51 = 2^-19 at the farthest position with f = 2.
    turn = torch.tensor(positions, dtype=torch.float64)[keep].abs()[:, None] * max(1.0, 1 / base) * 2.0 ** -51
    bk[at] = h * z.abs() + (2.0 ** -21 + turn) * (a + torch.cat([a[:, half:], a[:, :half]], 1))
    assert bool(((c0.double().cpu().view_as(rc) - rc).abs() <= bc).all())
    err = (k0.double().cpu().view_as(rk) - rk).abs()
    assert bool((err <= bk).all()), float((err / bk.clamp(min=1e-30)).max())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dims,wide", [(DS, None), (TINY, None), (ODD, 61), (dict(DS, d_kv=1536, d_rope=128), None),
                                       (dict(DS, d_kv=256), 326), (dict(DS, d_kv=768, d_rope=32), 801)])
@pytest.mark.parametrize("n", [1, 5, 130])
def test_append(dtype, dims, wide, n):
    if wide and (wide - dims["d_rope"]) * (4 if dtype == F32 else 2) % 16:
        wide += 8 - (wide - dims["d_rope"]) % 8   # the key band's first row stays on 16 bytes, rows need not
    check_append(dims, dtype, n, 16, 20, [3 * t for t in range(n)], wide=wide, seed=n)


def test_append_far_positions():
    pos = [0, 1, 4095, 65537, 1 << 20, (1 << 24) + 1, 123456789, 2 ** 31 - 1, -1, -70000]
    check_append(DS, F32, len(pos), 4, 8, pos)
    check_append(DS, F32, len(pos), 4, 8, pos, base=0.5)      # frequencies above a turn per position
    check_append(TINY, F32, len(pos), 4, 8, pos, base=5e6)


def test_append_skips_rows_without_a_slot():
    check_append(DS, BF16, 6, 8, 4, [1, 2, 3, 4, 5, 6], slots=[-1, 31, 32, 0, -2 ** 31, 2 ** 31 - 1])
    check_append(TINY, F32, 3, 8, 4, [1, 2, 3], slots=[-1, -1, -1])


def test_append_one_odd_pitch():
    # rows at a pitch that is no multiple of 16 bytes
    d = mla.dims(1, **DS)
    g = ref.generator(5)
    wide = torch.randn(9, 579, generator=g).to(BF16).cuda()
    w = torch.ones(512, dtype=BF16, device="cuda")
    kp = torch.randn(9, 67, generator=g).to(BF16).cuda()[:, :64]
    slots, pos = i32(list(range(9))), i32(list(range(9)))
    a = [torch.zeros(2, 8, n, dtype=BF16, device="cuda") for n in (512, 64, 512, 64)]
    mla.paged_append(d, wide[:, :512], kp, w, slots, pos, a[0], a[1])
    mla.paged_append(d, wide[:, :512].contiguous(), kp.contiguous(), w, slots, pos, a[2], a[3])
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])


def test_append_of_no_tokens():
    d = mla.dims(1, **TINY)
    e = torch.empty(0, 64, device="cuda")
    c, k = torch.ones(2, 4, 64, device="cuda"), torch.ones(2, 4, 16, device="cuda")
    mla.paged_append(d, e, e[:, :16], torch.ones(64, device="cuda"), i32([]), i32([]), c, k)
    assert bool((c == 1).all()) and bool((k == 1).all())


# ----------------------------------------------------------------------- decode ----
def decode_case(dims, heads, dtype, lens, page, seed=0, bad=(), scale=1.0, qscale=1.0, softmax_scale=0.0, **kw):
    d = mla.dims(heads, **dims, softmax_scale=softmax_scale)
    g = ref.generator(seed)
    c, k, table = ref.cache(g, d, dtype, lens, page, scale=scale, **kw)
    for b, j, v in bad:
        table[b, j] = v
    q, r, w = ref.queries(g, d, dtype, len(lens))
    q, r = (q * qscale).to(dtype), (r * qscale).to(dtype)
    return d, (q, r, c, k, table, torch.tensor(lens, dtype=torch.int32), w)


def run_decode(d, t, **kw):
    return mla.paged_decode(d, *[x.cuda() for x in t], **kw)


def check(d, t, **kw):
    out, lse = run_decode(d, t, **kw)
    assert mla.mla_check_device_error() == 0
    ref.check_decode(t[0].dtype, out, lse, ref.decode(d, *t))
    return out, lse


LENS = {
    "one": [1], "two": [2, 1], "page_ends": [15, 16, 17, 31, 32, 33], "empty": [0, 0, 0], "holes": [0, 70, 0, 0, 1, 200, 0],
    "tile_ends": [31, 32, 33, 63, 64, 65, 79, 80, 81, 160, 161], "long": [1500], "ragged": [700, 3, 0, 1100, 64, 257],
}


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("dims,heads,dtype,page", [
    (TINY, 4, F32, 7), (ODD, 3, F32, 16), (DS, 16, F32, 16), (TINY, 4, BF16, 1), (ODD, 17, BF16, 5), (DS, 8, BF16, 12),
    (DS, 16, BF16, 16), (DS, 128, BF16, 64), (DS, 1, BF16, 8), (DS, 20, BF16, 24),
])
def test_decode(name, dims, heads, dtype, page):
    check(*decode_case(dims, heads, dtype, LENS[name], page, seed=heads + page))


@pytest.mark.parametrize("heads", [2, 15, 31, 33, 64, 100, 129, 256])
def test_decode_heads(heads):
    check(*decode_case(DS, heads, BF16, [130, 0, 77], 32, seed=heads))


@pytest.mark.parametrize("page", [1, 2, 8, 16, 40, 48, 128, 512])
def test_decode_pages(page):
    check(*decode_case(DS, 16, BF16, [1, 513, 300], page, seed=page))


def test_decode_many_requests():
    g = ref.generator(9)
    lens = torch.randint(0, 130, (333,), generator=g).tolist()
    check(*decode_case(DS, 4, BF16, lens, 16))
    check(*decode_case(TINY, 2, F32, lens, 16))


@pytest.mark.parametrize("dims,heads,dtype", [(TINY, 4, F32), (DS, 16, BF16), (DS, 128, BF16)])
def test_decode_bad_pages(dims, heads, dtype):
    """Ids outside the cache hold no keys: in the middle, at the end, a whole request's."""
    bad = [(0, 1, -1), (0, 3, 10 ** 6), (1, 0, -2 ** 31), (1, 1, 2 ** 31 - 1), (2, 4, -5), (3, 0, 999)]
    check(*decode_case(dims, heads, dtype, [100, 32, 75, 16], 16, bad=bad))


@pytest.mark.parametrize("dims,heads,dtype", [(TINY, 4, F32), (DS, 16, BF16)])
def test_decode_lengths_outside_the_table(dims, heads, dtype):
    d, t = decode_case(dims, heads, dtype, [48, 32, 5], 16, extra_cols=0)
    lens = torch.tensor([10 ** 6, -4, -2 ** 31], dtype=torch.int32)
    check(d, (*t[:5], lens, t[6]))


@pytest.mark.parametrize("junk", [math.inf, -math.inf, math.nan, 3e38])
@pytest.mark.parametrize("heads,dtype", [(16, BF16), (128, BF16), (4, F32)])
def test_decode_junk_behind_the_end(junk, heads, dtype):
    check(*decode_case(DS, heads, dtype, [1, 37, 90, 81], 64, junk=junk))


@pytest.mark.parametrize("heads,dtype", [(16, BF16), (40, BF16), (128, BF16), (16, F32)])
def test_decode_nan_key_is_seen(heads, dtype):
    """A NaN in a key that is attended to reaches its request's results, and no other's."""
    d, t = decode_case(DS, heads, dtype, [40, 40], 8)
    row = int(t[4][0, 2]) * 8 + 3
    t[2].view(-1, 512)[row, 7] = math.nan
    out, lse = run_decode(d, t)
    assert bool(torch.isnan(lse[0]).all()) and bool(torch.isnan(out[0]).all())
    assert bool(torch.isfinite(lse[1]).all()) and bool(torch.isfinite(out[1]).all())


@pytest.mark.parametrize("heads,dtype", [(16, BF16), (128, BF16), (16, F32)])
def test_decode_growing_maximum(heads, dtype):
    """Keys that grow along the request: the maximum rises all the way, by less than a rescale."""
    d, t = decode_case(DS, heads, dtype, [900, 333], 16, qscale=0.25)
    q, r, c, k, table, lens, w = t
    for b, n in enumerate(lens.tolist()):
        for p in range(n):
            row = int(table[b, p // 16]) * 16 + p % 16
            c.view(-1, 512)[row] *= 0.25 + 6.0 * p / n
    check(d, t)


@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 128, BF16, 16), (DS, 16, BF16, 64), (DS, 72, BF16, 8), (DS, 16, F32, 16),
                                                   (TINY, 4, F32, 7)])
@pytest.mark.parametrize("rise", [6.0, -6.0])
def test_decode_rescaled_maximum(dims, heads, dtype, page, rise):
    """Scores of tens, rising (the accumulator rescaled at most tiles, by more than 2^8) or falling."""
    d, t = decode_case(dims, heads, dtype, [900, 333, 4500 if dims is DS else 70], page)
    q, r, c, k, table, lens, w = t
    for b, n in enumerate(lens.tolist()):
        for p in range(n):
            row = int(table[b, p // page]) * page + p % page
            c.view(-1, d.d_kv)[row] *= 0.25 + abs(rise) * (p if rise > 0 else n - p) / n
    check(d, t)


def test_decode_shared_pages():
    """Requests whose first pages are the same ones (a shared prompt)."""
    d, t = decode_case(DS, 16, BF16, [200, 200, 200], 32)
    t[4][1, :3] = t[4][0, :3]
    t[4][2, :6] = t[4][0, :6]
    check(d, t)


def test_decode_scale():
    check(*decode_case(DS, 16, BF16, [200, 9], 32, softmax_scale=0.02))
    check(*decode_case(TINY, 4, F32, [200, 9], 32, softmax_scale=0.5))


def test_decode_same_bits_and_untouched_inputs():
    d, t = decode_case(DS, 128, BF16, [3000, 1, 0, 700], 64, junk=1.0)
    dev = [x.cuda() for x in t]
    keep = [x.clone() for x in dev]
    ws = mla.paged_decode_workspace(d, dev[2], dev[4])
    first = [x.clone() for x in mla.paged_decode(d, *dev, workspace=ws)]
    ws.fill_(255)   # nothing in it is expected to hold anything
    for _ in range(3):
        for a, b in zip(first, mla.paged_decode(d, *dev, workspace=ws)):
            assert torch.equal(a, b)
    for a, b in zip(keep, dev):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 128, BF16, 64), (DS, 130, BF16, 16), (DS, 5, BF16, 8), (DS, 7, F32, 3),
                                                   (ODD, 17, BF16, 4)])
def test_decode_writes_its_outputs_only(dims, heads, dtype, page):
    """Outputs and a workspace of exactly the queried size, inside buffers whose other bytes stay."""
    lens = [150, 0, 1, 333, 64, 65, 7]
    d, t = decode_case(dims, heads, dtype, lens, page)
    dev = [x.cuda() for x in t]
    want = mla.paged_decode(d, *dev)
    n = mla.paged_decode_workspace(d, dev[2], dev[4]).numel()
    room = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")

    def inside(shape, ty):
        x = torch.full((math.prod(shape) + 512,), 7.0, dtype=ty, device="cuda")
        return x, x[256:256 + math.prod(shape)].view(shape)

    ob, out = inside((len(lens), heads, d.d_v), dtype)
    lb, lse = inside((len(lens), heads), F32)
    mla.paged_decode(d, *dev, out=out, lse=lse, workspace=room[4096:4096 + n])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert bool((room[:4096] == 0xA5).all()) and bool((room[4096 + n:] == 0xA5).all())
    for x in (ob, lb):
        assert bool((x[:256] == 7).all()) and bool((x[-256:] == 7).all())


def test_far_pages():
    """Slots whose element and byte offsets pass 2^31 and 2^32: written and attended to at a large
    cache's end, the pages at its start holding others' tokens."""
    d = mla.dims(16, **DS)
    pages, page = 140000, 64                       # 4.6e9 latent elements
    c = torch.empty(pages, page, 512, dtype=BF16, device="cuda")
    k = torch.empty(pages, page, 64, dtype=BF16, device="cuda")
    ids = [pages - 1, 3, pages - 70, 70000, pages - 2]
    c[[3, 70000]], k[[3, 70000]] = 0, 0
    g = ref.generator(31)
    n = 4 * page + 9
    x = torch.randn(n, 576, generator=g).to(BF16)
    w_norm = torch.ones(512, dtype=BF16)
    table = torch.tensor([ids], dtype=torch.int32)
    slots = [ids[p // page] * page + p % page for p in range(n)]
    mla.paged_append(d, x.cuda()[:, :512], x.cuda()[:, 512:], w_norm.cuda(), i32(slots), i32(list(range(n))), c, k)
    q, r, w = ref.queries(g, d, BF16, 1)
    lens = torch.tensor([n], dtype=torch.int32)
    out, lse = mla.paged_decode(d, q.cuda(), r.cuda(), c, k, table.cuda(), lens.cuda(), w.cuda())
    cc, kk = c[ids].cpu(), k[ids].cpu()
    y = ref.rmsnorm(x[:, :512], w_norm, d.rms_eps)
    assert float((cc.view(-1, 512)[:n].double() - y).abs().max()) <= 2.0 ** -8 * float(y.abs().max()) * 1.01
    ref.check_decode(BF16, out, lse, ref.decode(d, q, r, cc, kk, torch.arange(5, dtype=torch.int32)[None], lens, w))
    del c, k
    # the CUDA-core kernels, fp32
    d = mla.dims(2, **TINY)
    pages, page = 40_000_000 // 5, 5               # 2.6e9 latent elements
    c = torch.empty(pages, page, 64, device="cuda")
    k = torch.empty(pages, page, 16, device="cuda")
    ids = [pages - 1, 1, pages - 5]
    x = torch.randn(13, 80, generator=g)
    slots = [ids[p // page] * page + p % page for p in range(13)]
    mla.paged_append(d, x.cuda()[:, :64], x.cuda()[:, 64:], torch.ones(64, device="cuda"), i32(slots), i32(list(range(13))), c, k)
    q, r, w = ref.queries(g, d, F32, 1)
    lens = torch.tensor([13], dtype=torch.int32)
    out, lse = mla.paged_decode(d, q.cuda(), r.cuda(), c, k, i32([ids]), lens.cuda(), w.cuda())
    ref.check_decode(F32, out, lse, ref.decode(d, q, r, c[ids].cpu(), k[ids].cpu(), torch.arange(3, dtype=torch.int32)[None], lens, w))


def test_decode_batch_of_none():
    d, t = decode_case(TINY, 4, F32, [5], 4)
    dev = [x.cuda() for x in t]
    out, lse = mla.paged_decode(d, dev[0][:0], dev[1][:0], dev[2], dev[3], dev[4][:0], dev[5][:0], dev[6])
    assert out.shape == (0, 4, 32) and lse.shape == (0, 4)


def test_decode_on_another_stream():
    d, t = decode_case(DS, 16, BF16, [900, 40], 16)
    dev = [x.cuda() for x in t]
    want = mla.paged_decode(d, *dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = mla.paged_decode(d, *dev, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 128, BF16, 64), (DS, 16, F32, 16), (TINY, 4, F32, 7)])
def test_inputs_written_by_the_kernel_in_front(dims, heads, dtype, page):
    """Every input rewritten in place right before the call, call after call, has the bits of a call that
    finds them settled."""
    cases = [decode_case(dims, heads, dtype, lens, page, seed=k)[1] for k, lens in enumerate(([700, 30, 1], [64, 700, 9], [5, 8, 700]))]
    d = decode_case(dims, heads, dtype, [1], page)[0]
    cases = [[x.cuda() for x in t] for t in cases]
    rows = max(t[2].shape[0] for t in cases)
    want = [mla.paged_decode(d, *t) for t in cases]
    live = [torch.zeros(*([rows] if i in (2, 3) else [x.shape[0]]), *x.shape[1:], dtype=x.dtype, device="cuda")
            for i, x in enumerate(cases[0])]
    ws = mla.paged_decode_workspace(d, live[2], live[4])
    got = []
    torch.cuda.synchronize()
    for _ in range(4):
        for t in cases:
            for x, y in zip(live, t):
                x[:y.shape[0]].copy_(y)
            got.append(mla.paged_decode(d, *live, workspace=ws))
    torch.cuda.synchronize()
    for k, (o, l) in enumerate(got):
        assert torch.equal(o, want[k % 3][0]) and torch.equal(l, want[k % 3][1]), k


@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 16, BF16, 16), (DS, 128, BF16, 64), (TINY, 4, F32, 5)])
def test_decode_same_page_twice(dims, heads, dtype, page):
    """A request whose table names one page several times: its keys count as often."""
    d, t = decode_case(dims, heads, dtype, [5 * page, 3 * page + 2, 9], page)
    t[4][0, 1:4] = t[4][0, 0]
    t[4][1, 2] = t[4][0, 0]
    check(d, t)


@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 128, BF16, 64), (DS, 16, F32, 16)])
def test_decodes_on_two_streams_at_once(dims, heads, dtype, page):
    """Calls that run side by side, a workspace each, have the bits of calls alone."""
    cases = [decode_case(dims, heads, dtype, lens, page, seed=k) for k, lens in enumerate(([1500, 3, 800, 64], [70] * 90))]
    dev = [(d, [x.cuda() for x in t]) for d, t in cases]
    want = [mla.paged_decode(d, *x) for d, x in dev]
    ws = [mla.paged_decode_workspace(d, x[2], x[4]) for d, x in dev]
    streams = [torch.cuda.Stream() for _ in dev]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(12):
        for k, (d, x) in enumerate(dev):
            with torch.cuda.stream(streams[k]):
                got[k].append(mla.paged_decode(d, *x, workspace=ws[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for o, l in got[k]:
            assert torch.equal(o, want[k][0]) and torch.equal(l, want[k][1])
    assert mla.mla_check_device_error(None) == 0


def test_decode_agrees_with_the_dense_decode():
    """One length for all: the paged decode and the dense split-KV decode of the same cache."""
    d, t = decode_case(DS, 128, BF16, [640, 640], 64)
    q, r, c, k, table, lens, w = [x.cuda() for x in t]
    rows = (table[:, :10].long()[:, :, None] * 64 + torch.arange(64, device="cuda")).view(2, 640)
    o1, l1 = mla.paged_decode(d, q, r, c, k, table, lens, w)
    o2, l2 = mla.decode_splitkv(d, q, r, c.view(-1, 512)[rows].contiguous(), k.view(-1, 64)[rows].contiguous(), w, n_splits=3)
    assert float((l1 - l2).abs().max()) < 1e-3                      # the dense path's documented precision
    assert float((o1.float() - o2.float()).norm() / o1.float().norm()) < 1e-2


def test_refusals_on_the_device():
    d, t = decode_case(TINY, 4, F32, [5, 9], 4)
    dev = [x.cuda() for x in t]
    for i, bad, kind, match in ((0, dev[0][:1], ValueError, "q_pe: .* elements|q_pe: shape"), (1, dev[1].double(), TypeError, "q_pe: dtype"),
                                (2, dev[2][:, :3], ValueError, "c_cache: tensors must be contiguous"), (3, dev[3][:-1], ValueError, "kpe_cache"),
                                (4, dev[4].long(), TypeError, "block_table: dtype"), (5, dev[5][:1], ValueError, "kv_lens"),
                                (6, dev[6][:-1], ValueError, "w_kv_b"), (5, t[5], ValueError, "kv_lens: on cpu"),
                                (1, dev[1].view(2, 16, 4), ValueError, "q_pe: shape")):
        args = list(dev)
        args[i] = bad
        with pytest.raises(kind, match=match):
            mla.paged_decode(d, *args)
    with pytest.raises(mla.MlaError, match="WORKSPACE"):
        mla.paged_decode(d, *dev, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mla.MlaError, match="ALIAS"):
        mla.paged_decode(d, *dev, out=dev[0].view(-1)[:2 * 4 * 32].view(2, 4, 32))
    i = i32([1, 2])
    with pytest.raises(TypeError, match="past_lens"):
        mla.paged_tables(None, i, i, dev[4], page_size=4, n_tokens=2)
    with pytest.raises(ValueError, match="n_tokens or slots"):
        mla.paged_tables(i, i, i, dev[4], page_size=4)
    with pytest.raises(mla.MlaError, match="SHAPE"):
        mla.paged_tables(i, i, i, dev[4], page_size=0, n_tokens=2)
    rows = torch.zeros(2, 80, device="cuda")
    with pytest.raises(ValueError, match="adjacent"):
        mla.paged_append(d, rows[:, :64], torch.zeros(16, 2, device="cuda").t(), rows[0, :64], i, i, dev[2], dev[3])
    with pytest.raises(ValueError, match="slots"):
        mla.paged_append(d, rows[:, :64], rows[:, 64:], rows[0, :64].contiguous(), i[:1], i, dev[2], dev[3])


# --------------------------------------------------------------- the three in a row ----
@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 16, BF16, 16), (TINY, 4, F32, 5)])
def test_serving_steps_captured(dims, heads, dtype, page):
    """Prompts, then decode steps captured once and replayed while the requests grow: each
    step's result is the reference's over everything written so far."""
    d = mla.dims(heads, **dims)
    g = ref.generator(21)
    B, cols, pages = 3, 12, 40
    prompts = [17, 0, 2 * page]
    dev = dict(device="cuda")
    past, table = i32([0] * B), torch.full((B, cols), -1, dtype=torch.int32, **dev)
    free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    c = torch.full((pages, page, d.d_kv), math.nan, dtype=dtype, **dev)
    k = torch.full((pages, page, d.d_rope), math.nan, dtype=dtype, **dev)
    w_norm = (1 + 0.1 * torch.randn(d.d_kv, generator=g)).to(dtype).cuda()
    history = [torch.zeros(0, d.d_kv + d.d_rope) for _ in range(B)]

    def rows(lens):
        x = torch.randn(sum(lens), d.d_kv + d.d_rope, generator=g).to(dtype)
        for b, part in enumerate(x.split(lens)):
            history[b] = torch.cat([history[b], part.float()])
        return x.cuda()

    x = rows(prompts)
    t = mla.paged_tables(past, i32(prompts), free, table, page_size=page, n_tokens=sum(prompts) + 2)
    pad = torch.cat([x, x.new_full((2, x.shape[1]), math.nan)])
    mla.paged_append(d, pad[:, :d.d_kv], pad[:, d.d_kv:], w_norm, t.slots, t.positions, c, k)
    assert t.counts[0].item() == t.counts[1].item()
    past.copy_(t.kv_lens)
    free = free[int(t.counts[0]):].contiguous()
    # the step, captured: lengths, tables and inputs live in fixed tensors
    new, step = i32([1] * B), torch.zeros(B, d.d_kv + d.d_rope, dtype=dtype, **dev)
    q0, r0, w = [v.cuda() for v in ref.queries(g, d, dtype, B)]
    pool = torch.zeros(pages, dtype=torch.int32, **dev)
    out, lse = torch.empty(B, heads, d.d_v, dtype=dtype, **dev), torch.empty(B, heads, **dev)
    ws = mla.paged_decode_workspace(d, c, table)
    bufs = dict(kv_lens=i32([0] * B), cu_tokens=i32([0] * (B + 1)), slots=i32([0] * B), positions=i32([0] * B),
                counts=i32([0, 0]))

    def one():
        s = mla.paged_tables(past, new, pool, table, page_size=page, **bufs)
        mla.paged_append(d, step[:, :d.d_kv], step[:, d.d_kv:], w_norm, s.slots, s.positions, c, k)
        mla.paged_decode(d, q0, r0, c, k, table, s.kv_lens, w, out=out, lse=lse, workspace=ws)

    pool[:free.numel()].copy_(free)
    keep_table = table.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            one()
    torch.cuda.current_stream().wait_stream(side)
    table.copy_(keep_table)
    used = 0
    for _ in range(page + 3):
        step.copy_(rows([1] * B))
        rest = free[used:]
        pool.fill_(0)
        pool[:rest.numel()].copy_(rest)
        graph.replay()
        used += int(bufs["counts"][0])
        past.copy_(bufs["kv_lens"])
        lens = [h.shape[0] for h in history]
        assert bufs["kv_lens"].tolist() == lens
        # the reference from the history, in the cache's type
        cc = [ref.rmsnorm(h[:, :d.d_kv], w_norm.cpu(), d.rms_eps).to(dtype) for h in history]
        kk = [ref.rope(h[:, d.d_kv:], torch.arange(h.shape[0]), d.rope_base).to(dtype) for h in history]
        most = max(lens)
        dc = torch.stack([torch.cat([v, v.new_zeros(most - v.shape[0], v.shape[1])]) for v in cc])
        dk = torch.stack([torch.cat([v, v.new_zeros(most - v.shape[0], v.shape[1])]) for v in kk])
        want = list(ref.decode(d, q0.cpu(), r0.cpu(), dc, dk, torch.arange(B)[:, None], lens, w.cpu()))
        # a rounding of the cache that lands on the other side of a tie moves a key by a step:
        # far inside the bounds' mass term for bf16, a half step of fp32 for fp32
        ref.check_decode(dtype, out, lse, want)


def test_two_captured_decodes_with_a_workspace_each():
    d, t1 = decode_case(DS, 16, BF16, [500, 20], 16, seed=1)
    _, t2 = decode_case(DS, 16, BF16, [33, 1000], 16, seed=2)
    a, b = [x.cuda() for x in t1], [x.cuda() for x in t2]
    wa, wb = mla.paged_decode(d, *a), mla.paged_decode(d, *b)
    graphs, outs, keep = [], [], []
    for t in (a, b):
        o, l = torch.empty_like(wa[0]), torch.empty_like(wa[1])
        ws = mla.paged_decode_workspace(d, t[2], t[4])
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            mla.paged_decode(d, *t, out=o, lse=l, workspace=ws)
        graphs.append(g)
        outs.append((o, l))
        keep.append(ws)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, (wa, wb)):
        assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("dims,heads,dtype,page", [(DS, 128, BF16, 64), (TINY, 4, F32, 7)])
def test_captured_behind_a_join_of_streams(dims, heads, dtype, page):
    """Captured calls whose inputs come from two streams that meet right in front of them: the first kernel of
    each call depends on both."""
    d, t = decode_case(dims, heads, dtype, [300, 70, 1], page)
    dev = [x.cuda() for x in t]
    q, r, c, k, table, lens, w = dev
    src_q, src_c = q.clone(), c.clone()
    lens_src, past = lens.clone(), torch.zeros_like(lens)
    free = torch.arange(64, dtype=torch.int32, device="cuda")
    tab2 = torch.full((3, table.shape[1] + 1), -1, dtype=torch.int32, device="cuda")
    ws = mla.paged_decode_workspace(d, c, table)
    n = int(lens.sum())
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            c.copy_(src_c)
            past.copy_(lens_src * 0)
        q.copy_(src_q)
        here.wait_stream(side)
        tables = mla.paged_tables(past, lens_src, free, tab2, page_size=page, n_tokens=n)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            r2 = r * 1
        here.wait_stream(side)
        return tables, mla.paged_decode(d, q, r2, c, k, table, lens, w, workspace=ws)

    want = [x.clone() for x in step()[1]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tables, (out, lse) = step()
    for scale in (1.0, 0.5, 1.0):
        src_q.copy_(t[0].cuda() * scale)
        q.zero_(), c.zero_(), out.fill_(5), lse.fill_(5), tables.kv_lens.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tables.kv_lens, lens)
        if scale == 1.0:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        else:
            got = mla.paged_decode(d, src_q, r, c, k, table, lens, w)
            assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
