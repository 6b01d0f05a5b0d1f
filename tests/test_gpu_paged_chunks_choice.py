"""Which requests of a step take the explicit form: by the rule on their tokens and keys, and by the room that is left.

A request's rows in the explicit form are the same bits whichever other requests the step has, and those of the absorbed
form others: so each request is run alone with all the room it needs and with none, and its rows in the step have to be the one or
not the one."""
import pytest
import torch

import paged_step_ref as sref
import paged_ref as ref
from test_gpu_paged_chunks import CASES, check_rows, spread
from head_latent_attention_rmsnorm_gb300 import mla

pytestmark = pytest.mark.gpu

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
BF = torch.bfloat16


def rule(heads, lens, key_rows):
    """The requests that go explicit: from 11 r (tiled keys + 64) / (6 keys + 72 r) tokens on, at least 32 of tokens and of
    keys, r query rows an item of the absorbed form; in their order, each that fits in what is left of the rows."""
    tile = 64 if heads <= 64 else 128
    r = tile // heads * heads if heads <= tile else heads / -(-heads // tile)
    left, got = key_rows // 256 * 256, []
    for b, (past, new) in enumerate(lens):
        keys = past + new
        tiled = -(-keys // 128) * 128
        if min(new, keys) >= 32 and new * (6 * keys + 72 * r) >= 11 * r * (tiled + 64) and tiled <= left:
            left -= tiled
            got.append(b)
    return got


def alone(a, cu, b):
    """The step with the tokens of request b only."""
    only = torch.tensor([cu[b]] * (b + 1) + [cu[b + 1]] * (len(cu) - 1 - b), dtype=torch.int32).cuda()
    return a[:6] + [only] + a[7:]


def explicit(d, s, a, got, lens):
    """The requests whose rows of `got` are the explicit form's."""
    cu, found = s["cu_tokens"].tolist(), []
    room = 256 + sum(-(-(p + n) // 128) * 128 for p, n in lens)
    for b, (_, new) in enumerate(lens):
        if not new:
            continue
        t = slice(cu[b], cu[b + 1])
        x = alone(a, cu, b)
        there = [mla.paged_prefill(d, *x, key_rows=room)[i][t] for i in (0, 1)]
        off = [mla.paged_prefill(d, *x, key_rows=0)[i][t] for i in (0, 1)]
        same = torch.equal(got[0][t], there[0]) and torch.equal(got[1][t], there[1])
        differ = not (torch.equal(off[0], there[0]) and torch.equal(off[1], there[1]))
        if same and differ:
            found.append(b)
    return found


@pytest.mark.parametrize("heads,page,lens", [c[:3] for c in CASES] + [
    (130, 16, [(0, 200), (300, 40)]),
    (64, 64, [(0, 32), (0, 31), (100, 32), (1000, 60), (1000, 130)]),
])
def test_by_the_rule(heads, page, lens):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(heads + page), d, BF, lens, page, extra_rows=1)
    a = sref.on_gpu(s)
    want = rule(heads, lens, 1 << 30)
    assert want and explicit(d, s, a, mla.paged_prefill(d, *a), lens) == want
    assert explicit(d, s, a, mla.paged_prefill(d, *a, key_rows=0), lens) == []


LENS = [(600, 200), (700, 300), (900, 200)]          # 896, 1024 and 1152 rows


@pytest.mark.parametrize("lens,key_rows,want", [
    (LENS, 255, []), (LENS, 768, []), (LENS, 1023, []), (LENS, 1024, [0]), (LENS, 1280, [0]), (LENS, 2047, [0]), (LENS, 2048, [0, 1]),
    (LENS, 2304, [0, 1]), (LENS, 2900, [0, 1]), (LENS, 1 << 14, [0, 1, 2]),
    ([(3000, 300), (0, 300), (500, 200), (0, 5)], 1280, [1, 2]),       # a request longer than the room in front of others
    ([(0, 300), (2900, 300), (500, 200), (0, 100)], 1536, [0, 2, 3]),  # .. between them
    ([(5000, 300)] * 3 + [(0, 130)] * 5, 1024, [3, 4, 5, 6]),          # .. several; of five that would fit the first four
])
@pytest.mark.parametrize("heads", [16, 128])
def test_by_the_room(heads, lens, key_rows, want):
    d = mla.dims(heads, **V3)
    s = sref.step(ref.generator(8), d, BF, lens, 16)
    a = sref.on_gpu(s)
    out, lse = mla.paged_prefill(d, *a, key_rows=key_rows)
    assert rule(heads, lens, key_rows) == want
    assert explicit(d, s, a, (out, lse), lens) == want
    cu = s["cu_tokens"].tolist()
    for b in range(len(lens)):
        check_rows(d, s, out, lse, spread(cu, b, 4))


def test_behind_more_keys_than_the_default_room():
    """A request of more than 65536 keys goes absorbed by default, the one behind it explicit; both with the rows given."""
    d = mla.dims(3, **V3)
    lens = [(66000, 300), (0, 300)]
    s = sref.step(ref.generator(3), d, BF, lens, 64)
    a = sref.on_gpu(s)
    assert rule(3, lens, mla.PREFILL_KEY_ROWS) == [1] and rule(3, lens, 68000) == [0, 1]
    cu = s["cu_tokens"].tolist()
    for rows, want in ((None, [1]), (68000, [0, 1])):
        got = mla.paged_prefill(d, *a, key_rows=rows)
        assert explicit(d, s, a, got, lens) == want
        for b in range(2):
            check_rows(d, s, *got, spread(cu, b, 5))


def test_more_requests_than_a_block_has_threads():
    """Past 1024 requests the room is handed on from one part of them to the next."""
    d = mla.dims(16, **V3)
    lens = [(0, 0)] * 2600
    lens[3], lens[700], lens[1500], lens[1501], lens[2599] = (1000, 200), (0, 200), (2000, 300), (0, 200), (0, 40)
    s = sref.step(ref.generator(4), d, BF, lens, 64)
    a = sref.on_gpu(s)
    for key_rows, want in ((1536, [3, 700]), (1792, [3, 700, 1501]), (2048, [3, 700, 1501, 2599]), (1024, [700, 1501, 2599])):
        assert rule(16, lens, key_rows) == want
        assert explicit(d, s, a, mla.paged_prefill(d, *a, key_rows=key_rows), lens) == want
