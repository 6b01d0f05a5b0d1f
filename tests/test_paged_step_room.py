"""The room that paged prefill takes by default for its explicit form, without a GPU: enough for every step of its sizes
(by the rule of which requests go explicit, over random and worst divisions of the tokens), and not much more than such a step
can use."""
import ctypes
import random

import pytest
import torch

from head_latent_attention_rmsnorm_gb300 import build as mla_build
from head_latent_attention_rmsnorm_gb300 import mla

V3 = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)


@pytest.fixture(scope="module", autouse=True)
def built():
    mla_build.build()


def most(heads, B, n, page, cols, dtype=mla.MLA_BF16):
    return mla.mla_paged_prefill_key_rows(ctypes.byref(mla.dims(heads, **V3)), dtype, B, n, page, cols)


def item_rows(heads):
    tile = 64 if heads <= 64 else 128
    return tile // heads * heads if heads <= tile else heads // -(-heads // tile)


def takes(r, n, cap):
    """The most rows that a request of n tokens can take, over its number of keys."""
    best = 0
    for tiled in range(128, -(-cap // 128) * 128 + 1, 128):
        keys = min(tiled, cap)
        if n >= 32 and keys >= 32 and 6 * n * (keys + 12 * r) >= 11 * r * (tiled + 64):
            best = tiled
    return best


@pytest.mark.parametrize("heads", [1, 5, 16, 20, 64, 65, 128, 130, 200])
@pytest.mark.parametrize("page,cols", [(16, 9), (64, 33), (8, 700), (64, 300)])
def test_enough_for_every_division_of_the_tokens(heads, page, cols):
    r, cap, rng = item_rows(heads), page * cols, random.Random(heads)
    f = [takes(r, n, cap) for n in range(1, 300)]
    f = [0] + f + [f[-1]] * 4000
    best = [0] * 1200                       # over all divisions into any number of requests
    for n in range(32, 1200):
        best[n] = max([best[n - 1]] + [f[k] + best[n - k] for k in range(32, min(n, 260) + 1)])
    for n in list(range(64, 330)) + [511, 512, 777, 1024, 1199]:
        got = most(heads, 1 << 20, n, page, cols)
        # n tokens bring at most n f(k) / k < (n // k + 1) f(k) rows for the best k, and n // k >= 1 requests of k do bring theirs
        assert got % 256 == 0 and best[n] <= got <= 2 * best[n] + 255, n
        B = rng.randint(1, 4)               # few requests: no more than a row of the table each
        few = most(heads, B, n, page, cols)
        assert few <= got and few <= -(-B * (-(-cap // 128) * 128) // 256) * 256
        split = [n // B] * B
        assert sum(f[k] for k in split) <= few and f[n] <= few


def room(heads, B, n, page, cols, dtype=torch.bfloat16, **kw):
    a = dict(key_rows=None, head_shard=None)
    a.update(kw)
    code = mla.MLA_BF16 if dtype == torch.bfloat16 else mla.MLA_F32
    return mla._prefill_room(mla.dims(heads, **V3), code, n, (B, cols), page, **a)


def test_default_room():
    # a decode step, or steps of a few tokens, over long tables: nearly nothing
    assert room(128, 64, 63, 64, 2048) == (0, 0)
    rows, shard = room(128, 64, 64, 64, 2048)
    assert 0 < rows <= 512 and shard == 0
    # one long chunk: its table's row; many tokens over long tables: the most there is, in shards of heads
    assert room(128, 1, 2048, 64, 256) == (16384, mla.PREFILL_HEAD_SHARD)
    assert room(128, 64, 4096, 64, 2048) == (mla.PREFILL_KEY_ROWS, mla.PREFILL_HEAD_SHARD)
    # prompts of a table of 5120 rows at 128 heads: all heads at once
    assert room(128, 1, 2048, 64, 80) == (5120, 0)
    # what the caller says stays; kernels without the form take nothing
    assert room(128, 64, 64, 64, 2048, key_rows=4096, head_shard=3) == (4096, 3)
    assert room(128, 64, 64, 64, 2048, key_rows=0) == (0, 0)
    assert room(16, 4, 500, 64, 100, dtype=torch.float32)[0] == 0
    assert room(16, 4, 500, 60, 100)[0] == 0
    assert room(16, 0, 500, 64, 100)[0] == 0 and room(16, 4, 0, 64, 100)[0] == 0


def test_default_workspace_of_a_decode_step():
    """64 requests of one token over a table of 131072 keys, 128 heads: 0.1 GB at most (0.05 without the form)."""
    d = mla.dims(128, **V3)
    args = (ctypes.byref(d), mla.MLA_BF16, 64, 64, 64, 2048)
    assert mla.mla_paged_prefill_workspace(*args, *room(128, 64, 64, 64, 2048)) <= 100 << 20


@pytest.mark.parametrize("heads,B,page,cols", [(128, 64, 64, 100), (128, 3, 64, 128), (16, 8, 64, 700), (130, 64, 8, 3000), (20, 1, 64, 512)])
def test_a_workspace_does_for_steps_of_fewer_tokens(heads, B, page, cols):
    """A server allocates one for its largest step; smaller ones, whose rows may allow all heads at once, fit in it."""
    d = mla.dims(heads, **V3)
    cache, table = torch.empty(1, page, 512, dtype=torch.bfloat16, device="meta"), torch.empty(B, cols, dtype=torch.int32, device="meta")
    most = 0
    for n in (1, 32, 63, 64, 65, 100, 150, 180, 200, 220, 232, 233, 250, 300, 400, 511, 700, 1024, 2048, 4096, 5000):
        need = mla.mla_paged_prefill_workspace(ctypes.byref(d), mla.MLA_BF16, B, n, page, cols, *room(heads, B, n, page, cols))
        most = max(most, need)
        assert most <= mla.paged_prefill_workspace(d, n, cache, table).numel(), n
    for kw in (dict(key_rows=4096), dict(head_shard=5), dict(key_rows=0, head_shard=0)):
        want = mla.mla_paged_prefill_workspace(ctypes.byref(d), mla.MLA_BF16, B, 300, page, cols, *room(heads, B, 300, page, cols, **kw))
        assert mla.paged_prefill_workspace(d, 300, cache, table, **kw).numel() >= want


@pytest.mark.parametrize("v", [1 << 31, 1 << 32, (1 << 32) + 256, -(1 << 31) - 1])
def test_numbers_past_32_bits_are_refused(v):
    """ctypes would pass their low halves: 2^32 pages to keep would be none."""
    with pytest.raises(ValueError, match="key_rows: .* 32 bits"):
        room(128, 4, 100, 64, 100, key_rows=v)
    with pytest.raises(ValueError, match="head_shard: .* 32 bits"):
        room(128, 4, 100, 64, 100, head_shard=v)
    for name in ("page_size", "keep_pages", "first_pages", "last_pages"):
        with pytest.raises(ValueError, match=name + ": .* 32 bits"):
            mla.paged_evict(None, None, None, **{**dict(page_size=8, keep_pages=1), name: v})


def test_refused_sizes_have_no_room():
    assert most(128, -1, 100, 64, 100) == 0 == most(128, 4, -1, 64, 100) == most(128, 4, 100, 0, 100) == most(128, 4, 100, 64, 0)
    assert most(128, 4, 100, 64, 100, dtype=9) == 0
    assert mla.mla_paged_prefill_key_rows(None, mla.MLA_BF16, 4, 100, 64, 100) == 0
    assert most(1, 1 << 24, 1 << 24, 64, 1 << 24) == (2 ** 31 - 1) // 256 * 256
