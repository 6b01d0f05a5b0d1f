"""Paged prefill, page weights and eviction without a GPU: the tests' 64-bit reference against the decode's, the C
ABI's refusals (fake addresses, nothing is launched), workspace queries and the binding's argument checks."""
import ctypes
import math

import pytest
import torch

import paged_ref as ref
import paged_step_ref as sref
from head_latent_attention_rmsnorm_gb300 import build as mla_build
from head_latent_attention_rmsnorm_gb300 import mla

V3 = dict(n_heads=128, d_kv=512, d_nope=128, d_rope=64, d_v=128)
SMALL = dict(n_heads=3, d_kv=20, d_nope=8, d_rope=6, d_v=10)
BASE = 0x7f0000000000


def fake(i):
    return BASE + (i << 36)


@pytest.fixture(scope="module", autouse=True)
def built():
    mla_build.build()


def test_reference_prefill_is_decode_token_by_token():
    d = mla.dims(**SMALL)
    s = sref.step(ref.generator(1), d, torch.float64, [(0, 2), (4, 3), (0, 0)], 5, extra_rows=1, lead=1)
    out, lse, _, _ = sref.prefill(d, s)
    own = sref.owners(s)
    assert own == [-1, 0, 0, 1, 1, 1, -1]
    for t, b in enumerate(own):
        if b < 0:
            assert bool(lse[t].isnan().all())
            continue
        o, l, _, _ = ref.decode(d, s["q_nope"][t:t + 1], s["q_pe"][t:t + 1], s["c_cache"], s["kpe_cache"],
                                s["block_table"][b:b + 1], [int(s["positions"][t]) + 1], s["w_kv_b"])
        assert torch.allclose(o[0], out[t], rtol=0, atol=1e-12) and torch.allclose(l[0], lse[t], rtol=0, atol=1e-12)


def test_reference_weights_sum_to_one_a_head():
    d = mla.dims(**SMALL)
    s = sref.step(ref.generator(2), d, torch.float64, [(0, 2), (14, 3)], 5)
    w, _ = sref.weights(d, s, sref.prefill(d, s)[1])
    assert torch.allclose(w.sum(1), torch.tensor([6.0, 9.0], dtype=torch.float64), rtol=0, atol=1e-12)


def test_reference_eviction_by_hand():
    t, w, freed, counts = sref.evict(torch.tensor([40, 16]), torch.arange(10).view(2, 5),
                                     torch.tensor([[3.0, 1.0, 1.0, 2.0, 0.0], [0.0] * 5]), 8, 3, 0, 1, 9)
    assert t.tolist() == [[0, -1, -1, 3, 4], [5, 6, 7, 8, 9]] and freed == [1, 2] and counts == [2, 2]
    assert w.tolist() == [[3, 0, 0, 2, 0], [0] * 5]
    assert sref.evict(torch.tensor([24]), torch.arange(3).view(1, 3), torch.tensor([[math.nan, 1.0, 9.0]]), 8, 2, 0, 1, 9)[2] == [1]
    assert sref.evict(torch.tensor([24]), torch.arange(3).view(1, 3), torch.tensor([[1.0, 1.0, 1.0]]), 8, 0, 0, 1, 1)[2:] == ([0], [1, 2])


# ------------------------------------------------------------------------ C ABI ----
def prefill_args(**over):
    d = mla.dims(**{**V3, **over.pop("dims_over", {})})
    a = dict(dims=ctypes.byref(d), dtype=mla.MLA_BF16, B=4, n=9, pages=1000, page=64, max_pages=100, rows=4096, shard=16,
             q=fake(1), r=fake(2), c=fake(3), k=fake(4), table=fake(5), lens=fake(6), cu=fake(11), pos=fake(12), w=fake(7), out=fake(8), lse=fake(9),
             ws=fake(10), ws_bytes=1 << 31, stream=None)
    a.update(over)
    return list(a.values()), d


COMMON = [
    (dict(dims=None), -1), (dict(dtype=2), -3), (dict(B=-1), -2), (dict(B=(1 << 24) + 1), -2), (dict(n=-1), -2), (dict(pages=0), -2), (dict(page=0), -2),
    (dict(max_pages=0), -2), (dict(pages=1 << 26), -2), (dict(max_pages=1 << 26), -2), (dict(n=1 << 25), -2),
    (dict(q=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(cu=None), -1), (dict(pos=None), -1),
    (dict(lse=None), -1), (dict(ws=None), -1), (dict(w=None), -1),
    (dict(q=fake(1) + 8), -4), (dict(lens=fake(6) + 2), -4), (dict(cu=fake(11) + 1), -4), (dict(pos=fake(12) + 2), -4),
    (dict(ws=fake(10) + 8), -4), (dict(ws_bytes=4096), -5), (dict(ws=fake(3) + 4096), -9), (dict(ws=fake(12)), -9),
    (dict(dims_over=dict(d_kv=576)), -6), (dict(dims_over=dict(d_rope=130)), -6), (dict(dims_over=dict(d_nope=1026)), -6),
    (dict(B=0, q=None), 0),
]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(out=None), -1), (dict(out=fake(8) + 8), -4), (dict(lse=fake(9) + 4), -4), (dict(out=fake(1)), -9),
    (dict(lse=fake(11)), -9), (dict(lse=fake(8) + 256), -9), (dict(n=0, q=None), 0),
    (dict(rows=-1), -2), (dict(shard=-1), -2),
])
def test_prefill_rejects(over, status):
    args, _d = prefill_args(**dict(over))
    assert mla.mla_paged_prefill(*args) == status


def weights_args(**over):
    d = mla.dims(**{**V3, **over.pop("dims_over", {})})
    a = dict(dims=ctypes.byref(d), dtype=mla.MLA_BF16, B=4, n=9, pages=1000, page=64, max_pages=100, q=fake(1), r=fake(2),
             lse=fake(9), c=fake(3), k=fake(4), table=fake(5), lens=fake(6), cu=fake(11), pos=fake(12), w=fake(7),
             prior=fake(13), out=fake(8), ws=fake(10), ws_bytes=1 << 31, stream=None)
    a.update(over)
    return list(a.values()), d


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(out=None), -1), (dict(out=fake(8) + 2), -4), (dict(lse=fake(9) + 2), -4), (dict(prior=fake(13) + 1), -4),
    (dict(out=fake(1)), -9), (dict(out=fake(9)), -9), (dict(out=fake(13) + 4), -9), (dict(prior=fake(10)), -9),
])
def test_weights_rejects(over, status):
    args, _d = weights_args(**dict(over))
    assert mla.mla_paged_weights(*args) == status


def evict_args(**over):
    a = dict(B=4, page=64, max_pages=100, room=400, keep=50, first=1, last=2, lens=fake(1), table=fake(2), w=fake(3),
             to=fake(4), wo=fake(5), freed=fake(6), counts=fake(7), ws=fake(8), ws_bytes=1 << 16, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -2), (dict(B=16385), -2), (dict(page=0), -2), (dict(max_pages=0), -2), (dict(room=-1), -2), (dict(keep=-1), -2),
    (dict(first=-1), -2), (dict(last=0), -2), (dict(max_pages=1 << 26), -2), (dict(B=16384, max_pages=1 << 18, page=1), -2),
    (dict(lens=None), -1), (dict(table=None), -1), (dict(w=None), -1), (dict(to=None), -1), (dict(wo=None), -1),
    (dict(freed=None), -1), (dict(counts=None), -1), (dict(ws=None), -1),
    (dict(lens=fake(1) + 2), -4), (dict(freed=fake(6) + 1), -4), (dict(ws=fake(8) + 8), -4), (dict(ws_bytes=100), -5),
    (dict(to=fake(2) + 4), -9), (dict(wo=fake(2)), -9), (dict(to=fake(5)), -9), (dict(freed=fake(1)), -9), (dict(counts=fake(6)), -9),
    (dict(ws=fake(3)), -9),
])
def test_evict_rejects(over, status):
    assert mla.mla_paged_evict(*evict_args(**over)) == status


def test_workspace_queries():
    d = mla.dims(**V3)
    for query, call, args, room in ((mla.mla_paged_prefill_workspace, mla.mla_paged_prefill, prefill_args, (4096, 16)),
                                    (mla.mla_paged_weights_workspace, mla.mla_paged_weights, weights_args, ())):
        f = lambda *a: query(ctypes.byref(d), *a, *room)   # noqa: E731
        few, many = f(mla.MLA_BF16, 4, 9, 64, 100), f(mla.MLA_BF16, 4, 900, 64, 100)
        assert 0 < few < many
        assert f(mla.MLA_BF16, 0, 9, 64, 100) == 0 and f(9, 4, 9, 64, 100) == 0 and f(mla.MLA_BF16, 4, 9, 0, 100) == 0
        assert f(mla.MLA_BF16, 4, -1, 64, 100) == 0
        a, _ = args(n=900, ws_bytes=many - 1)
        assert call(*a) == -5
    f = lambda *a: mla.mla_paged_prefill_workspace(ctypes.byref(d), mla.MLA_BF16, 4, *a)   # noqa: E731
    none = f(900, 64, 100, 0, 16)
    assert none == f(900, 64, 100, 255, 16) < f(900, 64, 100, 4096, 16) < f(900, 64, 100, 4096, 0) == f(900, 64, 100, 4097, 999)
    assert f(900, 64, 100, -1, 16) == 0 == f(900, 64, 100, 4096, -1)
    assert f(900, 60, 100, 4096, 16) == f(900, 60, 100, 0, 16)   # pages that the tensor cores do not take
    f = mla.mla_paged_evict_workspace
    assert f(0, 9) == 0 == f(3, 0) < f(3, 9) < f(9000, 9) < f(9000, 70000)


# ---------------------------------------------------------------------- binding ----
def test_wrappers_refuse_host_tensors():
    d = mla.dims(**SMALL)
    s = sref.step(ref.generator(3), d, torch.float32, [(0, 2)], 2)
    a = [s[n] for n in sref.NAMES]
    with pytest.raises(ValueError, match="CUDA device"):
        mla.paged_prefill(d, *a)
    with pytest.raises(ValueError, match="CUDA device"):
        mla.paged_weights(d, *a[:2], torch.zeros(2, 3), *a[2:])
    with pytest.raises(ValueError, match="CUDA device"):
        mla.paged_evict(s["kv_lens"], s["block_table"], torch.zeros(1, 2), page_size=2, keep_pages=1)
    with pytest.raises(TypeError, match="expected a torch.Tensor"):
        mla.paged_evict(s["kv_lens"], None, None, page_size=2, keep_pages=1)
