"""The paged cache without a GPU: the tests' own 64-bit reference against the oracle, the C ABI's
refusals (fake addresses, nothing is launched) and the binding's argument checks."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
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


# ------------------------------------------------------------------ the reference ----
def test_reference_decode_is_the_oracles(oracle):
    d = mla.dims(**SMALL)
    g = ref.generator(1)
    lens = [1, 9, 14]
    c, k, table = ref.cache(g, d, torch.float64, lens, 5)
    q, r, w = ref.queries(g, d, torch.float64, len(lens))
    out, lse, _, _ = ref.decode(d, q, r, c, k, table, lens, w)
    for b, n in enumerate(lens):
        rows = [int(table[b, p // 5]) * 5 + p % 5 for p in range(n)]
        o, l = oracle.mla_decode(ref.to_numpy(q[b:b + 1]), ref.to_numpy(r[b:b + 1]),
                                 ref.to_numpy(c.reshape(-1, d.d_kv)[rows][None]),
                                 ref.to_numpy(k.reshape(-1, d.d_rope)[rows][None]), ref.to_numpy(w), n_splits=2,
                                 base=d.rope_base, partials=False)[:2]
        np.testing.assert_allclose(out[b].numpy(), np.asarray(o).reshape(d.n_heads, d.d_v), rtol=0, atol=1e-12)
        np.testing.assert_allclose(lse[b].numpy(), np.asarray(l).reshape(-1), rtol=0, atol=1e-12)


def test_reference_rows_are_the_oracles(oracle):
    g = ref.generator(2)
    x, w = torch.randn(4, 20, generator=g).double(), torch.randn(20, generator=g).double()
    np.testing.assert_allclose(ref.rmsnorm(x, w, 1e-6).numpy(), oracle.rmsnorm(x.numpy(), w.numpy(), 1e-6), atol=1e-13)
    y = torch.randn(4, 6, generator=g).double()
    for i, p in enumerate([0, 1, 77, 100000]):
        np.testing.assert_allclose(ref.rope(y[i:i + 1], torch.tensor([p]), 10000.0).numpy(),
                                   oracle.rope(y[i:i + 1].numpy(), p, 10000.0), atol=1e-11)


# ------------------------------------------------------------------------ C ABI ----
def tables_args(**over):
    a = dict(B=4, page=16, max_pages=8, n_free=9, n_tokens=20, past=fake(1), new=fake(2), free=fake(3), table=fake(4),
             kv=fake(5), cu=fake(6), slots=fake(7), positions=fake(8), counts=fake(9), stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), -2), (dict(B=16385), -2), (dict(page=0), -2), (dict(max_pages=0), -2), (dict(n_free=-1), -2),
    (dict(n_tokens=-1), -2), (dict(page=1 << 16, max_pages=1 << 15), -2),
    (dict(past=None), -1), (dict(new=None), -1), (dict(free=None), -1), (dict(table=None), -1), (dict(kv=None), -1),
    (dict(cu=None), -1), (dict(slots=None), -1), (dict(positions=None), -1), (dict(counts=None), -1),
    (dict(cu=fake(6) + 2), -4), (dict(table=fake(4) + 1), -4),
    (dict(kv=fake(1)), -9), (dict(slots=fake(8)), -9), (dict(table=fake(2)), -9),
])
def test_tables_rejects(over, status):
    assert mla.mla_paged_tables(*tables_args(**over)) == status


def append_args(**over):
    d = mla.dims(**V3)
    a = dict(dims=ctypes.byref(d), dtype=mla.MLA_BF16, n=64, pages=100, page=64, c=fake(1), cs=576, k=fake(2), ks=576,
             w=fake(3), slots=fake(4), positions=fake(5), cc=fake(6), kc=fake(7), stream=None)
    a.update(over)
    return list(a.values()), d


@pytest.mark.parametrize("over,status", [
    (dict(dims=None), -1), (dict(dtype=5), -3), (dict(n=-1), -2), (dict(pages=0), -2), (dict(page=0), -2),
    (dict(pages=1 << 20, page=1 << 12), -2), (dict(cs=511), -2), (dict(ks=63), -2), (dict(cs=1 << 31), -2),
    (dict(c=None), -1), (dict(slots=None), -1), (dict(kc=None), -1),
    (dict(c=fake(1) + 2), -4), (dict(positions=fake(5) + 2), -4),
    (dict(cc=fake(1) + 1024), -9), (dict(kc=fake(6) + 512), -9), (dict(cc=fake(4)), -9),
    (dict(n=0, c=None), 0),
])
def test_append_rejects(over, status):
    args, _d = append_args(**over)
    assert mla.mla_paged_append(*args) == status


def test_append_refuses_a_wide_band():
    d = mla.dims(n_heads=1, d_kv=64, d_nope=8, d_rope=642, d_v=8)
    args, _ = append_args(dims=ctypes.byref(d), ks=642)
    assert mla.mla_paged_append(*args) == -6


def decode_args(**over):
    d = mla.dims(**{**V3, **over.pop("dims_over", {})})
    a = dict(dims=ctypes.byref(d), dtype=mla.MLA_BF16, B=4, pages=1000, page=64, max_pages=100, q=fake(1), r=fake(2),
             c=fake(3), k=fake(4), table=fake(5), lens=fake(6), w=fake(7), out=fake(8), lse=fake(9), ws=fake(10),
             ws_bytes=1 << 31, stream=None)
    a.update(over)
    return list(a.values()), d


@pytest.mark.parametrize("over,status", [
    (dict(dims=None), -1), (dict(dtype=2), -3), (dict(B=-1), -2), (dict(pages=0), -2), (dict(page=0), -2),
    (dict(max_pages=0), -2), (dict(pages=1 << 26), -2), (dict(max_pages=1 << 26), -2), (dict(B=1 << 25), -2),
    (dict(q=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(lse=None), -1), (dict(ws=None), -1),
    (dict(out=fake(8) + 8), -4), (dict(lens=fake(6) + 2), -4), (dict(ws=fake(10) + 8), -4), (dict(ws_bytes=4096), -5),
    (dict(out=fake(1)), -9), (dict(lse=fake(6)), -9), (dict(ws=fake(3) + 4096), -9), (dict(lse=fake(8) + 256), -9),
    (dict(dims_over=dict(d_kv=576)), -6), (dict(dims_over=dict(d_rope=130)), -6), (dict(dims_over=dict(d_nope=1026)), -6),
    (dict(B=0, q=None), 0),
])
def test_decode_rejects(over, status):
    args, _d = decode_args(**dict(over))
    assert mla.mla_paged_decode(*args) == status


def test_decode_workspace_query():
    d = mla.dims(**V3)
    f = lambda *a: mla.mla_paged_decode_workspace(ctypes.byref(d), *a)   # noqa: E731
    one, many = f(mla.MLA_BF16, 1, 64, 512), f(mla.MLA_BF16, 64, 64, 512)
    assert 0 < one < many
    assert f(mla.MLA_BF16, 64, 64, 1 << 20) == many      # the work is divided by workers, not by length
    assert f(mla.MLA_BF16, 0, 64, 512) == 0 and f(9, 1, 64, 512) == 0 and f(mla.MLA_BF16, 1, 0, 512) == 0
    args, _ = decode_args(B=64, ws_bytes=many - 1)
    assert mla.mla_paged_decode(*args) == -5


# ---------------------------------------------------------------------- binding ----
def test_wrappers_refuse_host_tensors():
    d = mla.dims(**SMALL)
    g = ref.generator(3)
    c, k, table = ref.cache(g, d, torch.float32, [3], 2)
    q, r, w = ref.queries(g, d, torch.float32, 1)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        mla.paged_decode(d, q, r, c, k, table, i, w)
    with pytest.raises(ValueError, match="CUDA device"):
        mla.paged_tables(i, i, i, table, page_size=2, n_tokens=1)
    with pytest.raises(ValueError, match="CUDA device"):
        mla.paged_append(d, c[0], k[0], c[0, 0], i, i, c, k)


def test_row_pitch_check():
    x = torch.zeros(6, 30)
    f = lambda t, n=6, width=20, at=-1: mla._rows("x", t, n, width, torch.float32, at)   # noqa: E731 (-1: the host)
    assert f(x[:, :20]) == 30 and f(x[:, 10:]) == 30 and f(torch.zeros(6, 20)) == 20
    assert f(x[::2, :20], n=3) == 60
    assert f(x[:1, :20], n=1) == 20                         # one row has no pitch
    for bad in (x[:, ::2][:, :10].expand(6, 10), torch.zeros(20, 6).t(), torch.zeros(20).expand(6, 20)):
        with pytest.raises(ValueError, match="adjacent|shape"):
            f(bad)
    with pytest.raises(TypeError, match="dtype"):
        f(x[:, :20].double())
    with pytest.raises(ValueError, match="shape"):
        f(x)
    with pytest.raises(ValueError, match="CUDA device 0"):
        f(x[:, :20], at=0)
    with pytest.raises(TypeError, match="expected a torch.Tensor"):
        f(None)


def test_tensor_check():
    x = torch.zeros(4, 6)
    assert mla._need("x", x, (4, 6), torch.float32, -1) == x.data_ptr()   # (-1: the host)
    for t, shape, kind, match in (
            (x, (6, 4), ValueError, "x: on cpu"), (x, (4, 5), ValueError, "x: on cpu"),
            (torch.zeros(6, 4).t(), (4, 6), ValueError, "x: on cpu"), (x.double(), (4, 6), ValueError, "x: on cpu"),
            (None, (4, 6), TypeError, "expected a torch.Tensor"), (3, (4, 6), TypeError, "expected a torch.Tensor"),
            (np.zeros((4, 6), np.float32), (4, 6), TypeError, "expected a torch.Tensor")):
        with pytest.raises(kind, match=match):
            mla._need("x", t, shape, torch.float32, 0)
