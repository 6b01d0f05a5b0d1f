"""The paged latent cache in 64 bits, request by request, on the host: what the paged tests
compare the kernels with, and inputs and error bounds for them."""
import math

import numpy as np
import torch

EPS16, EPS32 = 2.0 ** -8, 2.0 ** -24   # half a step of bf16 and fp32, relative


def half_step(dtype):
    return EPS32 if dtype == torch.float32 else EPS16


def tables(past, new, free, table, page, n_tokens):
    """One step's tables token by token.  Returns (table, kv_lens, cu, slots, positions, counts)."""
    table = [list(r) for r in table]
    cap = len(table[0]) * page if table else 0
    free = list(free)
    slots, positions, kv, cu = [-1] * n_tokens, [0] * n_tokens, [], [0]
    taken = needed = 0
    for b, (p0, n) in enumerate(zip(past, new)):
        p0, n = min(max(p0, 0), cap), max(n, 0)
        length, open_ = p0, True
        held = -(-p0 // page)
        for i in range(n):
            row, pos = cu[-1] + i, p0 + i
            if row < n_tokens:
                positions[row] = pos
            if row >= n_tokens or pos >= cap:
                continue
            col = pos // page
            if col >= held:
                held += 1
                needed += 1
                if taken < len(free):
                    table[b][col] = free[taken]
                    taken += 1
                else:
                    open_ = False
            if open_:
                length = pos + 1
                if table[b][col] >= 0:
                    slots[row] = table[b][col] * page + pos % page
        kv.append(length)
        cu.append(cu[-1] + n)
    return table, kv, cu, slots, positions, [taken, needed]


def rope(x, pos, base):
    """x [..., d], pos broadcastable to x's leading dims; float64."""
    x = x.double()
    half = x.shape[-1] // 2
    inv = base ** (-2.0 * torch.arange(half, dtype=torch.float64) / x.shape[-1])
    a = torch.as_tensor(pos, dtype=torch.float64)[..., None] * inv
    c, s = a.cos(), a.sin()
    x1, x2 = x[..., :half], x[..., half:]
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)


def rmsnorm(x, w, eps):
    x = x.double()
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()


def decode(d, q_nope, q_pe, c_cache, kpe_cache, table, lens, w):
    """Returns (out, lse, score_mass, sq_mass): the last two, per request and head, are the largest
    over the keys of scale * sum_d |q_d k_d| and scale^2 * sum_d (q_d k_d)^2, which the error
    bounds need."""
    H, dn, dv, dk = d.n_heads, d.d_nope, d.d_v, d.d_kv
    num_pages, page = c_cache.shape[:2]
    scale = d.softmax_scale if d.softmax_scale > 0 else 1.0 / math.sqrt(dn + d.d_rope)
    w = w.double().view(H, dn + dv, dk)
    B = q_nope.shape[0]
    out = torch.zeros(B, H, dv, dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    mass, sq = torch.zeros(B, H, dtype=torch.float64), torch.zeros(B, H, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        ids = [int(table[b, p // page]) for p in range(n)]
        rows = [i * page + p % page for p, i in enumerate(ids) if 0 <= i < num_pages]
        if not rows:
            continue
        k = c_cache.reshape(-1, dk)[rows].double()
        kr = kpe_cache.reshape(-1, d.d_rope)[rows].double()
        q = torch.einsum("hn,hnk->hk", q_nope[b].double(), w[:, :dn])
        qr = rope(q_pe[b], torch.full((H,), n - 1), d.rope_base)
        full_q, full_k = torch.cat([q, qr], 1), torch.cat([k, kr], 1)
        s = full_q @ full_k.T * scale
        m = s.amax(1, keepdim=True)
        p = torch.exp(s - m)
        lse[b] = torch.log(p.sum(1)) + m[:, 0]
        o = p @ k / p.sum(1, keepdim=True)
        out[b] = torch.einsum("hk,hvk->hv", o, w[:, dn:])
        aq = torch.einsum("hn,hnk->hk", q_nope[b].double().abs(), w[:, :dn].abs())
        mass[b] = (torch.cat([aq, qr.abs()], 1) @ full_k.abs().T).amax(1) * scale / math.sqrt(dn)
        mass[b] = torch.maximum(mass[b], (full_q.abs() @ full_k.abs().T).amax(1) * scale)
        sq[b] = (full_q.square() @ full_k.square().T).amax(1) * scale * scale
    return out, lse, mass, sq


def decode_bounds(dtype, lse, mass, sq):
    """(bound of |lse - exact| per request and head, bound of the output's relative 2-norm error).

    fp32 arithmetic: a sum of n products of fp32 numbers is off by about sqrt(n) half steps of
    its mass sum |q_d k_d| (independent roundings); n <= 1024 operations and a factor 4 for the
    tail give 2^7 half steps = 2^-17 of the mass, and 2^-20 |lse| covers the exp, log and the
    merge.  A weight's relative error is its score's absolute one, so the output's relative
    error is at most that bound too, plus as much again for the second product.
    bf16 tensor-core path: the score product takes q rounded to bf16 (half a step per dim,
    uniform: variance step^2 / 3 of q_d k_d) and the mean effect on lse is put back exactly, which
    leaves half the variance of the scores' errors under the softmax: <= 4 times their largest
    variance with the factor for the tail.  The output meets that rounding's deviation, the
    probabilities' rounding to bf16 and its own: each at most half a step, deviation a third."""
    fin = torch.isfinite(lse)
    lse_bound = 2.0 ** -17 * (1 + mass) + 2.0 ** -20 * torch.where(fin, lse.abs(), torch.zeros_like(lse))
    rel = 2.0 * float(lse_bound.max()) if lse.numel() else 0.0
    if dtype != torch.float32:
        var = EPS16 ** 2 / 3 * sq
        lse_bound = lse_bound + 4 * var
        rel += EPS16 * (1 + 1) + math.sqrt(float(var.max())) if lse.numel() else 0.0
    return lse_bound, rel


def check_decode(dtype, out, lse, ref):
    ro, rl, mass, sq = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    bound, rel = decode_bounds(dtype, rl, mass, sq)
    fin = torch.isfinite(rl)
    assert torch.equal(lse[~fin], rl[~fin])
    err = (lse - rl)[fin].abs()
    assert bool((err <= bound[fin]).all()), (float(err.max()), float((err / bound[fin]).max()))
    dead = ~fin
    assert bool((out[dead] == 0).all())
    assert bool(torch.isfinite(out).all())
    if fin.any():
        e, n = (out - ro).norm(), ro.norm()
        assert float(e) <= rel * float(n), (float(e / n), rel)
        rows = (out - ro)[fin].norm(dim=-1) / ro[fin].norm(dim=-1)   # no row of its own far off
        assert float(rows.max()) <= 4 * rel, (float(rows.max()), rel)


def cache(g, d, dtype, lens, page, *, spare=3, extra_cols=1, junk=math.nan, scale=1.0):
    """A cache whose pages lie in random order, a table whose unused entries are -1, unused slots
    holding `junk`.  Returns (c_cache, kpe_cache, table) on the host."""
    per = [-(-n // page) for n in lens]
    pages = sum(per) + spare
    ids = torch.randperm(pages, generator=g).tolist()
    most = max(per + [1]) + extra_cols
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    c = torch.full((pages, page, d.d_kv), junk)
    k = torch.full((pages, page, d.d_rope), junk)
    for b, n in enumerate(lens):
        mine, ids = ids[:per[b]], ids[per[b]:]
        for j, i in enumerate(mine):
            table[b, j] = i
            m = min(page, n - j * page)
            c[i, :m] = torch.randn(m, d.d_kv, generator=g) * scale
            k[i, :m] = torch.randn(m, d.d_rope, generator=g) * scale
    return c.to(dtype), k.to(dtype), table


def queries(g, d, dtype, batch):
    q = torch.randn(batch, d.n_heads, d.d_nope, generator=g).to(dtype)
    r = torch.randn(batch, d.n_heads, d.d_rope, generator=g).to(dtype)
    w = (torch.randn(d.n_heads * (d.d_nope + d.d_v), d.d_kv, generator=g) / math.sqrt(d.d_kv)).to(dtype)
    return q, r, w


def generator(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def to_numpy(t):
    return np.ascontiguousarray(t.double().numpy())
