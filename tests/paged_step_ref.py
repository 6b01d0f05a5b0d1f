"""Several tokens a request over the paged cache, in 64 bits, token by token, on the host: what the tests of
paged prefill, page weights and eviction compare the kernels with."""
import math

import torch

import paged_ref as ref


def step(g, d, dtype, lens, page, *, extra_rows=0, junk=math.nan, scale=1.0, lead=0):
    """A step's inputs for requests of (past, new) lengths, on the host; `lead` rows in front belong to no request."""
    kv = [p + n for p, n in lens]
    c, k, table = ref.cache(g, d, dtype, kv, page, junk=junk, scale=scale)
    cu = [lead]
    for _, n in lens:
        cu.append(cu[-1] + n)
    n_tokens = cu[-1] + extra_rows
    positions = torch.full((n_tokens,), 7, dtype=torch.int32)
    for b, (p, n) in enumerate(lens):
        positions[cu[b]:cu[b + 1]] = torch.arange(p, p + n, dtype=torch.int32)
    q, r, w = ref.queries(g, d, dtype, n_tokens)
    i32 = dict(dtype=torch.int32)
    return dict(q_nope=q, q_pe=r, c_cache=c, kpe_cache=k, block_table=table, kv_lens=torch.tensor(kv, **i32),
                cu_tokens=torch.tensor(cu, **i32), positions=positions, w_kv_b=w)


NAMES = ("q_nope", "q_pe", "c_cache", "kpe_cache", "block_table", "kv_lens", "cu_tokens", "positions", "w_kv_b")


def on_gpu(s):
    return [s[n].cuda() for n in NAMES]


def owners(s):
    """Each token row's request, -1 for none."""
    cu, n = s["cu_tokens"].tolist(), s["positions"].numel()
    got = [-1] * n
    for b in range(len(cu) - 1):
        for t in range(max(cu[b], 0), min(cu[b + 1], n)):
            got[t] = b
    return got


def prefill(d, s):
    """(out, lse, mass, sq) of every token row as ref.decode's, rows of no request with lse NaN."""
    H, dn, dv, dk = d.n_heads, d.d_nope, d.d_v, d.d_kv
    num_pages, page = s["c_cache"].shape[:2]
    scale = d.softmax_scale if d.softmax_scale > 0 else 1.0 / math.sqrt(dn + d.d_rope)
    w = s["w_kv_b"].double().view(H, dn + dv, dk)
    table = s["block_table"]
    n_tokens = s["positions"].numel()
    out = torch.zeros(n_tokens, H, dv, dtype=torch.float64)
    lse = torch.full((n_tokens, H), math.nan, dtype=torch.float64)
    mass, sq = torch.zeros(n_tokens, H, dtype=torch.float64), torch.zeros(n_tokens, H, dtype=torch.float64)
    c, kr = s["c_cache"].reshape(-1, dk), s["kpe_cache"].reshape(-1, d.d_rope)
    for t, b in enumerate(owners(s)):
        if b < 0:
            continue
        pos = int(s["positions"][t])
        n = min(max(int(s["kv_lens"][b]), 0), table.shape[1] * page, pos + 1)
        ids = table[b, :-(-n // page)].tolist() if n > 0 else []
        rows = [i * page + o for j, i in enumerate(ids) if 0 <= i < num_pages for o in range(min(page, n - j * page))]
        if not rows:
            lse[t] = -math.inf
            continue
        q = torch.einsum("hn,hnk->hk", s["q_nope"][t].double(), w[:, :dn])
        full_q = torch.cat([q, ref.rope(s["q_pe"][t], torch.full((H,), pos), d.rope_base)], 1)
        full_k = torch.cat([c[rows].double(), kr[rows].double()], 1)
        x = full_q @ full_k.T * scale
        m = x.amax(1, keepdim=True)
        p = torch.exp(x - m)
        lse[t] = torch.log(p.sum(1)) + m[:, 0]
        out[t] = torch.einsum("hk,hvk->hv", p @ c[rows].double() / p.sum(1, keepdim=True), w[:, dn:])
        aq = torch.cat([torch.einsum("hn,hnk->hk", s["q_nope"][t].double().abs(), w[:, :dn].abs()) / math.sqrt(dn),
                        full_q[:, dk:].abs()], 1)
        mass[t] = torch.maximum((aq @ full_k.abs().T).amax(1), (full_q.abs() @ full_k.abs().T).amax(1)) * scale
        sq[t] = (full_q.square() @ full_k.square().T).amax(1) * scale * scale
    return out, lse, mass, sq


def check_prefill(dtype, out, lse, want, before=None):
    """Every computed row by ref.check_decode; rows of no request hold what they held (`before`: (out, lse))."""
    ro, rl, mass, sq = want
    mine = ~torch.isnan(rl[:, 0])
    if before is not None:
        assert torch.equal(out.cpu()[~mine], before[0].cpu()[~mine])
        assert torch.equal(lse.cpu()[~mine], before[1].cpu()[~mine])
    ref.check_decode(dtype, out.cpu()[mine], lse.cpu()[mine], (ro[mine], rl[mine], mass[mine], sq[mine]))


def weights(d, s, lse, prior=None):
    """(page weights [B, max_pages], bound of their error): each exp(s - lse) is off by its score's absolute error
    relative to it.  A score is a sum of up to 1024 products of which each and each partial sum is rounded:
    2^-17 of the largest mass sum |q_d k_d| (as decode_bounds has it), as much again for queries held as bf16
    pairs, and for the scale, exponent and lse's product with log2 e; the sums add 2^-17 of the whole (fewer than 128
    roundings each of rows and keys), the result half a step, each sum of up to 32 keys half a unit of the fixed point."""
    H, dk, page = d.n_heads, d.d_kv, s["c_cache"].shape[1]
    num_pages, table = s["c_cache"].shape[0], s["block_table"]
    scale = d.softmax_scale if d.softmax_scale > 0 else 1.0 / math.sqrt(d.d_nope + d.d_rope)
    w = s["w_kv_b"].double().view(H, d.d_nope + d.d_v, dk)[:, :d.d_nope]
    got = torch.zeros(table.shape, dtype=torch.float64) if prior is None else prior.double().clone()
    err = torch.zeros_like(got)
    c, kr = s["c_cache"].reshape(-1, dk), s["kpe_cache"].reshape(-1, d.d_rope)
    n_tokens = s["positions"].numel()
    unit = 2.0 ** -(61 - math.ceil(math.log2(max(2 * n_tokens * H * page, 1))))
    for t, b in enumerate(owners(s)):
        if b < 0:
            continue
        pos = int(s["positions"][t])
        n = min(max(int(s["kv_lens"][b]), 0), table.shape[1] * page, pos + 1)
        at = [(j // page, int(table[b, j // page]) * page + j % page) for j in range(n) if 0 <= int(table[b, j // page]) < num_pages]
        if not at:
            continue
        cols, rows = torch.tensor([x for x, _ in at]), [x for _, x in at]
        q = torch.einsum("hn,hnk->hk", s["q_nope"][t].double(), w)
        full_q = torch.cat([q, ref.rope(s["q_pe"][t], torch.full((H,), pos), d.rope_base)], 1)
        full_k = torch.cat([c[rows].double(), kr[rows].double()], 1)
        p = torch.exp(full_q @ full_k.T * scale - lse[t].double()[:, None])
        p = torch.where(torch.isneginf(lse[t])[:, None], 0.0, p).clamp(0, 2)
        mass = (full_q.abs() @ full_k.abs().T) * scale + lse[t].double().abs()[:, None].nan_to_num(0, 0, 0)
        got[b].index_add_(0, cols, p.sum(0))
        err[b].index_add_(0, cols, (p * 2.0 ** -16 * (1 + mass)).sum(0) + unit)
    return got, err + got.abs() * (2.0 ** -17 + 2.0 ** -24)


def evict(kv_lens, table, weights, page, keep, first, last, room):
    """(table, weights, freed, counts) of an eviction, page by page."""
    table, weights, freed, wanted = table.clone(), weights.clone(), [], 0
    for b, n in enumerate(kv_lens.tolist()):
        cols = -(-min(max(n, 0), table.shape[1] * page) // page)
        held = [c for c in range(cols) if table[b, c] >= 0]
        may = [c for c in held if first <= c < cols - last]
        value = {c: math.inf if math.isnan(float(weights[b, c])) else float(weights[b, c]) for c in may}
        order = sorted(may, key=lambda c: (math.isnan(float(weights[b, c])), value[c], c))
        for c in sorted(order[:max(0, len(held) - keep)]):
            wanted += 1
            if len(freed) < room:
                freed.append(int(table[b, c]))
                table[b, c] = -1
                weights[b, c] = 0.0
    return table, weights, freed, [len(freed), wanted]
