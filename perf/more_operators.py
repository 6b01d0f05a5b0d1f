"""Serving several tokens a request over the paged latent cache, and keeping the cache in a budget:
what the three operators compute, over what sizes, and at what cost.

* ``prefill``: the new tokens of every request (a prompt's chunk, a few speculated tokens, one)
  attend over the request's pages;
* ``weights``: the attention weight that each page received from the step's queries, added up;
* ``evict``: the pages of least weight leave the requests that hold more than a budget.

``run`` computes them from elementary torch operations, or, where ``own`` is true, through
the library.
"""
import math
import random

import torch

own = False

ROPE_BASE, EPS = 10000.0, 1e-6
DEEPSEEK = dict(d_kv=512, d_nope=128, d_rope=64, d_v=128)
TINY = dict(d_kv=64, d_nope=32, d_rope=16, d_v=32)


def listed():
    return [
        # a prompt's last chunk: 2048 tokens behind 14336, 128 heads
        dict(name="prefill_chunk_n2048_l16384_h128", op="prefill", dtype="bf16", batch=1, past=14336, new=2048, heads=128,
             page=64, spread="full", **DEEPSEEK),
        # whole prompts of a 16-head model, admitted together, at their own lengths
        dict(name="prefill_prompts_b3_n4096_h16", op="prefill", dtype="bf16", batch=3, past=0, new=4096, heads=16, page=16,
             spread="ragged", **DEEPSEEK),
        # a mixed step: most requests decode a token, a few run a chunk of their prompt
        dict(name="prefill_mixed_b48_l8192_h128", op="prefill", dtype="bf16", batch=48, past=8000, new=333, heads=128, page=64,
             spread="mixed", **DEEPSEEK),
        # speculated tokens: four a request
        dict(name="prefill_spec_b64_n4_l8192_h16", op="prefill", dtype="bf16", batch=64, past=8192, new=4, heads=16, page=64,
             spread="full", **DEEPSEEK),
        # latency: two tokens of one short request, 128 heads
        dict(name="prefill_b1_n2_l300_h128", op="prefill", dtype="bf16", batch=1, past=300, new=2, heads=128, page=64,
             spread="full", **DEEPSEEK),
        # fp32 at small dimensions, odd pages, empty requests, evicted pages
        dict(name="prefill_fp32_tiny", op="prefill", dtype="f32", batch=7, past=200, new=33, heads=4, page=7, spread="holes",
             **TINY),
        # the weights of a decode step: 64 requests of up to 32768 tokens, 128 heads
        dict(name="weights_b64_l32768_h128", op="weights", dtype="bf16", batch=64, past=32767, new=1, heads=128, page=64,
             spread="ragged", **DEEPSEEK),
        # the weights that a prompt's last 32 tokens give its pages, 16 heads
        dict(name="weights_window_b8_n32_l8192_h16", op="weights", dtype="bf16", batch=8, past=8160, new=32, heads=16, page=16,
             spread="full", **DEEPSEEK),
        # fp32 at small dimensions
        dict(name="weights_fp32_tiny", op="weights", dtype="f32", batch=5, past=300, new=3, heads=4, page=7, spread="holes",
             **TINY),
        # eviction to three quarters of the pages: 64 long requests
        dict(name="evict_b64_p512", op="evict", batch=64, page=64, length=32768, keep=384, first=1, last=4, spread="ragged"),
        # the same for a large batch of short requests, some empty
        dict(name="evict_b2001_p128", op="evict", batch=2001, page=32, length=4096, keep=50, first=2, last=2, spread="holes"),
        # one very long request of small pages
        dict(name="evict_b1_p65536", op="evict", batch=1, page=16, length=1048576, keep=8192, first=4, last=64, spread="full"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "weights", "weights", "evict"])
    if op == "evict":
        length = _log(rng, 1, 262144)
        page = rng.choice([7, 16, 32, 64, 128])
        batch = _log(rng, 1, max(1, min(4000, 16000000 // length)))
        pages = -(-length // page)
        return dict(op=op, batch=batch, page=page, length=length, keep=rng.choice([0, pages // 4, pages // 2, pages - pages // 8]),
                    first=rng.choice([0, 1, 4]), last=rng.choice([1, 2, 16]), spread=rng.choice(["full", "ragged", "holes"]))
    dtype, dims = rng.choice([("bf16", DEEPSEEK), ("bf16", DEEPSEEK), ("bf16", DEEPSEEK), ("bf16", DEEPSEEK), ("f32", DEEPSEEK),
                              ("f32", TINY), ("bf16", TINY)])
    small = dtype == "f32" or dims is TINY
    heads = rng.choice([1, 4, 8, 16]) if small else rng.choice([8, 16, 20, 32, 64, 128, 128])
    batch = _log(rng, 1, 16 if small else 64)
    pairs = (20000000 if small else 1000000000) // heads   # (token, key) pairs of the call
    new = _log(rng, 1, max(1, min(400 if small else 4096, pairs // batch, (400 if small else 6000) // batch)))
    if op == "weights":
        new = min(new, 64)
    past = rng.choice([0, 1, 1, 1]) and _log(rng, 1, max(1, min(3000 if small else 32000, 1000000 // batch,
                                                                  pairs // (batch * new) - new)))
    return dict(op=op, dtype=dtype, batch=batch, past=past, new=new, heads=heads,
                page=rng.choice([7, 16, 48]) if small else rng.choice([8, 16, 32, 64, 64, 128]),
                spread=rng.choice(["full", "ragged", "mixed", "holes"]), **dims)


def _pages(n, page):
    return -(-n // page)


def _lengths(case):
    """The requests' (past, new) lengths: a function of the case alone.  full: all the same; ragged:
    anywhere from an eighth up; mixed: one new token, a chunk for every twelfth request; holes:
    ragged, every fifth request empty."""
    r = random.Random(31 * case["batch"] + case["past"] * 1009 + case["new"])
    got = []
    for i in range(case["batch"]):
        past, new = case["past"], case["new"]
        if case["spread"] != "full":
            past = r.randint(past // 8, past)
            new = r.randint(max(1, new // 8), new)
        if case["spread"] == "mixed" and i % 12 != 3:
            new = 1
        if case["spread"] == "holes" and i % 5 == 2:
            past = new = 0
        got.append((past, new))
    return got


def _evict_lengths(case):
    r = random.Random(31 * case["batch"] + case["length"])
    got = [case["length"] if case["spread"] == "full" else r.randint(max(1, case["length"] // 8), case["length"])
           for _ in range(case["batch"])]
    return [0 if case["spread"] == "holes" and i % 5 == 2 else n for i, n in enumerate(got)]


def _evicted(case, b, column, columns):
    """Whether a page of an attention case has been evicted before ("holes" only): a function of the case alone."""
    return case["spread"] == "holes" and 0 < column < columns - 2 and (column * 7 + b) % 3 == 0


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _prepare_evict(case, g, dev):
    i32 = dict(dtype=torch.int32, device=dev)
    lens, page, batch = _evict_lengths(case), case["page"], case["batch"]
    most = _pages(max(max(lens), 1), page) + 1
    ids = torch.randperm(batch * most, generator=g, device=dev).to(torch.int32).view(batch, most)
    # some pages left earlier, some have weight zero (no query ever looked at them): ties
    table = torch.where(torch.rand(batch, most, generator=g, device=dev) < 0.05, -1, ids)
    weights = torch.exp(2 * torch.randn(batch, most, generator=g, device=dev))
    weights = torch.where(torch.rand(batch, most, generator=g, device=dev) < 0.2, 0.0, weights)
    return dict(case, kv_lens=torch.tensor(lens, **i32), table=table.contiguous(), page_weights=weights.contiguous(),
                table_out=torch.empty_like(table), weights_out=torch.empty_like(weights),
                freed=torch.full((batch * most,), -1, **i32), counts=torch.empty(2, **i32))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1 + seed)
    if case["op"] == "evict":
        return _prepare_evict(case, g, dev)

    def normal(*shape, scale=1.0):
        t = torch.randn(*shape, generator=g, device=dev, dtype=_dtype(case))
        return t if scale == 1.0 else t * scale

    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case)
    past, new = zip(*_lengths(case))
    page, heads, batch = case["page"], case["heads"], case["batch"]
    lens = [p + n for p, n in zip(past, new)]
    columns = [_pages(n, page) for n in lens]
    most = max(max(columns), 1) + 1
    ids = torch.randperm(sum(columns) + 5, generator=g, device=dev).to(torch.int32)
    table = torch.full((batch, most), -1, **i32)
    rows = torch.repeat_interleave(torch.arange(batch, device=dev), torch.tensor(columns, device=dev))
    start = torch.tensor([0] + columns, device=dev).cumsum(0)
    table[rows, torch.arange(sum(columns), device=dev) - start[rows]] = ids[:sum(columns)]
    gone = [(b, c) for b in range(batch) for c in range(columns[b]) if _evicted(case, b, c, columns[b])]
    if gone:
        at = torch.tensor(gone, device=dev)
        table[at[:, 0], at[:, 1]] = -1
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    n_tokens = cu[-1] + (2 if cu[-1] % 3 == 0 else 0)   # some steps are padded: the last rows belong to no request
    positions = torch.zeros(n_tokens, **i32)
    for b in range(batch):
        positions[cu[b]:cu[b + 1]] = torch.arange(past[b], lens[b], **i32)
    s.update(lens=lens, cu=cu, n_tokens=n_tokens, table=table, kv_lens=torch.tensor(lens, **i32),
             cu_tokens=torch.tensor(cu, **i32), positions=positions,
             q_nope=normal(n_tokens, heads, case["d_nope"]), q_pe=normal(n_tokens, heads, case["d_rope"]),
             c_cache=normal(sum(columns) + 5, page, case["d_kv"]), kpe_cache=normal(sum(columns) + 5, page, case["d_rope"]),
             w=normal(heads * (case["d_nope"] + case["d_v"]), case["d_kv"], scale=1.0 / math.sqrt(case["d_kv"])))
    if case["op"] == "prefill":   # rows of no request are left as they were
        s["out"] = torch.zeros(n_tokens, heads, case["d_v"], dtype=_dtype(case), device=dev)
        s["lse"] = torch.zeros(n_tokens, heads, dtype=torch.float32, device=dev)
    else:
        s["lse"] = _plain_prefill(dict(s, only_lse=True))["lse"]   # the attention call before it returned this
        s["prior"] = torch.rand(batch, most, generator=g, device=dev)
        s["weights_out"] = torch.empty_like(s["prior"])
    if own:
        from head_latent_attention_rmsnorm_gb300 import mla
        s["dims"] = mla.dims(heads, case["d_kv"], case["d_nope"], case["d_rope"], case["d_v"], ROPE_BASE, EPS)
        make = mla.paged_prefill_workspace if case["op"] == "prefill" else mla.paged_weights_workspace
        s["workspace"] = make(s["dims"], n_tokens, s["c_cache"], table)
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _plain_prefill, "weights": _plain_weights, "evict": _plain_evict}[s["op"]](s)


def _run_own(s):
    from head_latent_attention_rmsnorm_gb300 import mla
    if s["op"] == "evict":
        e = mla.paged_evict(s["kv_lens"], s["table"], s["page_weights"], page_size=s["page"], keep_pages=s["keep"],
                            first_pages=s["first"], last_pages=s["last"], table_out=s["table_out"],
                            weights_out=s["weights_out"], freed=s["freed"], counts=s["counts"])
        return dict(table=s["table_out"], page_weights=s["weights_out"], freed=e.freed, counts=e.counts)
    if s["op"] == "prefill":
        out, lse = mla.paged_prefill(s["dims"], s["q_nope"], s["q_pe"], s["c_cache"], s["kpe_cache"], s["table"], s["kv_lens"],
                                     s["cu_tokens"], s["positions"], s["w"], out=s["out"], lse=s["lse"],
                                     workspace=s["workspace"])
        return dict(out=out, lse=lse)
    got = mla.paged_weights(s["dims"], s["q_nope"], s["q_pe"], s["lse"], s["c_cache"], s["kpe_cache"], s["table"], s["kv_lens"],
                            s["cu_tokens"], s["positions"], s["w"], prior=s["prior"], out=s["weights_out"],
                            workspace=s["workspace"])
    return dict(page_weights=got)


# ------------------------------------------------------------------ plain forms ----
def _turn(x, pos):
    """RoPE of x [n, ..., d] at positions pos [n]: the angles in 64 bits, the rotation in 32."""
    half = x.shape[-1] // 2
    inv = ROPE_BASE ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / x.shape[-1])
    a = pos.double().reshape([-1] + [1] * (x.dim() - 1)) * inv
    c, n = a.cos().float(), a.sin().float()
    x1, x2 = x[..., :half].float(), x[..., half:].float()
    return torch.cat([x1 * c - x2 * n, x2 * c + x1 * n], -1)


def _plain_scores(s, b, t0, t1):
    """Scores [heads, tokens, keys] of request b's tokens t0 .. t1, -inf where a token sees no key; the
    keys' latent rows."""
    heads, dn, dk, page, n = s["heads"], s["d_nope"], s["d_kv"], s["page"], s["lens"][b]
    w = s["w"].float().view(heads, -1, dk)[:, :dn]
    ids = s["table"][b, :_pages(n, page)].long()
    held = (ids >= 0).repeat_interleave(page)[:n]
    ids = ids.clamp(min=0)
    c = s["c_cache"][ids].reshape(-1, dk)[:n].float().masked_fill(~held[:, None], 0.0)
    r = s["kpe_cache"][ids].reshape(-1, s["d_rope"])[:n].float().masked_fill(~held[:, None], 0.0)
    pos = s["positions"][t0:t1].long()
    q = s["q_nope"][t0:t1].float().transpose(0, 1)
    if t1 - t0 > 64:   # the same products in the cheaper order: keys of each head, or absorbed queries
        scores = torch.matmul(q, torch.matmul(w, c.T))
    else:
        scores = torch.matmul(torch.matmul(q, w), c.T)
    scores += torch.matmul(_turn(s["q_pe"][t0:t1], pos).transpose(0, 1), r.T)
    scores *= 1.0 / math.sqrt(dn + s["d_rope"])
    seen = held[None] & (torch.arange(n, device=pos.device)[None] <= pos[:, None])
    return scores.masked_fill_(~seen[None], -math.inf), c


def _steps(s, b):
    """Request b's tokens, cut where its scores would take more than 2 GB."""
    t0, t1 = s["cu"][b], s["cu"][b + 1]
    step = max(1, 500000000 // max(1, s["heads"] * s["lens"][b]))
    return [(t, min(t + step, t1)) for t in range(t0, t1, step)]


def _plain_prefill(s):
    heads, dn, dk = s["heads"], s["d_nope"], s["d_kv"]
    wv = s["w"].float().view(heads, -1, dk)[:, dn:]
    out = s.get("out")
    lse = s["lse"] if "lse" in s else torch.zeros(s["n_tokens"], heads, dtype=torch.float32, device=wv.device)
    for b in range(s["batch"]):
        for t0, t1 in _steps(s, b):
            x, c = _plain_scores(s, b, t0, t1)
            top = x.amax(-1, keepdim=True).clamp(min=-1e30)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            lse[t0:t1] = (total.log() + top)[..., 0].T
            if s.get("only_lse"):
                continue
            x /= total.clamp(min=1e-30)
            if t1 - t0 > 64:
                o = torch.matmul(x, torch.matmul(c, wv.transpose(1, 2)))
            else:
                o = torch.matmul(torch.matmul(x, c), wv.transpose(1, 2))
            out[t0:t1] = o.transpose(0, 1).to(out.dtype)
    return dict(out=out, lse=lse)


def _plain_weights(s):
    page, got = s["page"], s["weights_out"]
    got.copy_(s["prior"])
    for b in range(s["batch"]):
        for t0, t1 in _steps(s, b):
            x, _ = _plain_scores(s, b, t0, t1)
            lse = s["lse"][t0:t1].T[..., None]
            x = (x - lse).exp_().masked_fill_(lse == -math.inf, 0.0).sum((0, 1))
            columns = _pages(s["lens"][b], page)
            x = torch.cat([x, x.new_zeros(columns * page - x.numel())])
            got[b, :columns] += x.view(columns, page).sum(-1)
    return dict(page_weights=got)


def _plain_evict(s):
    table, w = s["table"], s["page_weights"]
    batch, most = table.shape
    columns = (s["kv_lens"].long().clamp(0, most * s["page"]) + s["page"] - 1) // s["page"]
    col = torch.arange(most, device=table.device)[None]
    held = (col < columns[:, None]) & (table >= 0)
    may = held & (col >= s["first"]) & (col < columns[:, None] - s["last"])
    want = torch.minimum((held.sum(1) - s["keep"]).clamp(min=0), may.sum(1))
    order = torch.argsort(torch.where(may, w, math.inf), dim=1, stable=True)   # (no weight of a page is infinite here)
    rank = torch.empty_like(order).scatter_(1, order, col.expand(batch, most).contiguous())
    leave = may & (rank < want[:, None])
    s["table_out"].copy_(torch.where(leave, -1, table))
    s["weights_out"].copy_(torch.where(leave, 0.0, w))
    at = (leave.view(-1).cumsum(0) - 1)
    total = want.sum()
    freed = s["freed"]
    spare = torch.cat([freed, freed.new_zeros(1)])
    spare[torch.where(leave.view(-1), at, freed.numel())] = table.view(-1)
    freed.copy_(spare[:-1])
    s["counts"].copy_(torch.stack([total, total]))
    return dict(table=s["table_out"], page_weights=s["weights_out"], freed=freed, counts=s["counts"])


# ------------------------------------------------------------------------ costs ----
def work(case):
    if case["op"] == "evict":
        lens, page = _evict_lengths(case), case["page"]
        most = _pages(max(max(lens), 1), page) + 1
        total = case["batch"] * most
        gone = sum(max(0, min(_pages(n, page) - case["keep"], _pages(n, page) - case["first"] - case["last"])) for n in lens)
        # table and weights in and out, lengths in, the list of evicted pages out
        return dict(bytes=4.0 * (4 * total + len(lens) + gone + 2), flops=0.0)
    e = 4 if case["dtype"] == "f32" else 2
    h, dn, dv, dk, dr, page = (case[k] for k in ("heads", "d_nope", "d_v", "d_kv", "d_rope", "page"))
    moved = flops = 0.0
    for b, (past, new) in enumerate(_lengths(case)):
        n, columns = past + new, _pages(past + new, page)
        if not new:
            continue
        gone = sum(1 for c in range(columns) if _evicted(case, b, c, columns)) * page
        moved += (n - gone) * (dk + dr) * e + 4 * columns
        pairs = h * (new * (past - gone) + new * (new + 1) // 2 if past > gone else new * n // 2)
        if case["op"] == "prefill":   # the cheaper of the two forms, request by request
            flops += min(pairs * 2 * (2 * dk + dr) + h * new * 2 * dk * (dn + dv),
                         pairs * 2 * (dn + dr + dv) + h * (n - gone) * 2 * dk * (dn + dv))
            moved += new * h * (dn + dr + dv) * e + new * h * 4
        else:
            flops += min(pairs * 2 * (dk + dr) + h * new * 2 * dk * dn, pairs * 2 * (dn + dr) + h * (n - gone) * 2 * dk * dn)
            moved += new * h * (dn + dr) * e + new * h * 4 + 8 * columns
    moved += h * (dn + (dv if case["op"] == "prefill" else 0)) * dk * e
    return dict(bytes=float(moved), flops=float(flops))


# ------------------------------------------------- the definitions, in 64 bits ----
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "evict":
        return dict(table=None, page_weights=_exact_evict(s), freed=None, counts=None)
    dev = s["c_cache"].device
    h, dn, dv, dk, dr, page = (case[k] for k in ("heads", "d_nope", "d_v", "d_kv", "d_rope", "page"))
    w = s["w"].to(f64).view(h, dn + dv, dk)
    out = torch.zeros(s["n_tokens"], h, dv, dtype=f64, device=dev)
    lse = torch.zeros(s["n_tokens"], h, dtype=f64, device=dev)
    got = s["prior"].to(f64) if case["op"] == "weights" else None
    theta = torch.exp(-torch.arange(0, dr, 2, device=dev, dtype=f64) / dr * math.log(ROPE_BASE))
    for b, (past, new) in enumerate(_lengths(case)):
        n, t0 = past + new, s["cu"][b]
        if new == 0:
            continue
        ids = s["table"][b, :_pages(n, page)].to(torch.int64)
        keys = torch.arange(n, device=dev)
        keys = keys[ids[keys // page] >= 0]   # the keys that are still there
        slot = ids[keys // page] * page + keys % page
        c = s["c_cache"].view(-1, dk).index_select(0, slot).to(f64)
        r = s["kpe_cache"].view(-1, dr).index_select(0, slot).to(f64)
        step = max(1, 60000000 // n)
        for a in range(0, new, step):
            t = slice(t0 + a, t0 + min(a + step, new))
            pos = s["positions"][t].to(f64)
            hidden = keys[None] > s["positions"][t].to(torch.int64)[:, None]
            z = torch.polar(torch.ones(1, dtype=f64, device=dev), pos[:, None] * theta)
            for i in range(h):   # head by head
                x = s["q_pe"][t, i].to(f64)
                y = torch.complex(x[:, :dr // 2], x[:, dr // 2:]) * z
                x = s["q_nope"][t, i].to(f64) @ (c @ w[i, :dn].T).T + torch.cat([y.real, y.imag], -1) @ r.T
                x = (x / math.sqrt(dn + dr)).masked_fill_(hidden, -math.inf)
                if got is not None:
                    mass = torch.exp(x - s["lse"][t, i].to(f64)[:, None]).sum(0)
                    got[b].index_add_(0, keys // page, mass)
                    continue
                total = torch.logsumexp(x, -1)
                lse[t, i] = total
                out[t, i] = torch.exp(x - total[:, None]) @ (c @ w[i, dn:].T)
    return dict(page_weights=got) if got is not None else dict(out=out, lse=lse)


def _exact_evict(s):
    """The pages of least weight, request by request, on the host."""
    w, table, lens = s["page_weights"].double().cpu(), s["table"].cpu().tolist(), s["kv_lens"].tolist()
    value = w.tolist()
    for b, n in enumerate(lens):
        columns = _pages(n, s["page"])
        held = [c for c in range(columns) if table[b][c] >= 0]
        may = [c for c in held if s["first"] <= c < columns - s["last"]]
        for c in sorted(may, key=lambda c: (value[b][c], c))[:max(0, len(held) - s["keep"])]:
            w[b, c] = 0.0
    return w.to(s["kv_lens"].device)
